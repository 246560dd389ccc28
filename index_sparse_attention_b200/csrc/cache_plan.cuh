// cache_plan.cuh -- how cache_attn_fwd splits its work over the CTAs and where the parts meet.
//
// The work is a row of units, one key tile each: first the prefix (for every KV head, every
// tile of query rows, the P keys), then the caches (for every sequence, every KV head, its
// own keys).  A run of units over one key set is a segment.  CTA c of C (at most U) takes the
// units [U c / C, U (c + 1) / C), so every CTA streams the same number of key tiles whatever the
// lengths are, and a segment that crosses a border is cut there.  A part (segment s, CTA c)
// writes its un-normalised output and its running max and sum to slot s + c: along the row
// of units each part has a larger s or a larger c than the one before, so no two share a
// slot, and the combining kernel finds a segment's parts from the same arithmetic.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "sa_device.cuh"

namespace sa {
namespace cache {

constexpr int kMaxCtas = 256;  // bound of C the workspace is sized for

struct Args {
  const __nv_bfloat16 *q, *k, *v, *kp, *vp;
  const int32_t* lens;
  __nv_bfloat16* o;
  float* lse;
  const float* w_in;
  float* w_out;
  // workspace: per prefix / cache part [slot][row] (max in log2 units, sum), [slot][row][Dv]
  // un-normalised output; scores (log2 units) [B][HQ][Sp] of the caches' keys
  float2 *ml_p, *ml_c;
  float *po_p, *po_c;
  float* scores;
  int B, HQ, HK, G, Dqk, Dv;
  int64_t S, P, Sp;  // Sp: row stride of scores
  int kn;            // keys of a unit
  int nb;            // sequences of one prefix row tile: rows g * nb + (b - nb * tile)
  int Rt;            // prefix row tiles per KV head
  int64_t Tp;        // prefix key tiles
  int rep_p, rep_c;    // copies of a part's rows in the TMEM lane quarters (4 or 1)
  int rows_p, rows_c;  // rows of a part
  int C;             // CTAs
  float scale_log2;
  int32_t* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ int64_t clamped_len(const Args& a, int b) {
  return min64(max64(static_cast<int64_t>(__ldg(a.lens + b)), 0), a.S);
}
__device__ __forceinline__ int64_t tiles_of(const Args& a, int64_t len) {
  return (len + a.kn - 1) / a.kn;
}
// CTAs that have work: no more than units, so that every CTA between a segment's first and
// last one holds a part of it
__device__ __forceinline__ int busy_ctas(const Args& a, int64_t U) {
  return static_cast<int>(min64(a.C, U));
}
// the CTA (of C busy ones) that holds unit u of U
__device__ __forceinline__ int cta_of(int64_t u, int64_t U, int C) {
  return static_cast<int>(((u + 1) * C - 1) / U);
}
__device__ __forceinline__ int64_t first_unit(int c, int64_t U, int C) { return U * c / C; }

// What the plan needs from the lengths, found by the whole block (`sh`: 66 int64 of shared
// memory).  total_tiles over all sequences; for the unit `u0` of CTA c the sequence it lies in
// and the tiles before that sequence.  Every thread of the block calls it; ends with a barrier.
struct Found {
  int64_t U, u0, u1, off;
  int b;
};
template <int kThreads>
__device__ __forceinline__ Found find_range(const Args& a, int c, int64_t* sh) {
  static_assert(kThreads % 32 == 0 && kThreads <= 1024, "block size");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = tid * per < a.B ? tid * per : a.B, b1 = b0 + per < a.B ? b0 + per : a.B;
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_of(a, clamped_len(a, b));
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t t = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += t;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t t = sh[w];
    if (w < warp) before += t;
    total += t;
  }
  Found f;
  const int64_t np = a.Tp * a.Rt * a.HK;
  f.U = np + total * a.HK;
  const int C = busy_ctas(a, f.U);
  f.u0 = c < C ? first_unit(c, f.U, C) : f.U;
  f.u1 = c < C ? first_unit(c + 1, f.U, C) : f.U;
  const int64_t target = f.u0 <= np ? 0 : (f.u0 - np) / a.HK;
  int64_t at = before + incl - mine;
  if (mine > 0 && target >= at && target < at + mine) {
    for (int b = b0; b < b1; ++b) {
      const int64_t t = tiles_of(a, clamped_len(a, b));
      if (target < at + t) {
        sh[64] = b;
        sh[65] = at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  f.b = total > 0 ? static_cast<int>(sh[64]) : 0;
  f.off = total > 0 ? sh[65] : 0;
  return f;
}

// One part's place while a CTA walks its units: segment, key tile, sequence.
struct Walk {
  bool prefix;
  int seg;         // prefix: hk * Rt + rt; cache: b * HK + hk
  int hk, rt, b;   // rt: prefix row tile; b: the sequence (cache)
  int64_t tile;    // key tile inside the segment
  int64_t tiles;   // of the segment
  int64_t keys;    // of the segment

  // the walk at unit u; off / first_b: tiles of all sequences before first_b, u lying in
  // first_b's segments (ignored for a prefix unit)
  __device__ __forceinline__ void init(const Args& a, int64_t u, int first_b, int64_t off) {
    const int64_t np = a.Tp * a.Rt * a.HK;
    prefix = u < np;
    if (prefix) {
      seg = static_cast<int>(u / a.Tp);
      tile = u - seg * a.Tp;
      hk = seg / a.Rt;
      rt = seg - hk * a.Rt;
      b = -1;
      tiles = a.Tp;
      keys = a.P;
    } else {
      b = first_b;
      keys = clamped_len(a, b);
      tiles = tiles_of(a, keys);
      const int64_t r = u - np - off * a.HK;
      hk = static_cast<int>(r / tiles);
      tile = r - hk * tiles;
      seg = b * a.HK + hk;
      rt = 0;
    }
  }
  // to the next unit (only called when there is one); true when it starts a segment
  __device__ __forceinline__ bool next(const Args& a) {
    if (++tile < tiles) return false;
    tile = 0;
    if (prefix) {
      ++seg;
      if (++rt < a.Rt) return true;
      rt = 0;
      if (++hk < a.HK) return true;
      prefix = false;
      b = -1;
      hk = a.HK - 1;
    }
    if (++hk < a.HK) {
      ++seg;
      return true;
    }
    hk = 0;
    do {
      ++b;
      keys = clamped_len(a, b);
    } while (keys == 0 && b + 1 < a.B);
    tiles = tiles_of(a, keys);
    seg = b * a.HK;
    return true;
  }
};

}  // namespace cache
}  // namespace sa
