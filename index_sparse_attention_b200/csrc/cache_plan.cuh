// cache_plan.cuh -- how cache_attn_fwd splits its work over the CTAs and where the parts meet.
//
// The work is a row of key tiles: first the prefix (for every KV head, every tile of query rows,
// the P keys: all of one row tile before the next one's), then the caches (for every sequence,
// every KV head, its own keys).  A run of tiles over one key set is a segment.  On a line a tile is
// as long as it takes (wt_p, wt_c) and behind a segment's tiles lies a stretch `we` for what its
// end takes (reading O, joining its row copies, the next rows' start).  CTA c takes the tiles that
// begin in [q c, q (c + 1)) of that line (q: its length U over the number of CTAs), so that the
// CTAs end together whatever the lengths are, and a segment that crosses a border is cut there.
// (Counting tiles alone left the CTA with the shortest sequences behind: 12 segments of one tile in
// its 15 tiles, 75000 cycles against 43000.)  q is at least the longer tile: then every CTA between
// a segment's first and last one holds a part of it.  A part (segment s, CTA c) writes its un-
// normalised output and its running max and sum to slot s + c: along the line each part has a
// larger s or a larger c than the one before, so no two share a slot, and the joining kernel finds
// a segment's parts from the same arithmetic.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "sa_device.cuh"

namespace sa {
namespace cache {

constexpr int kMaxCtas = 256;  // bound of C the workspace is sized for
// From so many (sequence, query head) rows on the join gives a row one warp instead of four
// (8192 rows of two or three parts: 36 us with four warps, 17 with one; the whole call for 256
// sequences of 1024 keys 235 and 205).
constexpr int kJoinRows = 2048;
// From so many sequences on such a join takes their places on the line from the workspace; with
// fewer each warp adds up the lengths itself while the parts are computed (32 heads, D=128, the
// whole call: 128 sequences of 1024 keys 97.9 us from the workspace, 97.3 without; 256 of 64 keys
// with a prefix of 8192 95.5 either way; 1024 of 256 keys 223 and 262; 4096 of 128 keys 593 and
// 1128).
constexpr int kLineSeqs = 256;

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
  int64_t* line;  // [B + 1] the lengths before each sequence, for one KV head, and of all; or null
  int B, HQ, HK, G, Dqk, Dv;
  int64_t S, P, Sp;  // Sp: row stride of scores
  int kshift;        // log2 of the keys of a tile
  int nb;            // sequences of one prefix row tile: rows g * nb + (b - nb * tile)
  int Rt;            // prefix row tiles per KV head
  int64_t Tp;        // prefix key tiles
  int rep_p, rep_c;    // copies of a part's rows in the TMEM lane quarters (4 or 1)
  int rows_p, rows_c;  // rows of a part
  int C;             // CTAs
  int wt_p, wt_c, we;  // lengths on the plan's line: a prefix tile, a cache tile, a segment's end
  float scale_log2;
  int32_t* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ int64_t clamped_len(const Args& a, int b) {
  return min64(max64(static_cast<int64_t>(ld_behind(a.lens + b)), 0), a.S);
}
__device__ __forceinline__ int64_t tiles_of(const Args& a, int64_t len) {
  return (len + (1 << a.kshift) - 1) >> a.kshift;
}
// a segment's length on the line
__device__ __forceinline__ int64_t length_of(const Args& a, int64_t tiles, int wt) {
  return tiles > 0 ? tiles * wt + a.we : 0;
}
__device__ __forceinline__ int64_t prefix_length(const Args& a) {
  return length_of(a, a.Tp, a.wt_p) * a.Rt * a.HK;
}
// Quotient of non-negative numbers; 32-bit division where both fit (the 64-bit one takes several
// times as long, and half a dozen of them in a row 2 us of every call; out of line, since its
// copies would be most of a short kernel's code).
static __device__ __noinline__ int64_t quotient64(int64_t x, int64_t d) { return x / d; }
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t d) {
  if ((static_cast<uint64_t>(x | d) >> 32) == 0)
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(d);
  return quotient64(x, d);
}
// what a CTA takes of a line of U (see above)
__device__ __forceinline__ int64_t share_of(const Args& a, int64_t U) {
  return max64(quotient(U + a.C - 1, a.C), max(a.wt_p, a.wt_c));
}

// What the plan needs from the lengths, found by the whole block (`sh`: 72 int64 of shared
// memory): this CTA's n tiles begin with tile `tile` (which may be the one past the last: the
// next segment's first) of a prefix segment `seg`, or of KV head seg of sequence b (b < 0: prefix).
// Every thread of the block calls it; ends with a barrier.
struct Found {
  int64_t tile;
  int n, b, seg;
};
template <int kThreads>
__device__ __forceinline__ Found find_range(const Args& a, int c, int64_t* sh) {
  static_assert(kThreads % 32 == 0 && kThreads <= 1024, "block size");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t len = 0, tiles = 0;  // of this thread's sequences, for one KV head
  for (int b = b0; b < b1; ++b) {
    const int64_t t = tiles_of(a, clamped_len(a, b));
    tiles += t;
    len += length_of(a, t, a.wt_c);
  }
  int64_t incl = len, incl_t = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, incl_t, d);
    if (lane >= d) {
      incl += x;
      incl_t += y;
    }
  }
  if (lane == 31) {
    sh[warp] = incl;
    sh[32 + warp] = incl_t;
  }
  __syncthreads();
  int64_t before = 0, before_t = 0, total = 0, total_t = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t x = sh[w], y = sh[32 + w];
    if (w < warp) {
      before += x;
      before_t += y;
    }
    total += x;
    total_t += y;
  }
  if (c == 0 && a.line) {
    int64_t at = before + incl - len;
    for (int b = b0; b < b1; ++b) {
      a.line[b] = at;
      at += length_of(a, tiles_of(a, clamped_len(a, b)), a.wt_c);
    }
    if (tid == 0) a.line[a.B] = total;
  }
  const int64_t np = prefix_length(a), U = np + total * a.HK;
  Found f{0, 0, -1, 0};
  if (U == 0) return f;  // (the same on every thread)
  const int64_t q = share_of(a, U);
  const int64_t x[2] = {min64(U, q * c), min64(U, q * (c + 1))};
  // the sequences in whose segments the stretch begins and ends
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (x[e] < np || x[e] >= U) continue;
    const int64_t target = quotient(x[e] - np, a.HK);
    int64_t at = before + incl - len, at_t = before_t + incl_t - tiles;
    if (target >= at && target < at + len) {
      for (int b = b0; b < b1; ++b) {
        const int64_t t = tiles_of(a, clamped_len(a, b)), l = length_of(a, t, a.wt_c);
        if (target < at + l) {
          sh[64 + 3 * e] = b;
          sh[65 + 3 * e] = at;
          sh[66 + 3 * e] = at_t;
          break;
        }
        at += l;
        at_t += t;
      }
    }
  }
  __syncthreads();
  // the first tile that begins at x[e] or behind it, and the tiles before it
  int64_t done[2];
  const int64_t prefix_tiles = a.Tp * a.Rt * a.HK;
#pragma unroll
  for (int e = 1; e >= 0; --e) {
    if (x[e] >= U) {
      done[e] = prefix_tiles + total_t * a.HK;
    } else if (x[e] < np) {
      const int64_t l = length_of(a, a.Tp, a.wt_p), s = quotient(x[e], l);
      f.tile = min64(a.Tp, quotient(x[e] - s * l + a.wt_p - 1, a.wt_p));
      f.seg = static_cast<int>(s);
      f.b = -1;
      done[e] = s * a.Tp + f.tile;
    } else {
      f.b = static_cast<int>(sh[64 + 3 * e]);
      const int64_t t = tiles_of(a, clamped_len(a, f.b)), l = length_of(a, t, a.wt_c);
      const int64_t r = x[e] - np - sh[65 + 3 * e] * a.HK, h = quotient(r, l);
      f.tile = min64(t, quotient(r - h * l + a.wt_c - 1, a.wt_c));
      f.seg = static_cast<int>(h);
      done[e] = prefix_tiles + sh[66 + 3 * e] * a.HK + h * t + f.tile;
    }
  }
  f.n = static_cast<int>(done[1] - done[0]);
  return f;
}

// The place of a tile while a CTA walks its own: segment, key tile, sequence.
struct Walk {
  bool prefix;
  int seg;         // prefix: hk * Rt + rt; cache: b * HK + hk
  int hk, rt, b;   // rt: prefix row tile; b: the sequence (cache)
  int64_t tile;    // key tile inside the segment
  int64_t tiles;   // of the segment
  int64_t keys;    // of the segment

  // to the first tile of f (there is one)
  __device__ __forceinline__ void init(const Args& a, const Found& f) {
    prefix = f.b < 0;
    tile = f.tile;
    b = f.b;
    if (prefix) {
      seg = f.seg;
      hk = seg / a.Rt;
      rt = seg - hk * a.Rt;
      tiles = a.Tp;
      keys = a.P;
    } else {
      keys = clamped_len(a, b);
      tiles = tiles_of(a, keys);
      hk = f.seg;
      seg = b * a.HK + hk;
      rt = 0;
    }
    if (tile >= tiles) {
      tile = tiles - 1;
      next(a);
    }
  }
  // to the next tile (only called when there is one); true when it starts a segment
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
