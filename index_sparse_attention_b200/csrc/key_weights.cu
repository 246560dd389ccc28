// key_weights.cu -- the attention weight every key has received in a forward pass
// (sparse_attn_key_weights): w[b][g][j] = sum over the group's heads h and the queries i that
// see j of P_ij = exp(scale q_i . k_j - lse_i).
//
// Mathematics: with the forward's lse no softmax state is needed; P is recomputed tile by tile
// and summed over its query side.  S^T = K Q^T puts a key on a TMEM lane, so the sum over
// queries is a sum along the columns one thread holds: no exchange between lanes, no atomics,
// one store per key, and a fixed order.
//
// B200 design: one persistent CTA per SM.  The work is a row of units, one 128 x 128 tile of
// one query head each: key tile after key tile (an item: 128 keys of one (batch, KV head)),
// inside it the query tiles of its list, inside them the heads of the group (which share the
// tile's masks).  CTA c of C takes units [U c / C, U (c + 1) / C), so that ragged lists and
// causal triangles load the SMs evenly.  An item inside one CTA is stored at once; the two ends
// of a CTA's range can be cut items, whose parts go to the workspace and are added by a second
// kernel in CTA order.
//   warp 0     TMA: an item's K tile and the Q tiles, several stages deep;
//   warp 1     tcgen05.mma S^T = K Q^T into one of four TMEM buffers;
//   warps 2-9  two warpgroups that take the units in turn (thread = key row):
//              exp2(S^T scale log2e - lse log2e) summed over the 128 queries.  A unit's lse
//              values (one per thread, fetched a unit ahead) pass through shared memory; the
//              presence words of index mode are transposed across the warp.  Each unit is summed
//              on its own before it joins the running sum, so that long query ranges do not lose
//              low bits.
// Every mbarrier wait is bounded (sa_device.cuh).
#include "sa_device.cuh"
#include "sa_kernels.h"

namespace sa {
namespace kweights {

constexpr int kThreads = 320;
constexpr int kMaxCtas = 256;

template <int DQK>
struct Cfg {
  static constexpr int kKStages = DQK <= 128 ? 2 : 1;
  static constexpr int kQStages = DQK == 64 ? 6 : DQK == 128 ? 4 : DQK == 192 ? 3 : 2;
  static constexpr int kPanel = 128 * 128;  // 64 columns x 128 rows
  static constexpr int kTile = 128 * DQK * 2;
  static constexpr int kQOff = kKStages * kTile;
  static constexpr int kLOff = kQOff + kQStages * kTile;  // lse [2 warpgroups][2][128]
  static constexpr int kXOff = kLOff + 2 * 2 * 128 * 4;   // part sums of warpgroup 1, [2][128]
  static constexpr int kFindOff = kXOff + 2 * 128 * 4;
  static constexpr int kBarOff = kFindOff + 80 * 4;
  static constexpr int kSmem = kBarOff + 256 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

enum : int { kBKF = 0, kBKE = 2, kBQF = 4, kBQE = 10, kBSF = 16, kBSE = 20, kBDrain = 24,
             kNumBars = 25 };

struct Args {
  AttnArgs t;
  const float* w_in;
  float* w_out;
  // workspace: the parts of cut items -- an item that begins in CTA c and goes on: tail[c],
  // then head[c + 1 ..]; fix[c]: that item (or -1) and the last CTA that holds a part of it
  float *head, *tail;  // [kMaxCtas][128]
  int2* fix;           // [kMaxCtas]
  int items, C, G;
};

// Place of a unit: item (key tile of a KV head), list entry, head of the group.
struct Cursor {
  int item, n, n_full;  // list entries of the item (> 0), the full ones
  int k, hh;
  int tile, tile_next;  // list entries k and k + 1
  const int32_t* list;
  __device__ __forceinline__ void open(const Args& a, int it, int kk) {
    item = it;
    n_full = __ldg(a.t.tcnt + 2 * static_cast<int64_t>(it));
    n = n_full + __ldg(a.t.tcnt + 2 * static_cast<int64_t>(it) + 1);
    list = a.t.tidx + static_cast<int64_t>(it) * a.t.Tm;
    k = kk;
    if (kk < n) {
      tile = __ldg(list + kk);
      tile_next = kk + 1 < n ? __ldg(list + kk + 1) : 0;
    }
  }
  // to the next unit; false past the last item
  __device__ __forceinline__ bool next(const Args& a) {
    if (++hh < a.G) return true;
    hh = 0;
    if (++k < n) {
      tile = tile_next;
      tile_next = k + 1 < n ? __ldg(list + k + 1) : 0;
      return true;
    }
    for (int i = item + 1; i < a.items; ++i) {
      open(a, i, 0);
      if (n > 0) return true;
    }
    return false;
  }
};

// This CTA's units, the item the first one lies in and the units before that item; called by
// the whole block, ends with a barrier.
struct Found {
  int64_t U, u0, u1, off;
  int item, C;
};
__device__ __forceinline__ Found find_range(const Args& a, int c, int* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.items + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, a.items), i1 = min(i0 + per, a.items);
  auto entries = [&](int i) {
    return __ldg(a.t.tcnt + 2 * static_cast<int64_t>(i)) +
           __ldg(a.t.tcnt + 2 * static_cast<int64_t>(i) + 1);
  };
  int mine = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) mine += entries(i);
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += t;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int t = sh[w];
    if (w < warp) before += t;
    total += t;
  }
  Found f;
  f.U = static_cast<int64_t>(total) * a.G;
  f.C = static_cast<int>(min64(a.C, f.U));
  f.u0 = c < f.C ? f.U * c / f.C : f.U;
  f.u1 = c < f.C ? f.U * (c + 1) / f.C : f.U;
  const int target = static_cast<int>(f.u0 / a.G);  // the entry that the first unit lies in
  int at = before + incl - mine;
  if (target >= at && target < at + mine) {
    for (int i = i0; i < i1; ++i) {
      const int t = entries(i);
      if (target < at + t) {
        sh[64] = i;
        sh[65] = at;
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  f.item = f.u0 < f.u1 ? sh[64] : 0;
  f.off = f.u0 < f.u1 ? static_cast<int64_t>(sh[65]) * a.G : 0;
  return f;
}

template <int DQK>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const Args ka) {
  using C = Cfg<DQK>;
  const AttnArgs& a = ka.t;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * kNumBars);
  volatile WaitCtl* ctl =
      reinterpret_cast<volatile WaitCtl*>(smem + C::kBarOff + 8 * kNumBars + 4);
  auto BAR = [&](int k) { return sbase + C::kBarOff + 8u * static_cast<uint32_t>(k); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int k = 0; k < kNumBars; ++k) mbar_init(BAR(k), k >= kBSE && k < kBSE + 4 ? 128 : 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const Found f = find_range(ka, cta, reinterpret_cast<int*>(smem + C::kFindOff));
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const int n_iter = static_cast<int>(f.u1 - f.u0);
  if (n_iter == 0 && threadIdx.x == 0) ka.fix[cta] = make_int2(-1, 0);
  Cursor cur{};
  if (n_iter > 0) {
    const int64_t r = f.u0 - f.off;
    cur.open(ka, f.item, static_cast<int>(r / ka.G));
    cur.hh = static_cast<int>(r - static_cast<int64_t>(cur.k) * ka.G);
  }
  int issued_q = 0, issued_k = 0;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    int item = -1;
    for (int it = 0; it < n_iter; ++it) {
      const int bg = cur.item / a.Tn, b = bg / a.HK, g = bg - b * a.HK;
      if (cur.item != item) {
        item = cur.item;
        const int ks = issued_k % C::kKStages, ku = issued_k / C::kKStages;
        if (!warp_wait(BAR(kBKE + ks), (ku & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(BAR(kBKF + ks), C::kTile);
          for (int c = 0; c < DQK / 64; ++c)
            tma_load_4d(sbase + ks * C::kTile + c * C::kPanel, &tm_k, BAR(kBKF + ks), c * 64,
                        (item - bg * a.Tn) * 128, g, b);
        }
        __syncwarp();
        ++issued_k;
      }
      const int st = it % C::kQStages, u = it / C::kQStages;
      if (!warp_wait(BAR(kBQE + st), (u & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
      const int m0 = __shfl_sync(0xFFFFFFFFu, cur.tile, 0) * 128;
      if (elect_one()) {
        mbar_arrive_expect_tx(BAR(kBQF + st), C::kTile);
        for (int c = 0; c < DQK / 64; ++c)
          tma_load_4d(sbase + C::kQOff + st * C::kTile + c * C::kPanel, &tm_q, BAR(kBQF + st),
                      c * 64, m0, g * ka.G + cur.hh, b);
      }
      __syncwarp();
      issued_q = it + 1;
      if (it + 1 < n_iter) cur.next(ka);
    }
    // the last arrivals on the stages' barriers have landed before the CTA may leave
    if (issued_q == n_iter) {
      for (int it = max(0, n_iter - C::kQStages); it < n_iter; ++it)
        if (!warp_wait(BAR(kBQE + it % C::kQStages), (it / C::kQStages) & 1, ctl, a.status,
                       a.wait_limit_ns))
          break;
      for (int k = max(0, issued_k - C::kKStages); k < issued_k; ++k)
        if (!warp_wait(BAR(kBKE + k % C::kKStages), (k / C::kKStages) & 1, ctl, a.status,
                       a.wait_limit_ns))
          break;
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = idesc_bf16(128, 128, 0, 0);
    int item = -1, part = -1;
    for (int it = 0; it < n_iter; ++it) {
      if (cur.item != item) {
        item = cur.item;
        ++part;
        if (!warp_wait(BAR(kBKF + part % C::kKStages), (part / C::kKStages) & 1, ctl, a.status,
                       a.wait_limit_ns))
          break;
      }
      const int st = it % C::kQStages, u = it / C::kQStages, sb = it & 3;
      if (!warp_wait(BAR(kBQF + st), u & 1, ctl, a.status, a.wait_limit_ns)) break;
      if (!warp_wait(BAR(kBSE + sb), ((it >> 2) & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
      tc_fence_after();
      const bool more = it + 1 < n_iter;
      if (more) cur.next(ka);
      const int ks = part % C::kKStages;
      const uint64_t kd = sw128_desc(sbase + ks * C::kTile, 16, 1024);
      const uint64_t qd = sw128_desc(sbase + C::kQOff + st * C::kTile, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < DQK / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kPanel + (kk & 3) * 32) >> 4;
          umma_ss(tmem + sb * 128, kd + off, qd + off, idesc, kk > 0 ? 1u : 0u);
        }
        umma_commit(BAR(kBSF + sb));
        umma_commit(BAR(kBQE + st));
        if (!more || cur.item != item) umma_commit(BAR(kBKE + ks));
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- exponentials and sums
    const int quarter = warp & 3, wg = (warp - 2) >> 2;
    const int r = quarter * 32 + lane;       // key row of the item = TMEM lane
    const int tq = (threadIdx.x - 64) & 127;  // the query of a unit whose lse this thread fetches
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* lbuf = reinterpret_cast<float*>(smem + C::kLOff) + wg * 256;
    float* xch = reinterpret_cast<float*>(smem + C::kXOff);
    const float sc = a.scale_log2;
    // `nxt` runs one of this warpgroup's units ahead of `cur` and fetches its lse
    float l_nxt = 0.f;
    Cursor nxt = cur;
    bool more = n_iter > 0;   // nxt is a unit of this CTA
    int it_n = 0;             // and its number
    auto fetch = [&]() {
      if (!more) return;
      const int bg = nxt.item / a.Tn, b = bg / a.HK, g = bg - b * a.HK;
      const int64_t i = static_cast<int64_t>(nxt.tile) * 128 + tq;
      // (a row past Sq, or one that saw no key, adds nothing: exp2(-inf))
      float l = -INFINITY;
      if (i < a.Sq)
        l = __ldg(a.lse + (static_cast<int64_t>(b) * a.HQ + g * ka.G + nxt.hh) * a.Sq + i);
      l_nxt = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
    };
    auto advance = [&](int by) {
      for (int x = 0; x < by && more; ++x) {
        ++it_n;
        more = it_n < n_iter && nxt.next(ka);
      }
    };
    advance(wg);
    fetch();
    uint32_t cm[4] = {0u, 0u, 0u, 0u};  // which of the tile's queries see this key
    int cm_item = -1, cm_k = -1;
    bool ok = true;
    int part = 0;
    int it = 0;
    int64_t start = f.off;  // first unit of the item
    bool cut_here = false;
    while (it < n_iter) {
      // ------------------------------------------------------------ one part: units of an item
      const int item = cur.item;
      const int64_t end = start + static_cast<int64_t>(cur.n) * ka.G;
      const int it_end = static_cast<int>(min64(end, f.u1) - f.u0);
      const int bg = item / a.Tn, nt = item - bg * a.Tn;
      const int64_t j = static_cast<int64_t>(nt) * 128 + r;
      const bool key_ok = j < a.Sk;
      float total = 0.f;
      for (; it < it_end; ++it) {
        if ((it & 1) == wg) {
          const int sb = it & 3;
          float* ls = lbuf + ((it >> 1) & 1) * 128;
          ls[tq] = l_nxt;
          advance(2);
          fetch();
          const bool partial = cur.k >= cur.n_full;
          if (partial && (cm_k != cur.k || cm_item != item)) {
            cm_k = cur.k;
            cm_item = item;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int64_t q0 = static_cast<int64_t>(cur.tile) * 128 + 32 * c;
              uint32_t x = key_ok ? 0xFFFFFFFFu : 0u;
              if (a.causal) {  // i >= j
                const int64_t lo = j - q0;
                x &= lo <= 0 ? 0xFFFFFFFFu : (lo >= 32 ? 0u : (0xFFFFFFFFu << lo));
              }
              if (a.mode == SA_MODE_BLOCK && a.bs == 64 && key_ok) {
                const int64_t mb = q0 / 64;
                if (!(mb < a.Mb &&
                      __ldg(a.mask + (static_cast<int64_t>(bg) * a.Mb + mb) * a.Nb + j / 64) != 0))
                  x = 0u;
              } else if (a.mode == SA_MODE_INDEX) {
                // lane L loads the presence word of query q0 + L over this warp's 32 keys; the
                // transpose leaves in lane L the word of key L over the 32 queries
                const int64_t i = q0 + lane;
                const int w = nt * 4 + quarter;
                const uint32_t bits =
                    (i < a.Sq && w < a.W)
                        ? __ldg(a.bitmap + (static_cast<int64_t>(bg) * a.Sq + i) * a.W + w)
                        : 0u;
                x &= warp_transpose32(bits, lane);
              }
              cm[c] = x;
            }
          }
          if (ok)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(BAR(kBSF + sb), (it >> 2) & 1, ctl, a.status,
                                                   a.wait_limit_ns));
          named_bar_sync(1 + wg, 128);  // the unit's lse values are in shared memory
          if (ok) {
            tc_fence_after();
            const float4* ls4 = reinterpret_cast<const float4*>(ls);
            float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t s[32];
              tmem_ld32(tl + sb * 128 + 32 * c, s);
              tmem_wait_ld();
              if (c == 3) {  // every column is read: the buffer is free
                tc_fence_before();
                mbar_arrive(BAR(kBSE + sb));
              }
              if (!partial) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 l = ls4[8 * c + e];
                  ps[0] += ex2(fmaf(__uint_as_float(s[4 * e]), sc, -l.x));
                  ps[1] += ex2(fmaf(__uint_as_float(s[4 * e + 1]), sc, -l.y));
                  ps[2] += ex2(fmaf(__uint_as_float(s[4 * e + 2]), sc, -l.z));
                  ps[3] += ex2(fmaf(__uint_as_float(s[4 * e + 3]), sc, -l.w));
                }
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 l = ls4[8 * c + e];
                  const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                  for (int t = 0; t < 4; ++t) {
                    const float p = ex2(fmaf(__uint_as_float(s[4 * e + t]), sc, -lv[t]));
                    ps[t] += ((cm[c] >> (4 * e + t)) & 1u) ? p : 0.f;
                  }
                }
              }
            }
            total += (ps[0] + ps[1]) + (ps[2] + ps[3]);
          }
        }
        if (it + 1 < n_iter) cur.next(ka);
      }
      // ------------------------------------------------------------ the part's sum
      float* xp = xch + (part & 1) * 128;
      if (wg == 1) xp[r] = total;
      named_bar_sync(3, 256);
      if (wg == 0) {
        total += xp[r];
        const bool begins = start >= f.u0, ends = end <= f.u1;
        if (begins && ends) {
          if (key_ok) {
            const int64_t at = static_cast<int64_t>(bg) * a.Sk + j;
            ka.w_out[at] = ka.w_in ? ka.w_in[at] + total : total;
          }
        } else if (begins) {
          ka.tail[cta * 128 + r] = total;
          cut_here = true;
          if (r == 0)
            ka.fix[cta] = make_int2(item, static_cast<int>((end * f.C - 1) / f.U));
        } else {
          ka.head[cta * 128 + r] = total;
        }
      }
      start = end;
      ++part;
    }
    if (n_iter > 0 && wg == 0 && r == 0 && !cut_here) ka.fix[cta] = make_int2(-1, 0);
  }

  tc_fence_before();
  __syncthreads();
  // Abort path: no warp issues anything past the barrier above.  Wait (with a limit) for the
  // copies and MMAs in flight before shared and tensor memory are released.
  if (ctl->abort) {
    if (warp == 0 && lane == 0) {
      for (int k = max(0, issued_k - C::kKStages); k < issued_k; ++k)
        mbar_wait_limited(BAR(kBKF + k % C::kKStages), (k / C::kKStages) & 1);
      for (int it = max(0, issued_q - C::kQStages); it < issued_q; ++it)
        mbar_wait_limited(BAR(kBQF + it % C::kQStages), (it / C::kQStages) & 1);
    }
    if (warp == 1) {
      tc_fence_after();
      if (elect_one()) {
        umma_commit(BAR(kBDrain));
        mbar_wait_limited(BAR(kBDrain), 0);
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Blocks c < C add the parts of the item that begins in CTA c and is cut; the others store the
// items that no query sees (32 items each).
__global__ void __launch_bounds__(128) key_weights_join_kernel(const Args ka) {
  const AttnArgs& a = ka.t;
  const int r = threadIdx.x, c = blockIdx.x;
  auto store = [&](int item, float sum) {
    const int bg = item / a.Tn;
    const int64_t j = static_cast<int64_t>(item - bg * a.Tn) * 128 + r;
    if (j >= a.Sk) return;
    const int64_t at = static_cast<int64_t>(bg) * a.Sk + j;
    ka.w_out[at] = ka.w_in ? ka.w_in[at] + sum : sum;
  };
  if (c < ka.C) {
    const int2 fx = ka.fix[c];
    if (fx.x < 0) return;
    float sum = ka.tail[c * 128 + r];
    for (int k = c + 1; k <= fx.y; ++k) sum += ka.head[k * 128 + r];
    store(fx.x, sum);
    return;
  }
  const int i0 = (c - ka.C) * 32;
  for (int i = i0; i < min(i0 + 32, ka.items); ++i)
    if (__ldg(a.tcnt + 2 * static_cast<int64_t>(i)) + __ldg(a.tcnt + 2 * static_cast<int64_t>(i) + 1) == 0)
      store(i, 0.f);
}

template <int DQK>
static int launch(const Args& a, const CUtensorMap& mq, const CUtensorMap& mk, cudaStream_t st) {
  using C = Cfg<DQK>;
  static PerDeviceOnce attr;
  const int rc = once_per_device(attr, [] {
    return cuda_error(cudaFuncSetAttribute(key_weights_kernel<DQK>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem),
                      "key weights smem attribute");
  });
  if (rc) return rc;
  key_weights_kernel<DQK><<<a.C, kThreads, C::kSmem, st>>>(mq, mk, a);
  return check_launch("key weights kernel launch");
}

}  // namespace kweights
}  // namespace sa

using namespace sa;

extern "C" size_t sparse_attn_key_weights_workspace_size(const sparse_attn_params* p) {
  if (!p || p->B <= 0 || p->HQ <= 0 || p->HK <= 0 || p->Sq <= 0 || p->Sk <= 0 || p->Dqk <= 0)
    return 0;
  return kweights::kMaxCtas * (2 * 128 * sizeof(float) + sizeof(int2));
}

extern "C" int sparse_attn_key_weights(const sparse_attn_params* p, const float* weights,
                                       float* weights_out, void* workspace,
                                       size_t workspace_bytes, sa_stream_t stream) {
  if (!p) return SA_ERR_INVALID;
  // the forward's checks, with the fields that are not read standing in for themselves
  sparse_attn_params fake = *p;
  fake.v = p->k;
  fake.o = const_cast<void*>(p->q);
  kweights::Args a{};
  int rc = fill_args(&fake, &a.t, false);
  if (rc) return rc;
  if (!weights_out) return SA_ERR_INVALID;
  const int64_t items = static_cast<int64_t>(p->B) * p->HK * a.t.Tn;
  if (items * a.t.Tm > 0x7FFFFFFF) return SA_ERR_UNSUPPORTED;
  const size_t need = sparse_attn_key_weights_workspace_size(p);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
    return SA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = check_stream_device(st);
  if (rc) return rc;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SA_ERR_CUDA;
  a.w_in = weights;
  a.w_out = weights_out;
  a.head = static_cast<float*>(workspace);
  a.tail = a.head + kweights::kMaxCtas * 128;
  a.fix = reinterpret_cast<int2*>(a.tail + kweights::kMaxCtas * 128);
  a.items = static_cast<int>(items);
  a.C = sms < kweights::kMaxCtas ? sms : kweights::kMaxCtas;
  a.G = p->HQ / p->HK;
  CUtensorMap mq, mk;
  if (!make_map(&mq, p->q, p->Dqk, p->Sq, p->HQ, p->B, 128)) return SA_ERR_CUDA;
  if (!make_map(&mk, p->k, p->Dqk, p->Sk, p->HK, p->B, 128)) return SA_ERR_CUDA;
  if (p->Dqk == 64) rc = kweights::launch<64>(a, mq, mk, st);
  else if (p->Dqk == 128) rc = kweights::launch<128>(a, mq, mk, st);
  else if (p->Dqk == 192) rc = kweights::launch<192>(a, mq, mk, st);
  else rc = kweights::launch<256>(a, mq, mk, st);
  if (rc) return rc;
  kweights::key_weights_join_kernel<<<static_cast<unsigned>(a.C + (a.items + 31) / 32), 128, 0, st>>>(a);
  return check_launch("key weights join kernel launch");
}
