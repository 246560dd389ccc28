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
// tile's masks).  CTA c takes the units that begin in its share of a line on which units and
// items' ends are as long as they take, so that ragged lists and causal triangles load the SMs
// evenly.  An item inside one CTA is stored at once; the two ends of a CTA's range can be cut
// items, whose parts go to the workspace and are added by a second kernel in CTA order.
//   warp 0     TMA: an item's K tile and the Q tiles, several stages deep;
//   warp 1     tcgen05.mma S^T = K Q^T into one of two to four TMEM buffers;
//   warps 2-17 exp2(S^T scale log2e - lse log2e), summed: thread = key row, a quarter of the
//              unit's 128 queries per warpgroup.  The presence words of index mode are
//              transposed across the warp, once for all heads of a tile.  Each unit is summed
//              on its own before it joins the running sum, so that long query ranges do not
//              lose low bits.
//   warp 18    feeds the units' lse values and list entries through shared memory.
// What bounds it: the special-function unit.  A unit's 16384 exponentials take an SM 1024 cycles
// (its MMAs 512 at head dim 128); measured 1300 to 1400 cycles a unit on long prompts (103 us for
// the causal prompt B=2 H=16 S=4096 D=128, 667 TFLOP/s of allowed pairs; 106 us for the
// block-sparse one with 32 / 8 heads, S=8192; 114 to 124 us for the index prompt with 32 / 4
// heads, S=4001, head dims 192/128: replayed graphs; 107, 115 and 126 us a call made from
// Python).  Tried and slower: a unit per warpgroup (a group stands idle while
// its buffer is refilled), eight warps with half a unit each and the next half's TMEM loads in
// flight (the remaining latency of a unit is shared by fewer warps), an eighth to a half of the
// exponentials by a polynomial of packed fused multiply-adds (equal to slower: the warps are
// short of issue slots and latency, not of that unit alone).
// Every mbarrier wait is bounded (sa_device.cuh).  The kernels start while the one ahead of them
// ends: what that one may still be writing (an lse that cache_attn_fwd joins, a caller's lists)
// is read by plain loads behind wait_previous_kernel(), never through the read-only path.
#include <type_traits>

#include "sa_device.cuh"
#include "sa_kernels.h"

namespace sa {
namespace kweights {

constexpr int kGroups = 4;                        // epilogue warpgroups
constexpr int kFeed = 2 + 4 * kGroups;            // the feeding warp
constexpr int kThreads = 32 * (kFeed + 1);
constexpr int kMaxCtas = 256;
constexpr int kNoLse = 1 << 30;  // added to a unit's list entry: some of its queries have no lse

template <int DQK>
struct Cfg {
  static constexpr int kKStages = DQK <= 128 ? 2 : 1;
  // Q stages and TMEM S buffers (and the lse slots): unit `it` uses number it % kStages of each,
  // so that one barrier tells the MMA warp that all are ready and one tells the epilogue that
  // its inputs are (each wait costs a warp 100 cycles even when the barrier is ready, each
  // commit 50, and MMAs do not queue up behind them: with a barrier for each a unit took 1000
  // cycles at head dim 128 for 545 cycles of MMAs)
  static constexpr int kStages = DQK <= 128 ? 4 : DQK == 192 ? 3 : 2;
  static constexpr int kPanel = 128 * 128;  // 64 columns x 128 rows
  static constexpr int kTile = 128 * DQK * 2;
  static constexpr int kQOff = kKStages * kTile;
  static constexpr int kLOff = kQOff + kStages * kTile;  // per slot: -lse [128] (log2 units)
  static constexpr int kDOff = kLOff + kStages * 128 * 4;  // per slot: query tile, list entry
  static constexpr int kXOff = kDOff + 4 * 8;             // part sums, [2][kGroups - 1][128]
  static constexpr int kFindOff = kXOff + 2 * (kGroups - 1) * 128 * 4;
  static constexpr int kBarOff = kFindOff + 48 * 8;
  static constexpr int kReadOff = kBarOff + 256;  // per epilogue warp: units read
  static constexpr int kSmem = kBarOff + 384 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

// kBFull: a unit's Q tile has landed (the producer) and its S buffer and lse slot have been
// read (by every epilogue warp, for the unit kStages before).  kBDone: its MMAs are done and its
// lse slot is filled (the feeding warp).  Every waiter waits for every unit in turn: a wait by
// parity that comes a phase early would be let through.
enum : int { kBKF = 0, kBKE = 2, kBFull = 4, kBDone = 8, kBDrain = 12, kNumBars = 13 };

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

// The units of one item that a CTA takes.  Every value is broadcast from lane 0, so that the
// compiler keeps them, and the descriptors and coordinates made from them, in uniform registers
// (a tcgen05.mma or TMA whose operands have to be moved there first waits for each move).
struct Part {
  int item, n, n_full;  // list entries of the item, the full ones
  int nt, b, h0;        // key tile, batch, first query head of the item
  int k, hh;            // list entry and head of the first unit
  int units;            // taken by this CTA
  const int32_t* list;
  __device__ __forceinline__ void open(const Args& a, int it, int64_t skip, int left) {
    item = __shfl_sync(0xFFFFFFFFu, it, 0);
    const int full = a.t.tcnt[2 * static_cast<int64_t>(item)];
    const int all = full + a.t.tcnt[2 * static_cast<int64_t>(item) + 1];
    n_full = __shfl_sync(0xFFFFFFFFu, full, 0);
    n = __shfl_sync(0xFFFFFFFFu, all, 0);
    list = a.t.tidx + static_cast<int64_t>(item) * a.t.Tm;
    const int bg = item / a.t.Tn;
    nt = item - bg * a.t.Tn;
    b = bg / a.t.HK;
    h0 = (bg - b * a.t.HK) * a.G;
    const int64_t most = static_cast<int64_t>(n) * a.G - skip;
    units = static_cast<int>(min64(most, left));
    k = static_cast<int>(skip / a.G);
    hh = static_cast<int>(skip - static_cast<int64_t>(k) * a.G);
    units = __shfl_sync(0xFFFFFFFFu, units, 0);
    k = __shfl_sync(0xFFFFFFFFu, k, 0);
    hh = __shfl_sync(0xFFFFFFFFu, hh, 0);
  }
  // the next item with units (there is one)
  __device__ __forceinline__ void next(const Args& a, int left) {
    int i = item;
    do {
      ++i;
      open(a, i, 0, left);
    } while (n == 0);
  }
};

// The query tiles of a part in the order of its units, 32 list entries at a time (a warp holds
// one per lane).
struct Tiles {
  int base, mine;
  __device__ __forceinline__ void start(const Part& p, int lane) {
    base = p.k;
    mine = base + lane < p.n ? p.list[base + lane] : 0;
  }
  __device__ __forceinline__ int at(const Part& p, int k, int lane) {
    if (k - base == 32) {
      base = k;
      mine = base + lane < p.n ? p.list[base + lane] : 0;
    }
    return __shfl_sync(0xFFFFFFFFu, mine, k - base);
  }
};

// The line the work lies on: a unit is kUnit long, and behind an item's units lies kEnd for what
// its end and the next one's start take.  In hundreds of cycles, measured: with units alone the
// CTAs with the most items, the short lists of a triangle's last key tiles, took 211 thousand
// cycles where others took 171 (block-sparse prompt with 32 / 8 heads, S=8192, D=128: 114 us;
// so 109).
constexpr int kUnit = 14, kEnd = 28;
__device__ __forceinline__ int64_t length_of(const Args& a, int64_t n) {
  return n > 0 ? n * a.G * kUnit + kEnd : 0;
}
// This CTA's units: n of them from unit `skip` of item `item` (skip may be the item's number of
// units: then they begin with the next item's); `at`: where that item begins on the line; q: what
// a CTA takes of the line, at least a unit, so that every CTA between an item's first and last
// one holds a part of it.  Called by the whole block, ends with a barrier.
struct Found {
  int64_t at, skip, q;
  int item, n;
};
__device__ __forceinline__ Found find_range(const Args& a, int c, int64_t* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.items + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, a.items), i1 = min(i0 + per, a.items);
  auto entries = [&](int i) {
    // (every other load depends on these)
    return ld_behind(a.t.tcnt + 2 * static_cast<int64_t>(i)) +
           ld_behind(a.t.tcnt + 2 * static_cast<int64_t>(i) + 1);
  };
  int64_t len = 0, num = 0;  // of this thread's items: length, list entries
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const int n = entries(i);
    num += n;
    len += length_of(a, n);
  }
  int64_t incl = len, incl_n = num;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, incl_n, d);
    if (lane >= d) {
      incl += x;
      incl_n += y;
    }
  }
  if (lane == 31) {
    sh[warp] = incl;
    sh[20 + warp] = incl_n;
  }
  __syncthreads();
  int64_t before = 0, before_n = 0, U = 0, all_n = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t x = sh[w], y = sh[20 + w];
    if (w < warp) {
      before += x;
      before_n += y;
    }
    U += x;
    all_n += y;
  }
  Found f{0, 0, 1, 0, 0};
  if (U == 0) return f;  // (the same on every thread)
  f.q = max64((U + a.C - 1) / a.C, kUnit);
  const int64_t x[2] = {min64(U, f.q * c), min64(U, f.q * (c + 1))};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    int64_t at = before + incl - len, at_n = before_n + incl_n - num;
    if (x[e] < U && x[e] >= at && x[e] < at + len) {
      for (int i = i0; i < i1; ++i) {
        const int n = entries(i);
        const int64_t l = length_of(a, n);
        if (x[e] < at + l) {
          sh[40 + 4 * e] = i;
          sh[41 + 4 * e] = at;
          sh[42 + 4 * e] = at_n;
          sh[43 + 4 * e] = n;
          break;
        }
        at += l;
        at_n += n;
      }
    }
  }
  __syncthreads();
  int64_t done[2];  // units before x[0] and x[1]
#pragma unroll
  for (int e = 1; e >= 0; --e) {
    if (x[e] >= U) {
      done[e] = all_n * a.G;
      continue;
    }
    f.item = static_cast<int>(sh[40 + 4 * e]);
    f.at = sh[41 + 4 * e];
    f.skip = min64(sh[43 + 4 * e] * a.G, (x[e] - f.at + kUnit - 1) / kUnit);
    done[e] = sh[42 + 4 * e] * a.G + f.skip;
  }
  f.n = static_cast<int>(done[1] - done[0]);
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
    for (int k = 0; k < kNumBars; ++k)
      mbar_init(BAR(k), k >= kBFull && k < kBFull + 4   ? 1 + 4 * kGroups
                        : k >= kBDone && k < kBDone + 4 ? 2
                                                        : 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  wait_previous_kernel();
  // (the join is not let in early: its blocks, waiting, slow the exponentials: 109 us for the
  // causal prompt against 103)
  const Found f = find_range(ka, cta, reinterpret_cast<int64_t*>(smem + C::kFindOff));
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const int n_iter = __shfl_sync(0xFFFFFFFFu, f.n, 0);
  if (n_iter == 0 && threadIdx.x == 0) ka.fix[cta] = make_int2(-1, 0);
  Part p{};
  if (n_iter > 0) {
    p.open(ka, f.item, f.skip, n_iter);
    if (p.units == 0) p.next(ka, n_iter);
  }
  int issued_q = 0, issued_k = 0;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    bool ok = true;
    for (int it = 0; ok && it < n_iter;) {
      const int ks = issued_k % C::kKStages, ku = issued_k / C::kKStages;
      if (!warp_wait(BAR(kBKE + ks), (ku & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(BAR(kBKF + ks), C::kTile);
        for (int c = 0; c < DQK / 64; ++c)
          tma_load_4d(sbase + ks * C::kTile + c * C::kPanel, &tm_k, BAR(kBKF + ks), c * 64,
                      p.nt * 128, p.h0 / ka.G, p.b);
      }
      __syncwarp();
      ++issued_k;
      Tiles tiles;
      tiles.start(p, lane);
      int k = p.k, hh = p.hh;
      for (int u = 0; u < p.units; ++u, ++it) {
        const int m0 = tiles.at(p, k, lane) * 128;
        const int st = it % C::kStages, su = it / C::kStages;
        if (!warp_wait(BAR(kBDone + st), (su & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(BAR(kBFull + st), C::kTile);
          for (int c = 0; c < DQK / 64; ++c)
            tma_load_4d(sbase + C::kQOff + st * C::kTile + c * C::kPanel, &tm_q, BAR(kBFull + st),
                        c * 64, m0, p.h0 + hh, p.b);
        }
        __syncwarp();
        issued_q = it + 1;
        if (++hh == ka.G) {
          hh = 0;
          ++k;
        }
      }
      if (ok && it < n_iter) p.next(ka, n_iter - it);
    }
    // the last arrivals on the stages' barriers have landed before the CTA may leave
    if (issued_q == n_iter) {
      for (int it = max(0, n_iter - C::kStages); it < n_iter; ++it)
        if (!warp_wait(BAR(kBDone + it % C::kStages), (it / C::kStages) & 1, ctl, a.status,
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
    int part = 0;
    bool ok = true;
    for (int it = 0; ok && it < n_iter; ++part) {
      const int ks = part % C::kKStages;
      if (!warp_wait(BAR(kBKF + ks), (part / C::kKStages) & 1, ctl, a.status, a.wait_limit_ns)) break;
      const uint64_t kd = sw128_desc(sbase + ks * C::kTile, 16, 1024);
      for (int u = 0; u < p.units; ++u, ++it) {
        const int st = it % C::kStages, su = it / C::kStages;
        ok = warp_wait(BAR(kBFull + st), su & 1, ctl, a.status, a.wait_limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = sw128_desc(sbase + C::kQOff + st * C::kTile, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kPanel + (kk & 3) * 32) >> 4;
            umma_ss(tmem + st * 128, kd + off, qd + off, idesc, kk > 0 ? 1u : 0u);
          }
          umma_commit(BAR(kBDone + st));
          if (u + 1 == p.units) umma_commit(BAR(kBKE + ks));
        }
        __syncwarp();
      }
      if (ok && it < n_iter) p.next(ka, n_iter - it);
    }
  } else if (warp == kFeed) {
    // ---------------------------------------------------------------- feeding warp
    // Four units at a time: their query tiles, list entries and lse values (in log2 units)
    // into the slots.  A row past Sq, or one that saw no key, adds nothing, whatever it holds:
    // exp2(s - inf) is 0 only for a score s that is a number below infinity, which rows of zeros
    // past Sq do not have with an infinite key, nor a caller's padded rows with anything in them.
    // So a unit with such rows is marked in its list entry, which makes it a masked one, with a
    // mask of its own (index mode's costs 5% more time where every ragged tile is marked; the
    // schedule of the whole loop changes by as much with where the mark is made and used).
    float* lse_s = reinterpret_cast<float*>(smem + C::kLOff);
    int2* desc = reinterpret_cast<int2*>(smem + C::kDOff);
    bool ok = true;
    Tiles tiles;
    tiles.start(p, lane);
    int k = p.k, hh = p.hh, left = p.units;
    for (int it = 0; ok && it < n_iter; it += 4) {
      float l[4][4];
      int2 d[4];
      int bits = 0;  // which units are masked by presence words, in which rows past Sq are 0
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (it + x >= n_iter) break;
        const int tile = tiles.at(p, k, lane);
        d[x] = make_int2(tile, k);
        bits |= (a.mode == SA_MODE_INDEX && k >= p.n_full) << x;
        const float* row = a.lse + (static_cast<int64_t>(p.b) * a.HQ + p.h0 + hh) * a.Sq;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int i = tile * 128 + 32 * y + lane;
          l[x][y] = i < a.Sq ? row[i] : -INFINITY;
        }
        if (++hh == ka.G) {
          hh = 0;
          ++k;
        }
        if (--left == 0 && it + x + 1 < n_iter) {
          p.next(ka, n_iter - (it + x + 1));
          tiles.start(p, lane);
          k = p.k;
          hh = p.hh;
          left = p.units;
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (it + x >= n_iter) break;
        const int st = (it + x) % C::kStages, u = (it + x) / C::kStages;
        ok = ok && warp_wait(BAR(kBFull + st), u & 1, ctl, a.status, a.wait_limit_ns);
        if (!ok) break;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          lse_s[st * 128 + 32 * y + lane] =
              l[x][y] == -INFINITY ? -INFINITY : l[x][y] * -1.4426950408889634f;
        bool none = false;
#pragma unroll
        for (int y = 0; y < 4; ++y)
          none |= l[x][y] == -INFINITY &&
                  (!(bits & (1 << x)) || d[x].x * 128 + 32 * y + lane < a.Sq);
        if (__any_sync(0xFFFFFFFFu, none)) d[x].y += kNoLse;
        if (lane == 0) desc[st] = d[x];
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(kBDone + st));
      }
    }
  } else {
    // ---------------------------------------------------------------- exponentials and sums
    const int quarter = warp & 3, wg = (warp - 2) >> 2;
    const int r = quarter * 32 + lane;  // key row of the item = TMEM lane
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float* lse_s = reinterpret_cast<const float*>(smem + C::kLOff);
    const int2* desc = reinterpret_cast<const int2*>(smem + C::kDOff);
    float* xch = reinterpret_cast<float*>(smem + C::kXOff);
    const float sc = a.scale_log2;
    if (n_iter > 0)  // every buffer is free at first
      for (int k = lane; k < C::kStages; k += 32) mbar_arrive(BAR(kBFull + k));
    uint32_t cm = 0u;  // which of the tile's queries [32 wg, 32 wg + 32) see this key
    bool ok = true, cut_here = false;
    int part = 0, it = 0;
    int64_t at = f.at;       // where the item begins on the line
    int64_t skip = f.skip;   // units of the item before this CTA's
    if (n_iter > 0 && p.item != f.item) {
      const int32_t* n = a.tcnt + 2 * static_cast<int64_t>(f.item);
      at += length_of(ka, n[0] + n[1]);
      skip = 0;
    }
    int left = n_iter;
    while (left > 0) {
      // ------------------------------------------------------------ one part: units of an item
      const int64_t all = static_cast<int64_t>(p.n) * ka.G;
      const int it_end = it + p.units;
      const int item = p.item, n_full = p.n_full, nt = p.nt, bg = p.item / a.Tn;
      const int64_t j = static_cast<int64_t>(nt) * 128 + r;
      const bool key_ok = j < a.Sk;
      float total = 0.f;
      int cm_k = -1;
      // (a warp whose wait gave up goes from part to part without work, so that the groups meet)
      for (; ok && it < it_end; ++it) {
        const int st = it % C::kStages;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(BAR(kBDone + st), (it / C::kStages) & 1, ctl,
                                               a.status, a.wait_limit_ns));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[32];
        tmem_ld32(tl + st * 128 + 32 * wg, s);
        const int2 d = desc[st];
        const bool partial = d.y >= n_full;
        if (partial && cm_k != d.y) {
          cm_k = d.y;
          const int64_t q0 = static_cast<int64_t>(d.x) * 128 + 32 * wg;
          cm = key_ok ? 0xFFFFFFFFu : 0u;
          if (a.causal) {  // i >= j
            const int64_t lo = j - q0;
            cm &= lo <= 0 ? 0xFFFFFFFFu : (lo >= 32 ? 0u : (0xFFFFFFFFu << lo));
          }
          if (a.mode == SA_MODE_BLOCK && a.bs == 64 && key_ok) {
            const int64_t mb = q0 / 64;
            if (!(mb < a.Mb &&
                  a.mask[(static_cast<int64_t>(bg) * a.Mb + mb) * a.Nb + j / 64] != 0))
              cm = 0u;
          } else if (a.mode == SA_MODE_INDEX) {
            // lane L loads the presence word of query q0 + L over this warp's 32 keys; the
            // transpose leaves in lane L the word of key L over the 32 queries
            const int64_t i = q0 + lane;
            const int w = nt * 4 + quarter;
            const uint32_t bits =
                (i < a.Sq && w < a.W)
                    ? a.bitmap[(static_cast<int64_t>(bg) * a.Sq + i) * a.W + w]
                    : 0u;
            cm &= warp_transpose32(bits, lane);
          }
          if (d.y >= kNoLse) {  // (this head's own rows)
            cm &= __ballot_sync(0xFFFFFFFFu, lse_s[st * 128 + 32 * wg + lane] != -INFINITY);
            cm_k = -1;
          }
        }
        const ulonglong2* ls2 = reinterpret_cast<const ulonglong2*>(lse_s + st * 128 + 32 * wg);
        uint64_t ps[2] = {0ull, 0ull};  // pairs of sums
        tmem_wait_ld();
        // Masked tiles: packed multiply-adds, and only what the key sees is added; the others:
        // scalar multiply-adds and packed sums (measured so: the compiler's schedules of the
        // four combinations differ by up to 6%).
        auto sweep = [&](auto masked) {
          constexpr bool kMasked = decltype(masked)::value;
          float seen[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float s0 = __uint_as_float(s[2 * e]), s1 = __uint_as_float(s[2 * e + 1]);
            const uint64_t l = (e & 1) ? ls2[e >> 1].y : ls2[e >> 1].x;
            if constexpr (kMasked) {
              const float2 t = unpack2(fma2(pack2(s0, s1), pack2(sc, sc), l));
              const float p0 = ex2(t.x), p1 = ex2(t.y);
              if (cm & (1u << (2 * e))) seen[(2 * e) & 3] += p0;
              if (cm & (2u << (2 * e))) seen[(2 * e + 1) & 3] += p1;
            } else {
              const float2 lv = unpack2(l);
              const float p0 = ex2(fmaf(s0, sc, lv.x)), p1 = ex2(fmaf(s1, sc, lv.y));
              ps[e & 1] = add2(ps[e & 1], pack2(p0, p1));
            }
          }
          if constexpr (kMasked) ps[0] = pack2(seen[0] + seen[1], seen[2] + seen[3]);
        };
        if (partial) sweep(std::true_type{});
        else sweep(std::false_type{});
        // S and lse are read.  One arrival for the warp: arrivals of 32 lanes on one barrier are
        // taken one after another, and 512 of them a unit cost more than its exponentials.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(kBFull + st));
        const float2 sum = unpack2(add2(ps[0], ps[1]));
        total += sum.x + sum.y;
      }
      // ------------------------------------------------------------ the part's sum
      float* xp = xch + (part & 1) * (kGroups - 1) * 128;
      if (wg > 0) xp[(wg - 1) * 128 + r] = total;
      named_bar_sync(1, 128 * kGroups);
      if (wg == 0) {
#pragma unroll
        for (int x = 0; x < kGroups - 1; ++x) total += xp[x * 128 + r];
        const bool begins = skip == 0, ends = skip + p.units == all;
        if (begins && ends) {
          if (key_ok) {
            const int64_t to = static_cast<int64_t>(bg) * a.Sk + j;
            ka.w_out[to] = ka.w_in ? ka.w_in[to] + total : total;
          }
        } else if (begins) {
          ka.tail[cta * 128 + r] = total;
          cut_here = true;
          if (r == 0)
            ka.fix[cta] = make_int2(item, static_cast<int>((at + (all - 1) * kUnit) / f.q));
        } else {
          ka.head[cta * 128 + r] = total;
        }
      }
      at += length_of(ka, p.n);
      skip = 0;
      ++part;
      left -= p.units;
      if (left > 0) p.next(ka, left);
    }
    // (for the abort path: the units whose S buffers this warp has read)
    if (lane == 0) reinterpret_cast<int*>(smem + C::kReadOff)[warp - 2] = it;
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
      // a Q tile's barrier also counts the readers of the unit that had its S buffer before:
      // for those that gave up there, the arrival is made here
      const int* read_s = reinterpret_cast<const int*>(smem + C::kReadOff);
      for (int it = max(0, issued_q - C::kStages); it < issued_q; ++it) {
        const uint32_t bar = BAR(kBFull + it % C::kStages);
        for (int w = 0; w < 4 * kGroups; ++w)
          if (it >= C::kStages && read_s[w] <= it - C::kStages) mbar_arrive(bar);
        mbar_wait_limited(bar, (it / C::kStages) & 1);
      }
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
  allow_next_kernel();
  wait_previous_kernel();
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
  for (int i = i0; i < min(i0 + 32, ka.items); ++i) {
    const int32_t* n = a.tcnt + 2 * static_cast<int64_t>(i);
    if (n[0] + n[1] == 0) store(i, 0.f);
  }
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
  return launch_early(key_weights_kernel<DQK>, dim3(a.C), dim3(kThreads), C::kSmem, st,
                      "key weights kernel launch", 1, mq, mk, a);
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
  if (partly_overlap(weights, static_cast<const float*>(weights_out),
                     static_cast<int64_t>(p->B) * p->HK * p->Sk))
    return SA_ERR_INVALID;
  const void* words[] = {p->lse, weights, weights_out, p->dev_status};
  for (const void* x : words)
    if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0) return SA_ERR_ALIGN;
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
  return launch_early(kweights::key_weights_join_kernel,
                      dim3(static_cast<unsigned>(a.C + (a.items + 31) / 32)), dim3(128), 0, st,
                      "key weights join kernel launch", 1, a);
}
