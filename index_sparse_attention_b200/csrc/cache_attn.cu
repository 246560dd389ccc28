// cache_attn.cu -- attention of one new token per sequence over a prefix that the batch
// shares and each sequence's own cache (cache_attn_fwd).
//
// Mathematics: softmax attention of a row over the union of two key sets, from parts.  A part
// over a run of keys holds m = max s_j, l = sum exp(s_j - m), o = sum exp(s_j - m) v_j; parts
// join as m' = max m, l' = sum l exp(m - m'), o' = sum o exp(m - m') (fp32 throughout), and
// lse = m' + ln l', o = o' / l'.
//
// B200 design: three launches, each started while the one before it ends (programmatic dependent
// launch): the parts, their join, and, when asked for, the keys' weights from the stored scores.
// The parts kernel is one persistent CTA per SM over an even share of all key tiles
// (cache_plan.cuh), so that one long sequence, a ragged batch and a long prefix all fill the GPU:
//   warp 0     TMA: Q rows of a part, K tiles (two to five stages); warp 10: V tiles;
//   warp 1     tcgen05.mma: S = Q K^T into one of two TMEM buffers, O += P V with P read from TMEM;
//              S of the next tile is issued before P V of this one;
//   warps 2-9  softmax, two warps per TMEM lane quarter: scores, running maximum and sum, P (bf16)
//              over S, the part's end.
// A prefix part holds the query rows of up to 128 / group sequences (box {64, sequences, group} of
// one TMA load), a row tile, so a prefix tile is read once for all of them.  More sequences make
// more row tiles, each with its own pass over the prefix, and one that the L2 does not hold from
// pass to pass comes from HBM each time (64 sequences of 4 heads a group over 32768 keys: two
// passes, 134 of 1098 MB read).  A cache part holds the group's rows.
// An MMA has 128 rows: parts of up to 32 rows load their Q into all four lane quarters, and each
// quarter's copy takes a quarter of the tile's keys (P is 0 elsewhere), so that all eight softmax
// warps share the exponentials; the copies are added when the part ends.
// P is rounded to bf16 for the MMA, as the forward does (its sum is taken before in fp32).  The
// running maximum moves only when a row's exceeds it by 8 (factors up to 2^8 in P, O and l).
// What bounds it: HBM where the caches are long (64 sequences of 4096 keys, 8 KV heads, D=128:
// 164 us, 6.5 TB/s, the copy bandwidth measured on this GPU); the softmax warps' chain on prefix
// tiles of many rows (2200 cycles per 128 x 128 tile, of which the exponentials 1200 and the MMAs
// 1050: 256 sequences over a prefix of 8192 alone 56 us, of which a CTA's 28 tiles are 32 and the
// join of 8192 rows and the set-up the rest); the parts' ends where there are many short caches
// (one own key for each of those 256 sequences: 92 us in all; 4096 sequences of 128 keys 593 to
// 670 us on two GPUs, 328 us of bytes); on short calls the launches, the set-up (lengths, plan,
// first loads: about 5 us) and the join (3 us).
// Tried without gain: a third K stage; both softmax groups with a tile and an O of their own by
// turns (2250 cycles a tile again: then the MMA warp's waits and issues bound); an eighth to a
// half of the exponentials by polynomial (2% on prefix tiles); joining and weighing in one launch
// (1.5 to 3 us slower).
#include <type_traits>

#include "cache_plan.cuh"
#include "sa_kernels.h"

namespace sa {
namespace cache {

template <int DQK, int DV>
struct Cfg {
  // keys of a tile (at head dims 192/128 128 keys take all shared memory; with 64, a second Q
  // buffer and a third V stage: 32 sequences over 16384 keys 46.4 us against 38.8, 16 of 8192
  // 70.7 against 65.1)
  static constexpr int kN = DQK <= 192 ? 128 : 64;
  // Q buffers: part p uses buffer p % 2; from head dim 192 on there is one, in which the copies of
  // up to 16 rows take rows [0, 16) or [16, 32) of each lane quarter by turns
  static constexpr int kQBufs = DQK >= 192 ? 1 : 2;
  static constexpr int kKStages = DQK == 64 ? 5 : 2;  // (a third one measured no faster)
  static constexpr int kVStages = DQK == 64 ? 5 : 2;
  static constexpr int kQPanel = 128 * 128;  // 64 columns x 128 rows
  static constexpr int kKPanel = kN * 128;   // 64 columns x kN rows (V too)
  static constexpr int kQBytes = 128 * DQK * 2;
  static constexpr int kKBytes = kN * DQK * 2;
  static constexpr int kVBytes = kN * DV * 2;
  static constexpr int kKOff = kQBufs * kQBytes;
  static constexpr int kVOff = kKOff + kKStages * kKBytes;
  // What the two warps of a quarter exchange, two buffers of [2 warps][128 rows]: tile `it` puts
  // its row maxima into buffer it % 2.  The pair's barrier lies between a tile's writes and its
  // reads, and that of the next tile between those reads and the writes of the tile after it
  // (with one buffer nothing did: S of the next tile may be there before P of this one, and a
  // warp would write its next maximum while the other still had to read this one).  A part that
  // ends with tile `it` puts its row sums into the other buffer, whose last readers are past the
  // barrier of tile `it`, and reads them before a barrier that tile it + 1 lies behind.
  static constexpr int kXOff = kVOff + kVStages * kVBytes;
  static constexpr int kMOff = kXOff + 2048;  // a part's row maxima, [128]
  // where the four copies of a row meet at a part's end: [2 column halves][4][32 rows][kCols]
  static constexpr int kCols = DQK == 192 ? 16 : 32;
  static constexpr int kMergeOff = kMOff + 512;
  // (what find_range needs lies there too: every warp is past it when the first part ends)
  static constexpr int kFindOff = kMergeOff;
  static constexpr int kBarOff = kMergeOff + kCols * 1024;
  static constexpr int kSmem = kBarOff + 272;  // (the tiles' base is declared 1024-aligned)
  static constexpr int kThreads = 352;
  static constexpr uint32_t kOCol = 256;  // S / P buffers at columns 0 and 128
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kKStages <= 5 && kVStages <= 5, "barrier slots");
};

enum : int { kBQF = 0, kBQE = 2, kBKF = 4, kBKE = 9, kBVF = 14, kBVE = 19, kBSF = 24, kBPF = 26,
             kBOD = 28, kBDrain = 29, kBOF = 30, kNumBars = 31 };

// maps: Q for prefix row tiles and for one sequence, K / V of the prefix and of the caches
struct Maps {
  CUtensorMap qp, qc, kp, vp, kc, vc;
};

template <int DQK, int DV>
__global__ void __launch_bounds__(352, 1)
    cache_part_kernel(const __grid_constant__ Maps maps, const Args a) {
  using C = Cfg<DQK, DV>;
  constexpr int kN = C::kN;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * kNumBars);
  volatile WaitCtl* ctl =
      reinterpret_cast<volatile WaitCtl*>(smem + C::kBarOff + 8 * kNumBars + 4);
  auto BAR = [&](int k) { return sbase + C::kBarOff + 8u * static_cast<uint32_t>(k); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int k = 0; k < kNumBars; ++k) mbar_init(BAR(k), k == kBPF || k == kBPF + 1 ? 256 : 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 10 && lane == 0) {
    prefetch_tensormap(&maps.qc);
    prefetch_tensormap(&maps.kc);
    prefetch_tensormap(&maps.vc);
    if (a.P > 0) {
      prefetch_tensormap(&maps.qp);
      prefetch_tensormap(&maps.kp);
      prefetch_tensormap(&maps.vp);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  wait_previous_kernel();
  if (warp == 10 && lane < 2 && a.P > 0) {
    // HBM has nothing to do while the plan is made: the head of an even share of the prefix goes
    // to L2 meanwhile (16 sequences over 8192 keys 37.5 -> 36.4 us; as much before the wait, and
    // 16 to 128 KB, within 0.4 us)
    const int64_t bytes = a.P * a.HK * (lane ? DV : DQK) * 2;
    const int64_t share = (bytes / a.C + 15) / 16 * 16, at = share * cta;
    const int64_t n = min64(min64(share, bytes - at), 64 * 1024);
    if (n > 0)
      prefetch_l2(reinterpret_cast<const char*>(lane ? a.vp : a.kp) + at, static_cast<uint32_t>(n));
  }
  const Found f = find_range<C::kThreads>(
      a, cta, reinterpret_cast<int64_t*>(smem + C::kFindOff));  // (ends with a barrier)
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const int n_iter = f.n;
  Walk w{};
  if (n_iter > 0) w.init(a, f);
  int issued_k = 0, issued_v = 0, issued_q = 0;  // loads issued (the abort path drains the last)

  if (warp == 0) {
    // ---------------------------------------------------------------- Q and K producer
    if (cta == 0)  // lengths out of range are reported once
      for (int b = lane; b < a.B; b += 32) {
        const int n = ld_behind(a.lens + b);
        if (n < 0 || n > a.S) report_status(a.status, kStatusIndex);
      }
    bool first = true, was_full = false;
    for (int it = 0; it < n_iter; ++it) {
      const int ks = it % C::kKStages, ku = it / C::kKStages;
      if (!warp_wait(BAR(kBKE + ks), (ku & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(BAR(kBKF + ks), C::kKBytes);
        const int k0 = static_cast<int>(w.tile) * kN;
        for (int c = 0; c < DQK / 64; ++c)
          tma_load_4d(sbase + C::kKOff + ks * C::kKBytes + c * C::kKPanel,
                      w.prefix ? &maps.kp : &maps.kc, BAR(kBKF + ks), c * 64, k0, w.hk,
                      w.prefix ? 0 : w.b);
      }
      __syncwarp();
      issued_k = it + 1;
      if (first) {
        const int qs = issued_q & 1, qu = issued_q >> 1;
        const int rep = w.prefix ? a.rep_p : a.rep_c, rows = w.prefix ? a.rows_p : a.rows_c;
        const bool full = rep == 1 || rows > 16;  // (a whole buffer)
        if (!warp_wait(BAR(kBQE + qs), (qu & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
        // one buffer: a part that takes all of it, or follows one that does, waits for that too
        if (C::kQBufs == 1 && issued_q > 0 && (full || was_full) &&
            !warp_wait(BAR(kBQE + (qs ^ 1)), ((issued_q - 1) >> 1) & 1, ctl, a.status,
                       a.wait_limit_ns))
          break;
        was_full = full;
        if (elect_one()) {
          mbar_arrive_expect_tx(BAR(kBQF + qs), rep * rows * DQK * 2);
          const uint32_t dst = sbase + (C::kQBufs == 2 ? qs * C::kQBytes : full ? 0 : qs * 16 * 128);
          for (int r = 0; r < rep; ++r)
            for (int c = 0; c < DQK / 64; ++c)
              tma_load_4d(dst + c * C::kQPanel + r * 32 * 128, w.prefix ? &maps.qp : &maps.qc,
                          BAR(kBQF + qs), c * 64, w.prefix ? w.rt * a.nb : w.b, w.hk * a.G, 0);
        }
        __syncwarp();
        ++issued_q;
      }
      if (it + 1 < n_iter) first = w.next(a);
    }
    // every arrival on the stages' barriers has landed before the CTA may leave
    if (issued_k == n_iter) {
      for (int it = max(0, n_iter - C::kKStages); it < n_iter; ++it)
        if (!warp_wait(BAR(kBKE + it % C::kKStages), (it / C::kKStages) & 1, ctl, a.status,
                       a.wait_limit_ns))
          break;
      for (int q = max(0, issued_q - 2); q < issued_q; ++q)
        if (!warp_wait(BAR(kBQE + (q & 1)), (q >> 1) & 1, ctl, a.status, a.wait_limit_ns)) break;
    }
  } else if (warp == 10) {
    // ---------------------------------------------------------------- V producer
    for (int it = 0; it < n_iter; ++it) {
      const int vs = it % C::kVStages, vu = it / C::kVStages;
      if (!warp_wait(BAR(kBVE + vs), (vu & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(BAR(kBVF + vs), C::kVBytes);
        const int k0 = static_cast<int>(w.tile) * kN;
        for (int c = 0; c < DV / 64; ++c)
          tma_load_4d(sbase + C::kVOff + vs * C::kVBytes + c * C::kKPanel,
                      w.prefix ? &maps.vp : &maps.vc, BAR(kBVF + vs), c * 64, k0, w.hk,
                      w.prefix ? 0 : w.b);
      }
      __syncwarp();
      issued_v = it + 1;
      if (it + 1 < n_iter) w.next(a);
    }
    if (issued_v == n_iter)
      for (int it = max(0, n_iter - C::kVStages); it < n_iter; ++it)
        if (!warp_wait(BAR(kBVE + it % C::kVStages), (it / C::kVStages) & 1, ctl, a.status,
                       a.wait_limit_ns))
          break;
    // (P V's own barrier, which the softmax warps wait for only where they rescale)
    if (issued_v == n_iter && n_iter > 0)
      warp_wait(BAR(kBOD), (n_iter - 1) & 1, ctl, a.status, a.wait_limit_ns);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16(128, kN, 0, 0);
    constexpr uint32_t idesc_o = idesc_bf16(128, DV, 0, 1);
    int part = 0;                 // part of the S being issued
    bool first_s = true, first_o = true;
    Walk wo = w;                  // the walk of the P V being issued (one tile behind)
    auto issue_s = [&](int it) -> bool {
      const int ks = it % C::kKStages, ku = it / C::kKStages;
      const int qs = part & 1, qu = part >> 1;
      if (first_s && !warp_wait(BAR(kBQF + qs), qu & 1, ctl, a.status, a.wait_limit_ns)) return false;
      if (!warp_wait(BAR(kBKF + ks), ku & 1, ctl, a.status, a.wait_limit_ns)) return false;
      tc_fence_after();
      const uint64_t kd = sw128_desc(sbase + C::kKOff + ks * C::kKBytes, 16, 1024);
      const uint64_t qd = sw128_desc(sbase + (C::kQBufs == 2 ? qs * C::kQBytes : 0), 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < DQK / 16; ++kk)
          umma_ss(tmem + (it & 1) * 128, qd + (((kk >> 2) * C::kQPanel + (kk & 3) * 32) >> 4),
                  kd + (((kk >> 2) * C::kKPanel + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
        umma_commit(BAR(kBSF + (it & 1)));
        umma_commit(BAR(kBKE + ks));
      }
      __syncwarp();
      const bool ends = it + 1 >= n_iter || w.next(a);  // the part's last tile
      if (ends) {
        if (elect_one()) umma_commit(BAR(kBQE + qs));
        __syncwarp();
      }
      first_s = ends;
      if (ends) ++part;
      return true;
    };
    bool ok = n_iter > 0 && issue_s(0);
    for (int it = 0; ok && it < n_iter; ++it) {
      // the next S before this P V, so that the softmax has its next tile; at a part's end
      // after it, because the epilogue waits for O and then takes longer than S
      const bool last = first_s;
      if (!last && it + 1 < n_iter && !issue_s(it + 1)) break;
      const int vs = it % C::kVStages, vu = it / C::kVStages;
      // (V first: it has long come when P has, and a wait costs 150 cycles)
      if (!warp_wait(BAR(kBVF + vs), vu & 1, ctl, a.status, a.wait_limit_ns)) break;
      if (!warp_wait(BAR(kBPF + (it & 1)), (it >> 1) & 1, ctl, a.status, a.wait_limit_ns)) break;
      tc_fence_after();
      const uint64_t vd = sw128_desc(sbase + C::kVOff + vs * C::kVBytes, C::kKPanel, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kN / 16; ++kk)
          umma_ts(tmem + C::kOCol, tmem + (it & 1) * 128 + kk * 8, vd + ((kk * 2048) >> 4), idesc_o,
                  (!first_o || kk > 0) ? 1u : 0u);
        umma_commit(BAR(kBOD));
        umma_commit(BAR(kBVE + vs));
        if (last) umma_commit(BAR(kBOF));  // the part's O is complete
      }
      __syncwarp();
      if (it + 1 < n_iter) first_o = wo.next(a);
      if (last && it + 1 < n_iter && !issue_s(it + 1)) break;
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int quarter = warp & 3, hc = (warp - 2) >> 2;
    const int pair_bar = 1 + quarter;  // the two warps of a TMEM lane quarter
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + C::kXOff);
    const int r = quarter * 32 + lane;
    float m_run = -INFINITY, l_run = 0.f;
    bool first = true, ok = true;
    int part = 0;
    auto both = [&](bool v) { return named_bar_and(pair_bar, 64, v); };
    // One tile: S columns [c0, c0 + NC) of this thread's row -> P.  kRep: the row's copy in
    // this quarter takes the quarter's kN / 4 columns, the others' P is zero.
    auto tile = [&](auto nc, bool rep, int it, bool active, int loff) -> bool {
      constexpr int NC = decltype(nc)::value;
      const int sb = it & 1;
      const uint32_t scol = tl + sb * 128;
      const int c0 = rep ? quarter * (kN / 4) + hc * NC : hc * NC;
      const int k0 = static_cast<int>(w.tile) * kN;
      const int lim = static_cast<int>(min64(kN, w.keys - k0));
      const bool there = __all_sync(0xFFFFFFFFu, mbar_wait(BAR(kBSF + sb), (it >> 1) & 1, ctl,
                                                           a.status, a.wait_limit_ns));
      tc_fence_after();
      uint32_t u[NC];
      if constexpr (NC >= 32) {
#pragma unroll
        for (int j = 0; j < NC / 32; ++j) tmem_ld32(scol + c0 + 32 * j, u + 32 * j);
      } else if constexpr (NC == 16) {
        tmem_ld16(scol + c0, u);
      } else {
        tmem_ld8(scol + c0, u);
      }
      tmem_wait_ld();
      float x[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) x[c] = __uint_as_float(u[c]);
      if (lim < kN) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (c0 + c >= lim) x[c] = -INFINITY;
      }
      const float sc = a.scale_log2;
      if (a.scores && !w.prefix && active && there) {
        const int g = rep ? lane - loff : r;
        float4* dst = reinterpret_cast<float4*>(
            a.scores + (static_cast<int64_t>(w.b) * a.HQ + w.hk * a.G + g) * a.Sp + k0 + c0);
#pragma unroll
        for (int e = 0; e < NC / 4; ++e)
          dst[e] = make_float4(x[4 * e] * sc, x[4 * e + 1] * sc, x[4 * e + 2] * sc,
                               x[4 * e + 3] * sc);
      }
      float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c + 4 < NC; c += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mx4[e] = max3(mx4[e], x[c + e], x[c + 4 + e]);
      }
      if constexpr (NC % 8 == 0) {  // (four are left over)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(mx4[e], x[NC - 4 + e]);
      }
      float mx = max3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]) * sc;
      float* xm = xch + (it & 1) * 256;
      xm[hc * 128 + r] = mx;
      // both warps have read their S columns past this barrier: P may be written over them
      // (one whose wait gave up has read what was there, and both leave)
      if (!both(there)) return false;
      mx = fmaxf(xm[r], xm[128 + r]);
      const bool need = active && mx > m_run + 8.0f;
      const float alpha = need ? ex2(m_run - mx) : 1.f;
      if (__any_sync(0xFFFFFFFFu, need)) {
        // O holds P V up to the tile before: rescale this warp's O columns.  (A wait by parity
        // needs the barrier in that phase or the next: P V of tile it - 2 was queued before
        // S of tile it, which is done, and P V of this tile waits for the P below.)
        if (!first) {
          if (!both(__all_sync(0xFFFFFFFFu, mbar_wait(BAR(kBOD), (it - 1) & 1, ctl, a.status,
                                                      a.wait_limit_ns))))
            return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = hc * (DV / 2); c < (hc + 1) * (DV / 2); c += 32) {
            uint32_t ov[32];
            tmem_ld32(tl + C::kOCol + c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tl + C::kOCol + c, ov);
          }
          tmem_wait_st();
        }
        if (need) {
          l_run *= alpha;
          m_run = mx;
        }
      }
      const float m_eff = m_run == -INFINITY ? 0.f : m_run;
      uint64_t ps[2] = {0ull, 0ull};  // pairs of sums
      uint32_t pk[NC / 2];
#pragma unroll
      for (int e = 0; e < NC / 2; ++e) {
        const float2 t =
            unpack2(fma2(pack2(x[2 * e], x[2 * e + 1]), pack2(sc, sc), pack2(-m_eff, -m_eff)));
        const float p0 = ex2(t.x), p1 = ex2(t.y);
        ps[e & 1] = add2(ps[e & 1], pack2(p0, p1));
        pk[e] = pack_bf16x2(p0, p1);
      }
      const float2 sum = unpack2(add2(ps[0], ps[1]));
      l_run += sum.x + sum.y;
      if constexpr (NC >= 32) {
#pragma unroll
        for (int j = 0; j < NC / 32; ++j) tmem_st16(scol + (c0 >> 1) + 16 * j, pk + 16 * j);
      } else {
        // this warp writes the P chunks of its parity: its own, and zeros in the other quarters'
        uint32_t z[NC / 2];
#pragma unroll
        for (int e = 0; e < NC / 2; ++e) z[e] = 0u;
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const uint32_t at = scol + (2 * qq + hc) * (NC / 2);
          const uint32_t* src = qq == quarter ? pk : z;
          if constexpr (NC == 16) tmem_st8(at, src);
          else tmem_st4(at, src);
        }
      }
      return true;
    };
    for (int it = 0; it < n_iter; ++it) {
      const bool rep = (w.prefix ? a.rep_p : a.rep_c) > 1;
      const int rows = w.prefix ? a.rows_p : a.rows_c;
      // where the copies' rows begin in each lane quarter
      const int loff = C::kQBufs == 1 && rep && rows <= 16 ? 16 * (part & 1) : 0;
      const int mine = rep ? lane - loff : r;
      const bool active = mine >= 0 && mine < rows;
      // (after a wait that gave up the loop goes on without work, so that the warps still meet
      // at the barriers of a part's end)
      if (ok)
        ok = rep ? tile(std::integral_constant<int, kN / 8>{}, true, it, active, loff)
                 : tile(std::integral_constant<int, kN / 2>{}, false, it, active, 0);
      const int lim = static_cast<int>(min64(kN, w.keys - w.tile * kN));
      if (ok && !w.prefix && lim < kN) {
        // the V rows behind the sequence hold anything, and 0 x NaN is NaN: clear them
        const int vs = it % C::kVStages, vu = it / C::kVStages;
        ok = both(__all_sync(0xFFFFFFFFu, mbar_wait(BAR(kBVF + vs), vu & 1, ctl, a.status,
                                                    a.wait_limit_ns)));
        if (ok) {
          uint8_t* vt = smem + C::kVOff + vs * C::kVBytes;
          const int n = (kN - lim) * (DV / 8);
          for (int e = threadIdx.x - 64; e < n; e += 256) {
            const int row = lim + e / (DV / 8), ch = e % (DV / 8);
            *reinterpret_cast<uint4*>(vt + (ch >> 3) * C::kKPanel + row * 128 + (ch & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
      }
      if (ok) {
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(kBPF + (it & 1)));
      }
      const Walk at = w;
      first = it + 1 == n_iter || w.next(a);
      if (first) {
        // ------------------------------------------------------------ a part ends
        if (ok)
          // (a barrier of its own, one phase per part: P V of the tile before may still wait for
          // its V here, and the other barrier would then be a phase early)
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(BAR(kBOF), part & 1, ctl, a.status,
                                                 a.wait_limit_ns));
        ++part;
        float* xs = xch + ((it + 1) & 1) * 256;
        if (hc == 1) xs[128 + r] = l_run;
        ok = named_bar_and(8, 256, ok);
        if (!ok) continue;
        tc_fence_after();
        const int64_t slot = at.seg + cta;
        float2* mls = (at.prefix ? a.ml_p : a.ml_c) + slot * rows;
        float* po = (at.prefix ? a.po_p : a.po_c) + slot * rows * DV;
        if (!rep) {
          if (active && hc == 0) mls[r] = make_float2(m_run, l_run + xs[128 + r]);
          named_bar_sync(pair_bar, 64);  // (the next tile's maxima go where the sum was)
#pragma unroll 1
          for (int c = hc * (DV / 2); c < (hc + 1) * (DV / 2); c += 32) {
            uint32_t ov[32];
            tmem_ld32(tl + C::kOCol + c, ov);
            tmem_wait_ld();
            if (active) {
              float* dst = po + static_cast<int64_t>(r) * DV + c;
#pragma unroll
              for (int e = 0; e < 4; ++e) st_global_v8(dst + 8 * e, ov + 8 * e);
            }
          }
        } else {
          // the four copies of a row (each over its own keys) become one result
          float* xm = reinterpret_cast<float*>(smem + C::kMOff);
          if (hc == 0) {
            xm[r] = m_run;
            xs[r] = l_run + xs[128 + r];
          }
          // (behind it nothing reads the second half of xs; the first half is read by a warp that
          // meets the writers of the next tile's maxima there, the hc == 0 warps, when they merge)
          named_bar_sync(5, 256);
          float mm = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) mm = fmaxf(mm, xm[32 * q + lane]);
          const float me = mm == -INFINITY ? 0.f : mm;
          const float f = ex2(m_run - me);
          if (active && quarter == 0 && hc == 0) {
            float l = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              l += xs[32 * q + lane] * ex2(xm[32 * q + lane] - me);
            mls[mine] = make_float2(mm, l);
          }
          // up to eight rows: all columns of this half at once, else kCols at a time
          constexpr int kCols = C::kCols;
          static_assert(kCols * 512 >= 4 * 8 * (DV / 2) * 4, "eight rows, half the columns");
          float* stage = reinterpret_cast<float*>(smem + C::kMergeOff + hc * kCols * 512);
          const int cp = rows <= 8 ? DV / 2 : kCols;
#pragma unroll 1
          for (int c0 = hc * (DV / 2); c0 < (hc + 1) * (DV / 2); c0 += cp) {
            if (c0 != hc * (DV / 2)) named_bar_sync(6 + hc, 128);  // the last pass is read
#pragma unroll 1
            for (int c = 0; c < cp; c += kCols) {
              uint32_t ov[kCols];
              if constexpr (kCols == 32) tmem_ld32(tl + C::kOCol + c0 + c, ov);
              else tmem_ld16(tl + C::kOCol + c0 + c, ov);
              tmem_wait_ld();
              if (active) {
                float4* dst = reinterpret_cast<float4*>(stage + (quarter * rows + mine) * cp + c);
#pragma unroll
                for (int e = 0; e < kCols / 4; ++e)  // (turned by the row: bank conflicts)
                  dst[e ^ (mine & (kCols / 4 - 1))] = make_float4(
                      __uint_as_float(ov[4 * e]) * f, __uint_as_float(ov[4 * e + 1]) * f,
                      __uint_as_float(ov[4 * e + 2]) * f, __uint_as_float(ov[4 * e + 3]) * f);
              }
            }
            named_bar_sync(6 + hc, 128);
            const int per = cp / 4;  // float4 of a row
            for (int e = quarter * 32 + lane; e < rows * per; e += 128) {
              const int row = e / per, ch = e - row * per;
              float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 x = *reinterpret_cast<const float4*>(
                    stage + (q * rows + row) * cp + 4 * (ch ^ (row & (kCols / 4 - 1))));
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
              }
              *reinterpret_cast<float4*>(po + static_cast<int64_t>(row) * DV + c0 + 4 * ch) = o;
            }
          }
        }
        tc_fence_before();
        m_run = -INFINITY;
        l_run = 0.f;
      }
    }
  }

  allow_next_kernel();  // (not before: the join's blocks, waiting, would take issue slots)
  tc_fence_before();
  __syncthreads();
  // Abort path: no warp issues anything past the barrier above.  Wait (with a limit) for the
  // copies and MMAs in flight before shared and tensor memory are released.
  if (ctl->abort) {
    if (lane == 0 && warp == 0) {
      for (int q = max(0, issued_q - 2); q < issued_q; ++q)
        mbar_wait_limited(BAR(kBQF + (q & 1)), (q >> 1) & 1);
      for (int it = max(0, issued_k - C::kKStages); it < issued_k; ++it)
        mbar_wait_limited(BAR(kBKF + it % C::kKStages), (it / C::kKStages) & 1);
    }
    if (lane == 0 && warp == 10)
      for (int it = max(0, issued_v - C::kVStages); it < issued_v; ++it)
        mbar_wait_limited(BAR(kBVF + it % C::kVStages), (it / C::kVStages) & 1);
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

// ------------------------------------------------------------------------------------
// join: kW warps per (sequence, query head) row, 4 / kW rows per block.  Every warp finds the
// parts' common maximum and sum (one part per lane), then takes every kW-th part's output, four
// loads in flight.  Few rows have many parts (up to one per CTA) and take four warps each; from
// kJoinRows rows on the blocks are many and the parts few, and a warp does a row.
// ------------------------------------------------------------------------------------
constexpr int kJoin = 128;

// An infinite value v_jd makes a row's column d infinite, however small p_j is, but the products
// of the parts hold 0 x infinity = NaN too: a row's copies meet every key of a tile, with P = 0
// where another copy has it, and P or a rescaling underflows.  So where a part's column is NaN
// though the row's probabilities are numbers, the largest and the smallest of its values decide:
// this gives their sum where they are no numbers (NaN with a NaN or both infinities), 0 if all
// are.  A warp looks at 32 columns of n keys, whose rows begin at v; this lane's answer is for
// column 8 (lane % 4) + lane / 4.  Rarely called (never on finite values), so it is kept
// short, with 16 keys in flight: eight loads per lane instead of two cost every call registers
// and instruction fetches (8 sequences over a prefix of 4097 at D=256 34.0 us against 32.9, 4096
// sequences of 128 keys 692 against 659).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
__device__ __forceinline__ float column_of_specials(const __nv_bfloat16* v, int64_t n,
                                                    int64_t pitch) {
  const int lane = threadIdx.x & 31;
  uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};  // pairs of bf16
  v += 8 * (lane & 3);
#pragma unroll 1
  for (int64_t j = lane >> 2; j < n; j += 16) {
    uint4 x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      x[e] = j + 8 * e < n ? __ldcg(reinterpret_cast<const uint4*>(v + (j + 8 * e) * pitch))
                           : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t y[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[i] = max_bf16x2(hi[i], y[i]);
        lo[i] = min_bf16x2(lo[i], y[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll 1
    for (int d = 4; d < 32; d <<= 1) {
      hi[i] = max_bf16x2(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], d));
      lo[i] = min_bf16x2(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], d));
    }
  const int i = lane >> 3;
  const uint32_t hw = i < 2 ? (i ? hi[1] : hi[0]) : (i < 3 ? hi[2] : hi[3]);
  const uint32_t lw = i < 2 ? (i ? lo[1] : lo[0]) : (i < 3 ? lo[2] : lo[3]);
  const float p = __uint_as_float(lane & 4 ? hw & 0xFFFF0000u : hw << 16);
  const float m = __uint_as_float(lane & 4 ? lw & 0xFFFF0000u : lw << 16);
  return (p < INFINITY ? 0.f : p) + (m > -INFINITY ? 0.f : m);
}

template <int DV, int kW>
__global__ void __launch_bounds__(kJoin) cache_join_kernel(const Args a) {
  constexpr int kD = DV / 32, kRows = 4 / kW;
  __shared__ float sh_o[kW > 1 ? kW : 1][DV];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = kW > 1 ? tid >> 5 : 0;
  allow_next_kernel();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (kW > 1 ? 0 : tid >> 5);
  if (row >= static_cast<int64_t>(a.B) * a.HQ) return;  // (kW == 1 only: a whole warp)
  const int b = static_cast<int>(row / a.HQ), h = static_cast<int>(row - static_cast<int64_t>(b) * a.HQ);
  const int hk = h / a.G, g = h - hk * a.G;
  // the plan's line up to this sequence and in all
  int64_t before = 0, total = 0;
  const bool summed = kW == 1 && a.line;
  if (summed) {
    wait_previous_kernel();
    before = a.line[b];
    total = a.line[a.B];
  } else {
    for (int x = lane; x < a.B; x += 32) {
      const int64_t t = length_of(a, tiles_of(a, clamped_len(a, x)), a.wt_c);
      total += t;
      if (x < b) before += t;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
      total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    }
  }
  const int64_t np = prefix_length(a), U = np + total * a.HK;
  const int64_t q = share_of(a, U);
  const int64_t tb = tiles_of(a, clamped_len(a, b));
  // parts of the prefix (of this row's tile) and of the own cache: rows of ml / po, `step` apart
  int n_p = 0, n_c = 0;
  int64_t at_p = 0, at_c = 0;
  if (np > 0) {
    const int rt = b / a.nb;
    const int64_t seg = static_cast<int64_t>(hk) * a.Rt + rt;
    const int64_t x = seg * length_of(a, a.Tp, a.wt_p);
    const int c0 = static_cast<int>(quotient(x, q));
    const int c1 = static_cast<int>(quotient(x + (a.Tp - 1) * a.wt_p, q));
    n_p = c1 - c0 + 1;
    at_p = (seg + c0) * a.rows_p + g * a.nb + (b - rt * a.nb);
  }
  if (tb > 0) {
    const int64_t x = np + before * a.HK + hk * length_of(a, tb, a.wt_c);
    const int c0 = static_cast<int>(quotient(x, q));
    const int c1 = static_cast<int>(quotient(x + (tb - 1) * a.wt_c, q));
    n_c = c1 - c0 + 1;
    at_c = (static_cast<int64_t>(b) * a.HK + hk + c0) * a.rows_c + g;
  }
  const int n = n_p + n_c;
  auto ml_of = [&](int i) {
    return i < n_p ? a.ml_p + at_p + static_cast<int64_t>(i) * a.rows_p
                   : a.ml_c + at_c + static_cast<int64_t>(i - n_p) * a.rows_c;
  };
  auto po_of = [&](int i) {
    return i < n_p ? a.po_p + (at_p + static_cast<int64_t>(i) * a.rows_p) * DV
                   : a.po_c + (at_c + static_cast<int64_t>(i - n_p) * a.rows_c) * DV;
  };
  if (!summed) wait_previous_kernel();
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, ml_of(i)->x);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  const float me = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[kD];
#pragma unroll
  for (int e = 0; e < kD; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    // of part i0 + lane (0: a part without keys; else a normal number, which an infinity in the
    // part's output outlasts)
    float f = 0.f;
    if (i0 + lane < n) {
      const float2 v = *ml_of(i0 + lane);
      if (v.y != 0.f) {
        f = ex2(fmaxf(v.x - me, -126.f));
        l += v.y * f;
      }
    }
    const int left = min(32, n - i0);
    for (int x = warp; x < left; x += 4 * kW) {
      float v[4][kD], fx[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int i = x + y * kW;
        fx[y] = __shfl_sync(0xFFFFFFFFu, f, i & 31);
        if (i >= left) fx[y] = 0.f;
        if (fx[y] != 0.f) {
          const float* po = po_of(i0 + i);
#pragma unroll
          for (int e = 0; e < kD; ++e) v[y][e] = po[e * 32 + lane];
        }
      }
#pragma unroll
      for (int y = 0; y < 4; ++y)
        if (fx[y] != 0.f) {
#pragma unroll
          for (int e = 0; e < kD; ++e) acc[e] = fmaf(v[y][e], fx[y], acc[e]);
        }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  bool bad = false;
  if constexpr (kW > 1) {
#pragma unroll
    for (int e = 0; e < kD; ++e) sh_o[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    for (int d = tid; d < DV; d += kJoin) {
      float o = 0.f;
#pragma unroll
      for (int x = 0; x < kW; ++x) o += sh_o[x][d];
      o *= inv;
      bad |= o != o;
      a.o[row * DV + d] = __float2bfloat16(o);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kD; ++e) {
      const float o = acc[e] * inv;
      bad |= o != o;
      a.o[row * DV + e * 32 + lane] = __float2bfloat16(o);
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && l == l) {
    // The infinities of the parts' columns add up, and the keys of those that are NaN are looked
    // at again: a long row's parts are many (131072 keys with one infinity: 0.3 ms, with a look
    // at all of them 5.6).  With a warp per row at all keys of the two sets: the places of few
    // and short parts are not worth the code (4096 sequences of 128 finite keys 682 us with it).
    const int64_t pitch = static_cast<int64_t>(a.HK) * DV;
    __syncwarp();  // (the warp's own stores are read back)
#pragma unroll 1
    for (int d = warp * 32; d < DV; d += kW * 32) {
      const int col = d + 8 * (lane & 3) + (lane >> 2);
      __nv_bfloat16* o = a.o + row * DV + col;
      float sum = __hisnan(*o) ? 0.f : __uint_as_float(0x7FC00000u);  // (NaN: nothing to do)
#pragma unroll 1
      for (int i = 0; i < (kW > 1 ? n : 2) && __any_sync(0xFFFFFFFFu, sum == sum); ++i) {
        const bool prefix = i < (kW > 1 ? n_p : 1);
        const int64_t keys = prefix ? a.P : clamped_len(a, b);
        int64_t j0 = 0, j1 = keys;
        float x = __uint_as_float(0x7FC00000u);
        if constexpr (kW > 1) {
          if (ml_of(i)->y == 0.f) continue;
          x = po_of(i)[col];
          // the part's tiles: those that begin in its CTA's share of the line
          const int wt = prefix ? a.wt_p : a.wt_c;
          const int64_t at = prefix ? (static_cast<int64_t>(hk) * a.Rt + b / a.nb) *
                                          length_of(a, a.Tp, a.wt_p)
                                    : np + before * a.HK + hk * length_of(a, tb, a.wt_c);
          const int64_t c = quotient64(at, q) + (prefix ? i : i - n_p);
          j0 = quotient64(max64(c * q - at, 0) + wt - 1, wt) << a.kshift;
          j1 = min64(quotient64((c + 1) * q - at + wt - 1, wt) << a.kshift, keys);
        }
        if (__any_sync(0xFFFFFFFFu, x != x && sum == sum)) {
          const float y = column_of_specials(
              (prefix ? a.vp : a.v + b * a.S * pitch) + j0 * pitch + hk * DV + d, j1 - j0, pitch);
          if (x != x) x = y;
        }
        if (x - x != 0.f) sum += x;
      }
      // (none at all: finite values overflowed, and NaN stays)
      if (__hisnan(*o) && sum != 0.f) *o = __float2bfloat16(sum);
    }
  }
  if (lane == 0 && warp == 0)
    a.lse[row] = l == 0.f ? -INFINITY : (me + __log2f(l)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------------------------
// weights: one thread per key of a (sequence, KV head) sums the group's probabilities from the
// scores that the parts kernel stored (fp32, log2 units) and the joined lse.  A few microseconds,
// launch-bound: 16 sequences of 2049 keys, 32 heads, read 4 MB that the L2 holds.
// ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) cache_weights_kernel(const Args a) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int hk = blockIdx.y, b = blockIdx.z;
  allow_next_kernel();
  if (j >= a.S) return;  // (a block that leaves early has nothing to wait for)
  const int64_t at = (static_cast<int64_t>(b) * a.HK + hk) * a.S + j;
  const bool live = j < clamped_len(a, b);
  wait_previous_kernel();
  if (!live && a.w_in == a.w_out) return;
  float w = a.w_in ? a.w_in[at] : 0.f;
  if (live) {
    const int64_t r0 = static_cast<int64_t>(b) * a.HQ + hk * a.G;
    float sum = 0.f;
    for (int g = 0; g < a.G; ++g) {
      const float lse = a.lse[r0 + g];
      // (lse is -inf only where every score is)
      if (lse != -INFINITY)
        sum += ex2(a.scores[(r0 + g) * a.Sp + j] - lse * 1.4426950408889634f);
    }
    w += sum;
  }
  a.w_out[at] = w;
}

template <int DQK, int DV>
static int launch(const Args& a, cudaStream_t st) {
  using C = Cfg<DQK, DV>;
  static PerDeviceOnce attr;
  int rc = once_per_device(attr, [] {
    return cuda_error(cudaFuncSetAttribute(cache_part_kernel<DQK, DV>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem),
                      "cache attention smem attribute");
  });
  if (rc) return rc;
  Maps m;
  if (!make_map(&m.qc, a.q, DQK, a.B, a.HQ, 1, 1, a.G) ||
      !make_map(&m.kc, a.k, DQK, a.S, a.HK, a.B, C::kN) ||
      !make_map(&m.vc, a.v, DV, a.S, a.HK, a.B, C::kN))
    return SA_ERR_CUDA;
  m.qp = m.qc;
  m.kp = m.kc;
  m.vp = m.vc;
  if (a.P > 0 && (!make_map(&m.qp, a.q, DQK, a.B, a.HQ, 1, a.nb, a.G) ||
                  !make_map(&m.kp, a.kp, DQK, a.P, a.HK, 1, C::kN) ||
                  !make_map(&m.vp, a.vp, DV, a.P, a.HK, 1, C::kN)))
    return SA_ERR_CUDA;
  rc = launch_early(cache_part_kernel<DQK, DV>, dim3(a.C), dim3(C::kThreads), C::kSmem, st,
                    "cache attention kernel launch", 1, m, a);
  if (rc) return rc;
  const int64_t rows = static_cast<int64_t>(a.B) * a.HQ;
  rc = rows < kJoinRows
           ? launch_early(cache_join_kernel<DV, 4>, dim3(static_cast<unsigned>(rows)), dim3(kJoin), 0,
                          st, "cache join kernel launch", 1, a)
           : launch_early(cache_join_kernel<DV, 1>, dim3(static_cast<unsigned>((rows + 3) / 4)),
                          dim3(kJoin), 0, st, "cache join kernel launch", 1, a);
  if (rc || !a.w_out) return rc;
  return launch_early(cache_weights_kernel, dim3(static_cast<unsigned>((a.S + 255) / 256), a.HK, a.B),
                      dim3(256), 0, st, "cache weights kernel launch", 1, a);
}

static size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The plan's sizes and the workspace's layout; returns its bytes.  Partial outputs are stored in
// 32-byte pieces (st_global_v8): the layout begins at the first 32-byte boundary of a workspace
// that need only be 16-byte aligned.
static size_t lay_out(const cache_attn_params* p, Args* a, char* ws) {
  if (ws) ws += reinterpret_cast<uintptr_t>(ws) & 16u;
  a->B = p->B;
  a->HQ = p->HQ;
  a->HK = p->HK;
  a->G = p->HQ / p->HK;
  a->Dqk = p->Dqk;
  a->Dv = p->Dv;
  a->S = p->S;
  a->P = p->P;
  a->kshift = p->Dqk <= 192 ? 7 : 6;
  a->Sp = (p->S + 127) / 128 * 128;
  a->nb = 128 / a->G;
  if (a->nb > p->B) a->nb = p->B;
  a->Rt = (p->B + a->nb - 1) / a->nb;
  a->Tp = (p->P + (1 << a->kshift) - 1) >> a->kshift;
  a->rows_p = a->nb * a->G;
  a->rows_c = a->G;
  a->rep_p = a->rows_p <= 32 ? 4 : 1;  // (few rows: a copy in each TMEM lane quarter)
  a->rep_c = a->rows_c <= 32 ? 4 : 1;
  // in hundreds of cycles, measured: a tile of few rows takes what its keys take from HBM, one of
  // many rows its exponentials
  const int many = p->Dqk == 64 ? 22 : p->Dqk == 192 ? 29 : 27;
  const int few = p->Dqk == 64 ? 12 : p->Dqk == 192 ? 25 : 24;
  a->wt_p = a->rep_p > 1 ? few : many;
  a->wt_c = a->rep_c > 1 ? few : many;
  a->we = 30;
  const size_t parts_p = p->P ? (static_cast<size_t>(a->HK) * a->Rt + kMaxCtas) * a->rows_p : 0;
  const size_t parts_c = (static_cast<size_t>(p->B) * p->HK + kMaxCtas) * a->rows_c;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* q = ws ? ws + off : nullptr;
    off += round256(bytes);
    return q;
  };
  a->ml_p = reinterpret_cast<float2*>(take(parts_p * sizeof(float2)));
  a->po_p = reinterpret_cast<float*>(take(parts_p * p->Dv * sizeof(float)));
  a->ml_c = reinterpret_cast<float2*>(take(parts_c * sizeof(float2)));
  a->po_c = reinterpret_cast<float*>(take(parts_c * p->Dv * sizeof(float)));
  a->line = nullptr;
  if (p->B >= kLineSeqs && static_cast<int64_t>(p->B) * p->HQ >= kJoinRows)
    a->line = reinterpret_cast<int64_t*>(take((static_cast<size_t>(p->B) + 1) * sizeof(int64_t)));
  a->scores = nullptr;
  if (p->weights_out)
    a->scores = reinterpret_cast<float*>(
        take(static_cast<size_t>(p->B) * p->HQ * static_cast<size_t>(a->Sp) * sizeof(float)));
  return off + 16;
}

static int check(const cache_attn_params* p) {
  if (!p) return SA_ERR_INVALID;
  if (p->B <= 0 || p->HQ <= 0 || p->HK <= 0 || p->S <= 0 || p->P < 0) return SA_ERR_INVALID;
  if (p->HQ % p->HK != 0) return SA_ERR_INVALID;
  const bool dims = (p->Dqk == 64 && p->Dv == 64) || (p->Dqk == 128 && p->Dv == 128) ||
                    (p->Dqk == 192 && p->Dv == 128) || (p->Dqk == 256 && p->Dv == 256);
  if (!dims || p->HQ / p->HK > 128) return SA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->B) * p->HQ > 0x7FFFFFFF) return SA_ERR_UNSUPPORTED;
  if (p->B > 65535 || p->HQ > 65535 || p->S > 0x7FFFFF00 || p->P > 0x7FFFFF00)
    return SA_ERR_UNSUPPORTED;
  // (beyond any memory; keeps the workspace's size in range)
  if (p->S > (int64_t(1) << 40) / (static_cast<int64_t>(p->B) * p->HQ)) return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

}  // namespace cache
}  // namespace sa

using namespace sa;

extern "C" size_t cache_attn_workspace_size(const cache_attn_params* p) {
  if (cache::check(p) != SA_OK) return 0;
  cache::Args a{};
  return cache::lay_out(p, &a, nullptr);
}

extern "C" int cache_attn_fwd(const cache_attn_params* p, void* workspace, size_t workspace_bytes,
                              sa_stream_t stream) {
  int rc = cache::check(p);
  if (rc) return rc;
  if (!p->q || !p->k_cache || !p->v_cache || !p->lens || !p->o || !p->lse) return SA_ERR_INVALID;
  if ((p->P > 0) != (p->k_prefix != nullptr) || (p->P > 0) != (p->v_prefix != nullptr))
    return SA_ERR_INVALID;
  if (p->weights && !p->weights_out) return SA_ERR_INVALID;
  if (partly_overlap(p->weights, static_cast<const float*>(p->weights_out),
                     static_cast<int64_t>(p->B) * p->HK * p->S))
    return SA_ERR_INVALID;
  if (!(p->softmax_scale > 0.f)) return SA_ERR_INVALID;
  const void* ptrs[] = {p->q, p->k_cache, p->v_cache, p->k_prefix, p->v_prefix, p->o};
  for (const void* x : ptrs)
    if ((reinterpret_cast<uintptr_t>(x) & 15u) != 0) return SA_ERR_ALIGN;
  const void* words[] = {p->lens, p->lse, p->weights, p->weights_out, p->dev_status};
  for (const void* x : words)
    if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0) return SA_ERR_ALIGN;
  cache::Args a{};
  const size_t need = cache::lay_out(p, &a, static_cast<char*>(workspace));
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
    return SA_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = check_stream_device(st);
  if (rc) return rc;
  a.q = static_cast<const __nv_bfloat16*>(p->q);
  a.k = static_cast<const __nv_bfloat16*>(p->k_cache);
  a.v = static_cast<const __nv_bfloat16*>(p->v_cache);
  a.kp = static_cast<const __nv_bfloat16*>(p->k_prefix);
  a.vp = static_cast<const __nv_bfloat16*>(p->v_prefix);
  a.lens = p->lens;
  a.o = static_cast<__nv_bfloat16*>(p->o);
  a.lse = p->lse;
  a.w_in = p->weights;
  a.w_out = p->weights_out;
  a.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  a.status = p->dev_status;
  const uint64_t lim = g_wait_limit_ns.load(std::memory_order_relaxed);
  a.wait_limit_ns = lim ? lim : kWaitLimitNs;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SA_ERR_CUDA;
  a.C = sms < cache::kMaxCtas ? sms : cache::kMaxCtas;
  if (p->Dqk == 64) return cache::launch<64, 64>(a, st);
  if (p->Dqk == 128) return cache::launch<128, 128>(a, st);
  if (p->Dqk == 192) return cache::launch<192, 128>(a, st);
  return cache::launch<256, 256>(a, st);
}
