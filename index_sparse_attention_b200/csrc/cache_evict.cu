// cache_evict.cu -- eviction from a cache by accumulated attention weight (cache_evict).
//
// Per (sequence, KV head) of n > budget keys: the first `sinks`, the last `recent` and the
// budget - sinks - recent heaviest keys between them stay, in their order.  First the selection
// (which positions stay), then the copy of the kept rows.
//   selection  a cluster of 1 to 8 CTAs per (sequence, KV head), a slice of the row each, held
//              in registers as order-preserving keys (4, 8 or 16 per thread; longer slices are
//              read again in every sweep).  Radix select of the smallest kept weight in up to
//              three digit passes (12, 12, 8 bits): each CTA counts its keys in shared memory
//              and adds up a share of the bins over the cluster (distributed shared memory) for
//              all.  Where all keys of the digit found are needed, as mostly after 24 bits, no
//              further pass follows (11, 11 and 10 bits without that end: one cache of 4096 keys
//              11.1 us in all against 9.9, 16 of 8191 55.8 against 55.3, 8 of 65536 83 against
//              84).
//              Then every warp counts its stretch of the row, one scan over the warps and CTAs
//              gives each its place, and a last sweep writes the positions in order: keys above
//              the threshold, and of those equal to it the first ones that are still needed.
//              Bound by the sweeps' instructions and the cluster's meetings, not by bytes: 25 us
//              for 32 rows of 65536 (with the slice in shared memory and 64-bit positions 39).
//   copy       16-byte pieces, four rows per thread in flight; by the selection's own CTAs where
//              they fill the SMs, else by a kernel of its own (writes contiguous over all heads
//              of a row).  Bound by HBM (each kept row is read and written once): 16 sequences of
//              8 heads of 4352 to 8191 keys, one of 511, cut to 2048, D=128, 52 us in all, 5.1 TB/s
//              of its bytes.
//              (Asking L2 for the rows that are sure to stay while the selection still runs made
//              it slower: its warps have no time for that.)
#include "sa_device.cuh"
#include "sa_kernels.h"

namespace sa {
namespace evict {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBits = 12;  // of the first two digits
constexpr int kBins = 1 << kBits;
constexpr int kPerThread = kBins / kThreads;
constexpr int kSlice = 8192;        // keys a CTA takes before the row is spread over more of them
constexpr int kMaxCluster = 8;
constexpr int kMaxCtas = 128;       // CTAs that run at once (clusters do not fill every SM)

struct Args {
  const uint4 *k, *v;
  uint4 *ko, *vo;
  const float* w;
  float* wo;
  const int32_t* lens;
  int32_t *lens_o, *keep;
  int B, HK, kp, vp;  // kp, vp: 16-byte pieces of a K / V row of one head
  int64_t S, So;
  int budget, sinks, recent;
  int cluster;
  int rows;  // of a CTA of the copy
  bool fused;  // the selection's CTAs copy the rows themselves
  int32_t* status;
};

// Order-preserving key of a weight: larger weight, larger key; -0 as +0, every NaN on top.
__device__ __forceinline__ uint32_t weight_key(float v) {
  uint32_t u = __float_as_uint(v);
  if (u == 0x80000000u) u = 0u;
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int cluster_load(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Inclusive sum over the lanes of a warp.
__device__ __forceinline__ int warp_scan(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += t;
  }
  return x;
}

// The weights, and the rows copied, may come from a kernel that let this one start before it had
// written them (the key weights' join, a decoding step's weights, an eviction's copy): they are
// read by coherent loads, behind wait_previous_kernel().  The read-only path (__ldg) is for data
// that nothing writes while a kernel runs, from its start on.  From L2, since the copies read a
// row once.

// The kept rows of one (sequence, KV head), this CTA's share of them: 16-byte pieces, four rows
// per thread in flight.  keep null: row i is row i.
template <int kN>
__device__ __forceinline__ void copy_head(const uint4* src, uint4* dst,
                                          const int32_t* keep, int64_t pitch, int per_head, int n,
                                          int rank, int cl) {
  const int at_once = kThreads / per_head, r = threadIdx.x / per_head,
            p = threadIdx.x - r * per_head;
  if (r >= at_once) return;
  const int step = at_once * cl;
  for (int i0 = rank * at_once + r; i0 < n; i0 += kN * step) {
    int64_t from[kN];
    uint4 x[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int i = i0 + e * step;
      from[e] = i;
      if (i < n && keep) from[e] = keep[i];
    }
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (i0 + e * step < n) x[e] = __ldcg(src + from[e] * pitch + p);
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (i0 + e * step < n) dst[(i0 + e * step) * pitch + p] = x[e];
  }
}

// KPT: keys per thread held in registers; 0: read from memory in every sweep.
template <int KPT>
__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const Args a) {
  __shared__ __align__(16) int own[kBins], all[kBins];  // own counts of a digit, the cluster's
  __shared__ int warp_sum[kWarps], warp_eq[kWarps];
  __shared__ int pick[3];    // digit, keys above it, keys of it
  __shared__ int counts[2];  // this CTA's keys above the threshold and equal to it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), cl = a.cluster;
  const int64_t row = blockIdx.x / cl;
  const int b = static_cast<int>(row / a.HK), hk = static_cast<int>(row - static_cast<int64_t>(b) * a.HK);
  wait_previous_kernel();
  const int raw = ld_behind(a.lens + b);  // (every other load depends on it)
  const int n = static_cast<int>(min64(max64(static_cast<int64_t>(raw), 0), a.S));
  if (tid == 0 && hk == 0 && rank == 0) {
    if (raw != n) report_status(a.status, kStatusIndex);
    a.lens_o[b] = min(n, a.budget);
  }
  const float* w = a.w + row * a.S;
  float* wo = a.wo + row * a.So;
  int32_t* keep = a.keep + row * a.budget;
  const int n_out = min(n, a.budget);
  const int step = cl * kThreads, first = rank * kThreads + tid;
  auto fill_tails = [&] {
    for (int64_t i = n_out + first; i < a.So; i += step) wo[i] = 0.f;
    for (int i = n_out + first; i < a.budget; i += step) keep[i] = -1;
  };
  auto copy_all = [&](const int32_t* from) {
    const int64_t pk = static_cast<int64_t>(a.HK) * a.kp, pv = static_cast<int64_t>(a.HK) * a.vp;
    copy_head<4>(a.k + b * a.S * pk + hk * a.kp, a.ko + b * a.So * pk + hk * a.kp, from, pk, a.kp,
                 n_out, rank, cl);
    copy_head<4>(a.v + b * a.S * pv + hk * a.vp, a.vo + b * a.So * pv + hk * a.vp, from, pv, a.vp,
                 n_out, rank, cl);
  };
  if (n <= a.budget) {  // (the same on every CTA of the cluster)
    for (int i0 = first; i0 < n_out; i0 += 4 * step) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e * step < n_out) x[e] = __ldcg(w + i0 + e * step);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e * step < n_out) {
          keep[i0 + e * step] = i0 + e * step;
          wo[i0 + e * step] = x[e];
        }
    }
    fill_tails();
    if (a.fused) copy_all(nullptr);
    return;
  }
  const int lo = a.sinks, hi = n - a.recent;         // the candidates
  const int chosen = a.budget - a.sinks - a.recent;  // of which so many stay (fewer than hi - lo)
  // this warp's stretch [w0, w1) of this CTA's slice of the row, both in whole 32s
  const int per_cta = ((n + cl - 1) / cl + 31) / 32 * 32;
  const int s0 = min(n, rank * per_cta), s1 = min(n, s0 + per_cta);
  const int per_warp = ((s1 - s0 + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int w0 = min(s1, s0 + warp * per_warp), w1 = min(s1, w0 + per_warp);
  const int sweeps = KPT > 0 ? KPT : (w1 - w0 + 31) / 32;
  constexpr int kUnroll = KPT > 0 ? KPT : 1;
  constexpr int kHeld = KPT > 0 ? KPT : 1;
  static_assert(KPT <= 32, "a bit per key");
  uint32_t held[kHeld];
  uint32_t cand = 0;  // bit j: this lane's key of sweep j is a candidate
  if constexpr (KPT > 0) {
    float x[kHeld];
#pragma unroll
    for (int j = 0; j < KPT; ++j)
      x[j] = w0 + 32 * j + lane < w1 ? __ldcg(w + w0 + 32 * j + lane) : 0.f;
    fill_tails();  // (while the loads are on their way)
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int i = w0 + 32 * j + lane;
      held[j] = weight_key(x[j]);
      cand |= static_cast<uint32_t>(i < w1 && i >= lo && i < hi) << j;
    }
  } else {
    fill_tails();
  }
  // the key of this lane in sweep j (position w0 + 32 j + lane, below w1)
  auto key_of = [&](int j) -> uint32_t {
    if constexpr (KPT > 0) return held[j];
    else return weight_key(w[w0 + 32 * j + lane]);
  };
  auto meet = [&] {
    if (cl > 1) cluster_meet();
    else __syncthreads();
  };
  uint32_t prefix = 0;
  int need = chosen;
  bool whole = false;  // every key that begins with the digits found stays
  if (chosen > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3 && !whole; ++pass) {
      const int shift = pass == 0 ? 32 - kBits : pass == 1 ? 32 - 2 * kBits : 0;
      const uint32_t digit = pass == 2 ? (1u << (32 - 2 * kBits)) - 1u : kBins - 1;
      const uint32_t fixed = pass == 0 ? 0u : 0xFFFFFFFFu << (pass == 1 ? 32 - kBits : 32 - 2 * kBits);
      // (every CTA has read the last pass's counts: they met behind that)
      for (int e = tid; e < kBins / 4; e += kThreads)
        reinterpret_cast<int4*>(own)[e] = make_int4(0, 0, 0, 0);
      __syncthreads();
#pragma unroll(kUnroll)
      for (int j = 0; j < sweeps; ++j) {
        bool count;
        uint32_t key;
        if constexpr (KPT > 0) {
          key = held[j];
          count = ((cand >> j) & 1u) && (key & fixed) == prefix;
        } else {
          const int i = w0 + 32 * j + lane;
          count = i < w1 && i >= lo && i < hi;
          key = count ? key_of(j) : 0u;
          count = count && (key & fixed) == prefix;
        }
        const uint32_t bin = (key >> shift) & digit;
        // (a warp whose keys all fall into one bin adds once: 32 adds to one address are taken
        // one after another)
        const uint32_t bin0 = __shfl_sync(0xFFFFFFFFu, bin, 0);
        if (__all_sync(0xFFFFFFFFu, count && bin == bin0)) {
          if (lane == 0) atomicAdd(&own[bin], 32);
        } else if (count) {
          atomicAdd(&own[bin], 1);
        }
      }
      meet();
      if (cl > 1) {
        // every CTA adds up its share of the bins and hands the sums to all
        const int share = kBins / cl;
#pragma unroll 1
        for (int e = rank * share + tid; e < (rank + 1) * share; e += kThreads) {
          int sum = 0;
#pragma unroll 1
          for (int r0 = 0; r0 < cl; r0 += 4) {
            int part[4];  // (loads in flight)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              part[r] = r0 + r < cl ? cluster_load(mapa_shared(smem_u32(&own[e]), r0 + r)) : 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) sum += part[r];
          }
#pragma unroll 1
          for (int r = 0; r < cl; ++r)
            st_shared_cluster_u32(mapa_shared(smem_u32(&all[e]), r), static_cast<uint32_t>(sum));
        }
        cluster_meet();
      }
      // digits from the top: the one in which the need-th key lies (a stretch of bins per thread)
      const int top = kBins - kPerThread * (tid + 1);
      const int* counted = (cl > 1 ? all : own) + top;
      int mine = 0;
#pragma unroll
      for (int e = 0; e < kPerThread; e += 4) {
        const int4 v = *reinterpret_cast<const int4*>(counted + e);
        mine += v.x + v.y + v.z + v.w;
      }
      const int incl = warp_scan(mine);
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      const int sums = warp_scan(warp_sum[lane]);
      const int before = __shfl_sync(0xFFFFFFFFu, sums, (warp + 31) & 31);
      int above = incl - mine + (warp > 0 ? before : 0);
      if (above < need && above + mine >= need) {
#pragma unroll 1
        for (int e = kPerThread - 1; e >= 0; --e) {
          const int n = counted[e];
          if (above < need && above + n >= need) {
            pick[0] = top + e;
            pick[1] = above;
            pick[2] = n;
          }
          above += n;
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      need -= pick[1];
      whole = need == pick[2];
    }
  }
  // All keys from `prefix` on stay where it stands for a whole digit; else those above it and
  // `need` of the keys equal to it, the first ones.  Which of this lane's keys are kept for sure,
  // and which are equal:
  auto sure_at = [&](int j, bool& equal) {
    const int i = w0 + 32 * j + lane;
    equal = false;
    if (i >= w1) return false;
    if (i < lo || i >= hi) return true;
    if (chosen == 0) return false;
    const uint32_t key = key_of(j);
    equal = !whole && key == prefix;
    return key > prefix || (whole && key == prefix);
  };
  uint32_t sure = 0, equal = 0;  // as bits (registers)
  int n_in = 0, n_eq = 0;
  if constexpr (KPT > 0) {
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const bool in = (cand >> j) & 1u;
      const bool at = held[j] == prefix;
      sure |= static_cast<uint32_t>(in ? chosen > 0 && (held[j] > prefix || (whole && at))
                                       : w0 + 32 * j + lane < w1)
              << j;
      equal |= static_cast<uint32_t>(in && chosen > 0 && !whole && at) << j;
    }
    n_in = __reduce_add_sync(0xFFFFFFFFu, __popc(sure));
    n_eq = __reduce_add_sync(0xFFFFFFFFu, __popc(equal));
  } else {
    for (int j = 0; j < sweeps; ++j) {
      bool e;
      const bool in = sure_at(j, e);
      n_in += __popc(__ballot_sync(0xFFFFFFFFu, in));
      n_eq += __popc(__ballot_sync(0xFFFFFFFFu, e));
    }
  }
  if (lane == 0) {
    warp_sum[warp] = n_in;
    warp_eq[warp] = n_eq;
  }
  __syncthreads();
  const int in_scan = warp_scan(warp_sum[lane]), eq_scan = warp_scan(warp_eq[lane]);
  int in_before = __shfl_sync(0xFFFFFFFFu, in_scan, (warp + 31) & 31);
  int eq_before = __shfl_sync(0xFFFFFFFFu, eq_scan, (warp + 31) & 31);
  if (warp == 0) in_before = eq_before = 0;
  if (tid == 31) {
    counts[0] = in_scan;
    counts[1] = eq_scan;
  }
  meet();
  if (rank > 0) {  // lane r asks CTA r, all in flight
    const int c = lane < rank ? cluster_load(mapa_shared(smem_u32(&counts[0]), lane)) : 0;
    const int e = lane < rank ? cluster_load(mapa_shared(smem_u32(&counts[1]), lane)) : 0;
    in_before += __reduce_add_sync(0xFFFFFFFFu, c);
    eq_before += __reduce_add_sync(0xFFFFFFFFu, e);
  }
  const uint32_t below = (1u << lane) - 1u;
  // the weights themselves (their own bits: -0 and every NaN share a key), all loads in flight
  // before the first store
  float value[kHeld];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int j = 0; j < KPT; ++j)
      if (((sure | equal) >> j) & 1u) value[j] = __ldcg(w + w0 + 32 * j + lane);
  }
#pragma unroll(kUnroll)
  for (int j = 0; j < sweeps; ++j) {
    const int i = w0 + 32 * j + lane;
    bool in, eq;
    if constexpr (KPT > 0) {
      in = (sure >> j) & 1u;
      eq = (equal >> j) & 1u;
    } else {
      in = sure_at(j, eq);
    }
    const uint32_t ins = __ballot_sync(0xFFFFFFFFu, in);
    const uint32_t eqs = n_eq > 0 ? __ballot_sync(0xFFFFFFFFu, eq) : 0u;
    // place among the kept: all sure ones and the needed equal ones before it
    const int eq_at = eq_before + __popc(eqs & below);
    if (in || (eq && eq_at < need)) {
      const int at = in_before + __popc(ins & below) + min(eq_at, need);
      keep[at] = i;
      if constexpr (KPT > 0) wo[at] = value[j];
      else wo[at] = w[i];
    }
    in_before += __popc(ins);
    eq_before += __popc(eqs);
  }
  if (!a.fused) allow_next_kernel();
  meet();  // (no CTA leaves while another may read its counts; keep is written)
  if (a.fused) copy_all(keep);
}

// One CTA per a.rows output rows of a sequence; a thread keeps its 16-byte column of a row and
// takes every 256-th, four rows at once (with eight pieces of K and V mixed per thread, and a
// quotient for each, the large copies took half as long again).
template <int kN>
__device__ __forceinline__ void copy_rows(const uint4* src, uint4* dst, const int32_t* keep,
                                          int budget, int HK, int per_head, int i0, int rows) {
  const int per_row = HK * per_head;
  for (int p = threadIdx.x; p < per_row; p += 256) {
    const int32_t* kp = keep + static_cast<int64_t>(p / per_head) * budget + i0;
    for (int r = 0; r < rows; r += kN) {
      int64_t from[kN];
      uint4 x[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (r + e < rows) from[e] = kp[r + e];
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (r + e < rows) x[e] = __ldcg(src + from[e] * per_row + p);
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (r + e < rows) dst[static_cast<int64_t>(i0 + r + e) * per_row + p] = x[e];
    }
  }
}
__global__ void __launch_bounds__(256) evict_copy_kernel(const Args a) {
  const int b = blockIdx.y;
  allow_next_kernel();
  wait_previous_kernel();
  const int n_out = static_cast<int>(min64(max64(static_cast<int64_t>(ld_behind(a.lens + b)), 0),
                                           min64(a.S, a.budget)));
  const int i0 = blockIdx.x * a.rows, rows = min(a.rows, n_out - i0);
  if (rows <= 0) return;
  const int32_t* keep = a.keep + static_cast<int64_t>(b) * a.HK * a.budget;
  const int64_t pk = static_cast<int64_t>(a.HK) * a.kp, pv = static_cast<int64_t>(a.HK) * a.vp;
  copy_rows<4>(a.k + b * a.S * pk, a.ko + b * a.So * pk, keep, a.budget, a.HK, a.kp, i0, rows);
  copy_rows<4>(a.v + b * a.S * pv, a.vo + b * a.So * pv, keep, a.budget, a.HK, a.vp, i0, rows);
}

}  // namespace evict
}  // namespace sa

using namespace sa;

extern "C" int cache_evict(const cache_evict_params* p, sa_stream_t stream) {
  if (!p) return SA_ERR_INVALID;
  if (!p->k_cache || !p->v_cache || !p->weights || !p->lens || !p->k_out || !p->v_out ||
      !p->weights_out || !p->lens_out || !p->keep)
    return SA_ERR_INVALID;
  if (p->B <= 0 || p->HK <= 0 || p->S <= 0 || p->budget <= 0 || p->sinks < 0 || p->recent < 0)
    return SA_ERR_INVALID;
  if (static_cast<int64_t>(p->sinks) + p->recent > p->budget || p->budget > p->S_out)
    return SA_ERR_INVALID;
  const bool dims = (p->Dqk == 64 && p->Dv == 64) || (p->Dqk == 128 && p->Dv == 128) ||
                    (p->Dqk == 192 && p->Dv == 128) || (p->Dqk == 256 && p->Dv == 256);
  if (!dims) return SA_ERR_UNSUPPORTED;
  if (p->B > 65535 || p->S > 0x7FFFFF00 || p->S_out > 0x7FFFFF00 || p->HK > 65535 ||
      static_cast<int64_t>(p->B) * p->HK > 0x7FFFFFFF)
    return SA_ERR_UNSUPPORTED;
  // no output may share memory with an input or another output
  const int64_t BH = static_cast<int64_t>(p->B) * p->HK;
  if (p->S > (int64_t(1) << 40) / BH || p->S_out > (int64_t(1) << 40) / BH)
    return SA_ERR_UNSUPPORTED;  // (beyond any memory; keeps the products below in range)
  struct Span {
    const void* at;
    int64_t bytes;
  } const spans[] = {{p->k_cache, BH * p->S * p->Dqk * 2}, {p->v_cache, BH * p->S * p->Dv * 2},
                     {p->weights, BH * p->S * 4},          {p->lens, p->B * 4ll},
                     {p->k_out, BH * p->S_out * p->Dqk * 2}, {p->v_out, BH * p->S_out * p->Dv * 2},
                     {p->weights_out, BH * p->S_out * 4},  {p->lens_out, p->B * 4ll},
                     {p->keep, BH * p->budget * 4}};
  for (int i = 4; i < 9; ++i)
    for (int j = 0; j < i; ++j) {
      const char *x = static_cast<const char*>(spans[i].at), *y = static_cast<const char*>(spans[j].at);
      if (x < y + spans[j].bytes && y < x + spans[i].bytes) return SA_ERR_INVALID;
    }
  const void* ptrs[] = {p->k_cache, p->v_cache, p->k_out, p->v_out};
  for (const void* x : ptrs)
    if ((reinterpret_cast<uintptr_t>(x) & 15u) != 0) return SA_ERR_ALIGN;
  const void* words[] = {p->weights, p->lens, p->weights_out, p->lens_out, p->keep, p->dev_status};
  for (const void* x : words)
    if ((reinterpret_cast<uintptr_t>(x) & 3u) != 0) return SA_ERR_ALIGN;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int rc = check_stream_device(st);
  if (rc) return rc;
  evict::Args a{};
  a.k = static_cast<const uint4*>(p->k_cache);
  a.v = static_cast<const uint4*>(p->v_cache);
  a.ko = static_cast<uint4*>(p->k_out);
  a.vo = static_cast<uint4*>(p->v_out);
  a.w = p->weights;
  a.wo = p->weights_out;
  a.lens = p->lens;
  a.lens_o = p->lens_out;
  a.keep = p->keep;
  a.B = p->B;
  a.HK = p->HK;
  a.kp = p->Dqk / 8;
  a.vp = p->Dv / 8;
  a.S = p->S;
  a.So = p->S_out;
  a.budget = p->budget;
  a.sinks = p->sinks;
  a.recent = p->recent;
  a.status = p->dev_status;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SA_ERR_CUDA;
  // rows of a copy CTA: 16, or 4 (one round of loads) where that leaves SMs without work
  const int64_t most = min64(p->budget, p->S);
  a.rows = (most + 15) / 16 * p->B >= 4 * sms ? 16 : 4;
  // A row is spread over more CTAs while its slices are long, as long as all clusters run at
  // once (32 rows of 65536 in all: 115 us over 256 CTAs, 80 over 128), or until a slice fits in
  // registers.
  a.cluster = 1;
  while (a.cluster < evict::kMaxCluster &&
         (static_cast<int64_t>(a.cluster) * 2 * evict::kSlice < p->S ||
          (static_cast<int64_t>(a.cluster) * evict::kSlice < p->S &&
           BH * a.cluster * 2 <= evict::kMaxCtas)))
    a.cluster *= 2;
  // Selection CTAs that fill the SMs copy their own rows (no second launch, and rows that are
  // selected early are copied while others are not): 64 full sequences of 8 heads, 8191 to 2048
  // keys, D=128, 193 us against 209, 16 of them 56 against 61.  Few CTAs, or a last wave of them
  // that leaves SMs idle, would copy with part of the GPU: 20 of 8191 (160 CTAs) 89 us against 76;
  // 2 sequences of 131072 (128 CTAs) take 108 either way.  The rule knows the shapes only: one
  // long sequence among short ones is copied by its own heads' CTAs.
  const int64_t ctas = BH * a.cluster, waves = (ctas + sms - 1) / sms;
  a.fused = ctas * 5 >= waves * sms * 4;
  if (BH * a.cluster > 0x7FFFFFFF) return SA_ERR_UNSUPPORTED;
  // keys per thread: a warp's stretch of the longest slice, in whole 32s
  const int64_t slice = ((p->S + a.cluster - 1) / a.cluster + 31) / 32 * 32;
  const int64_t stretch = ((slice + evict::kWarps - 1) / evict::kWarps + 31) / 32;
  auto select = stretch <= 4    ? evict::evict_select_kernel<4>
                : stretch <= 8  ? evict::evict_select_kernel<8>
                : stretch <= 16 ? evict::evict_select_kernel<16>
                                : evict::evict_select_kernel<0>;
  rc = launch_early(select, dim3(static_cast<unsigned>(BH * a.cluster)), dim3(evict::kThreads), 0, st,
                    "eviction select kernel launch", a.cluster, a);
  if (rc) return rc;
  if (a.fused) return SA_OK;
  return launch_early(evict::evict_copy_kernel,
                      dim3(static_cast<unsigned>((most + a.rows - 1) / a.rows),
                           static_cast<unsigned>(p->B)),
                      dim3(256), 0, st, "eviction copy kernel launch", 1, a);
}
