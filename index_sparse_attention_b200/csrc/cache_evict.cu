// cache_evict.cu -- eviction from a cache by accumulated attention weight (cache_evict).
//
// Per (sequence, KV head) of n > budget keys: the first `sinks`, the last `recent` and the
// budget - sinks - recent heaviest keys between them stay, in their order.  Two launches:
// selection (which positions stay) and the copy of the kept rows.
//   selection  one CTA per (sequence, KV head): radix select of the smallest kept weight in
//              four digit passes of 8 bits over order-preserving keys (every pass reads the row
//              again, from L2), then one pass in position order that writes the positions whose
//              key is above the threshold, and of those equal to it the first ones that are
//              still needed.
//   copy       one CTA per eight output rows of a sequence: 16-byte pieces, writes contiguous
//              over all heads of a row, reads a contiguous piece per (row, head).
#include "sa_device.cuh"
#include "sa_kernels.h"

namespace sa {
namespace evict {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

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
  int32_t* status;
};

// Order-preserving key of a weight: larger weight, larger key; -0 as +0, every NaN on top.
__device__ __forceinline__ uint32_t weight_key(float v) {
  uint32_t u = __float_as_uint(v);
  if (u == 0x80000000u) u = 0u;
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of `v` over the block in thread order; `sum` gets the total.
__device__ __forceinline__ int block_prefix(int v, int* sh, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += t;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int t = lane < kWarps ? sh[lane] : 0, y = t;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xFFFFFFFFu, y, d);
    if (lane >= d) y += z;
  }
  sum = __shfl_sync(0xFFFFFFFFu, y, 31);
  return x - v + __shfl_sync(0xFFFFFFFFu, y - t, warp);
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const Args a) {
  __shared__ int hist[256];
  __shared__ int sh[kWarps];
  __shared__ int pick[2];  // digit, keys above it
  const int tid = threadIdx.x;
  const int b = blockIdx.x / a.HK, hk = blockIdx.x - b * a.HK;
  const int raw = __ldg(a.lens + b);
  const int64_t n = min64(max64(static_cast<int64_t>(raw), 0), a.S);
  if (tid == 0 && hk == 0) {
    if (raw != n) report_status(a.status, kStatusIndex);
    a.lens_o[b] = static_cast<int32_t>(min64(n, a.budget));
  }
  const int64_t row = static_cast<int64_t>(b) * a.HK + hk;
  const float* w = a.w + row * a.S;
  float* wo = a.wo + row * a.So;
  int32_t* keep = a.keep + row * a.budget;
  const int n_out = static_cast<int>(min64(n, a.budget));
  for (int64_t i = n_out + tid; i < a.So; i += kThreads) wo[i] = 0.f;
  for (int i = n_out + tid; i < a.budget; i += kThreads) keep[i] = -1;
  if (n <= a.budget) {
    for (int i = tid; i < n_out; i += kThreads) {
      keep[i] = i;
      wo[i] = w[i];
    }
    return;
  }
  const int64_t lo = a.sinks, hi = n - a.recent;  // the candidates
  int need = a.budget - a.sinks - a.recent;       // of which so many stay (fewer than hi - lo)
  uint32_t prefix = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int e = tid; e < 256; e += kThreads) hist[e] = 0;
      __syncthreads();
      const uint32_t fixed = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int64_t i = lo + tid; i < hi; i += kThreads) {
        const uint32_t key = weight_key(__ldg(w + i));
        if ((key & fixed) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      // digits from the top: the one in which the need-th key lies
      const int mine = tid < 256 ? hist[255 - tid] : 0;
      int sum;
      const int above = block_prefix(mine, sh, sum);
      if (tid < 256 && above < need && above + mine >= need) {
        pick[0] = 255 - tid;
        pick[1] = above;
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      need -= pick[1];
      __syncthreads();
    }
  }
  // `need` of the keys equal to `prefix` stay, the first ones
  const bool any = a.budget - a.sinks - a.recent > 0;
  int out = 0, equal = 0;
  for (int64_t i0 = 0; i0 < n; i0 += kThreads) {
    const int64_t i = i0 + tid;
    float x = 0.f;
    bool in = false, eq = false;
    if (i < n) {
      x = __ldg(w + i);
      if (i < lo || i >= hi) {
        in = true;
      } else if (any) {
        const uint32_t key = weight_key(x);
        in = key > prefix;
        eq = key == prefix;
      }
    }
    int sum;
    const int e = block_prefix(eq, sh, sum);
    if (eq && equal + e < need) in = true;
    equal += sum;
    const int at = block_prefix(in, sh, sum);
    if (in) {
      keep[out + at] = static_cast<int32_t>(i);
      wo[out + at] = x;
    }
    out += sum;
  }
}

constexpr int kRows = 8;
__global__ void __launch_bounds__(256) evict_copy_kernel(const Args a) {
  const int b = blockIdx.y;
  const int n_out = static_cast<int>(min64(max64(static_cast<int64_t>(__ldg(a.lens + b)), 0),
                                           min64(a.S, a.budget)));
  const int i0 = blockIdx.x * kRows, rows = min(kRows, n_out - i0);
  if (rows <= 0) return;
  const int pk = a.HK * a.kp, pv = a.HK * a.vp;
  auto copy = [&](const uint4* src, uint4* dst, int per_head, int per_row) {
    for (int e = threadIdx.x; e < rows * per_row; e += 256) {
      const int i = i0 + e / per_row, p = e % per_row, hk = p / per_head;
      const int64_t from = __ldg(a.keep + (static_cast<int64_t>(b) * a.HK + hk) * a.budget + i);
      dst[(static_cast<int64_t>(b) * a.So + i) * per_row + p] =
          __ldg(src + (static_cast<int64_t>(b) * a.S + from) * per_row + p);
    }
  };
  copy(a.k, a.ko, a.kp, pk);
  copy(a.v, a.vo, a.vp, pv);
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
  evict::evict_select_kernel<<<static_cast<unsigned>(p->B * p->HK), evict::kThreads, 0, st>>>(a);
  rc = check_launch("eviction select kernel launch");
  if (rc) return rc;
  const int64_t most = min64(p->budget, p->S);
  evict::evict_copy_kernel<<<dim3(static_cast<unsigned>((most + evict::kRows - 1) / evict::kRows),
                                  static_cast<unsigned>(p->B)),
                             256, 0, st>>>(a);
  return check_launch("eviction copy kernel launch");
}
