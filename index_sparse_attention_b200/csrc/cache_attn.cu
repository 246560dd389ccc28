// cache_attn.cu -- attention of one new token per sequence over a prefix that the batch
// shares and each sequence's own cache (cache_attn_fwd).
//
// Mathematics: softmax attention of a row over the union of two key sets, from parts.  A part
// over a run of keys holds m = max s_j, l = sum exp(s_j - m), o = sum exp(s_j - m) v_j; parts
// join as m' = max m, l' = sum l exp(m - m'), o' = sum o exp(m - m') (fp32 throughout), and
// lse = m' + ln l', o = o' / l'.
// Three launches: the parts (this file's main kernel, work split as in cache_plan.cuh), their
// join, and, when asked for, the keys' weights from the stored scores.
#include "cache_plan.cuh"
#include "sa_kernels.h"

namespace sa {
namespace cache {

constexpr int kSimple = 256;  // threads of the main kernel
constexpr int kRowBlk = 8;

template <int DQK, int DV>
__global__ void __launch_bounds__(kSimple) cache_part_kernel(const Args a) {
  __shared__ int64_t sh[66];
  __shared__ float qs[kRowBlk][DQK];
  __shared__ float ss[kRowBlk][128];
  __shared__ float mrow[kRowBlk], lrow[kRowBlk], arow[kRowBlk];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  const Found f = find_range<kSimple>(a, c, sh);
  if (c == 0)
    for (int b = tid; b < a.B; b += kSimple) {
      const int n = __ldg(a.lens + b);
      if (n < 0 || n > a.S) report_status(a.status, kStatusIndex);
    }
  Walk w;
  if (f.u0 < f.u1) w.init(a, f.u0, f.b, f.off);
  int64_t u = f.u0;
  while (u < f.u1) {
    const int64_t n_tiles = min64(w.tiles - w.tile, f.u1 - u);
    const int rows = w.prefix ? a.nb * a.G : a.G;
    const int64_t slot = w.seg + c;
    for (int r0 = 0; r0 < rows; r0 += kRowBlk) {
      __syncthreads();
      for (int e = tid; e < kRowBlk * DQK; e += kSimple) {
        const int r = r0 + e / DQK, d = e % DQK;
        float x = 0.f;
        if (r < rows) {
          const int g = w.prefix ? r / a.nb : r;
          const int b = w.prefix ? w.rt * a.nb + r % a.nb : w.b;
          if (b < a.B)
            x = __bfloat162float(a.q[(static_cast<int64_t>(b) * a.HQ + w.hk * a.G + g) * DQK + d]);
        }
        qs[e / DQK][d] = x;
      }
      if (tid < kRowBlk) {
        mrow[tid] = -INFINITY;
        lrow[tid] = 0.f;
      }
      float acc[kRowBlk];
      for (int r = 0; r < kRowBlk; ++r) acc[r] = 0.f;
      for (int64_t t = w.tile; t < w.tile + n_tiles; ++t) {
        const int64_t k0 = t * a.kn;
        const int nk = static_cast<int>(min64(a.kn, w.keys - k0));
        const int64_t row0 = w.prefix ? k0 : static_cast<int64_t>(w.b) * a.S + k0;
        const __nv_bfloat16* kb = (w.prefix ? a.kp : a.k) + (row0 * a.HK + w.hk) * DQK;
        const __nv_bfloat16* vb = (w.prefix ? a.vp : a.v) + (row0 * a.HK + w.hk) * DV;
        __syncthreads();
        for (int e = tid; e < kRowBlk * 128; e += kSimple) {
          const int r = e / 128, j = e % 128;
          float x = -INFINITY;
          if (j < nk) {
            x = 0.f;
            const __nv_bfloat16* kr = kb + static_cast<int64_t>(j) * a.HK * DQK;
            for (int d = 0; d < DQK; ++d) x = fmaf(qs[r][d], __bfloat162float(kr[d]), x);
            x *= a.scale_log2;
            if (!w.prefix && a.scores && r0 + r < a.G)
              a.scores[(static_cast<int64_t>(w.b) * a.HQ + w.hk * a.G + r0 + r) * a.Sp + k0 + j] = x;
          }
          ss[r][j] = x;
        }
        __syncthreads();
        {  // warp r: the row's max and sum
          const int r = warp;
          float mx = mrow[r];
          for (int j = lane; j < 128; j += 32) mx = fmaxf(mx, ss[r][j]);
          for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
          const float me = mx == -INFINITY ? 0.f : mx;
          float sum = 0.f;
          for (int j = lane; j < 128; j += 32) {
            const float p = ex2(ss[r][j] - me);
            ss[r][j] = p;
            sum += p;
          }
          for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
          __syncwarp();
          if (lane == 0) {
            const float al = ex2(mrow[r] - me);
            arow[r] = al;
            lrow[r] = lrow[r] * al + sum;
            mrow[r] = mx;
          }
        }
        __syncthreads();
        if (tid < DV) {
          for (int r = 0; r < kRowBlk; ++r) acc[r] *= arow[r];
          for (int j = 0; j < nk; ++j) {
            const float x = __bfloat162float(vb[static_cast<int64_t>(j) * a.HK * DV + tid]);
            for (int r = 0; r < kRowBlk; ++r) acc[r] = fmaf(ss[r][j], x, acc[r]);
          }
        }
      }
      __syncthreads();
      float* po = w.prefix ? a.po_p + slot * a.rows_p * DV : a.po_c + slot * a.rows_c * DV;
      float2* ml = w.prefix ? a.ml_p + slot * a.rows_p : a.ml_c + slot * a.rows_c;
      for (int r = 0; r < kRowBlk && r0 + r < rows; ++r) {
        if (tid < DV) po[static_cast<int64_t>(r0 + r) * DV + tid] = acc[r];
        if (tid == 0) ml[r0 + r] = make_float2(mrow[r], lrow[r]);
      }
    }
    u += n_tiles;
    w.tile += n_tiles - 1;
    if (u < f.u1) w.next(a);
  }
}

// ------------------------------------------------------------------------------------
// join: one block per (sequence, query head)
// ------------------------------------------------------------------------------------
constexpr int kJoin = 128;

template <int DV>
__global__ void __launch_bounds__(kJoin) cache_join_kernel(const Args a) {
  constexpr int kW = kJoin / 32, kD = DV / 32;
  __shared__ int64_t shs[2][kW];
  __shared__ float sh_o[kW][DV], sh_m[kW], sh_l[kW];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / a.HQ, h = blockIdx.x - b * a.HQ;
  const int hk = h / a.G, g = h - hk * a.G;
  // tiles before this sequence and in all
  int64_t before = 0, total = 0;
  for (int x = tid; x < a.B; x += kJoin) {
    const int64_t t = tiles_of(a, clamped_len(a, x));
    total += t;
    if (x < b) before += t;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
    total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
  }
  if (lane == 0) {
    shs[0][warp] = before;
    shs[1][warp] = total;
  }
  __syncthreads();
  before = total = 0;
  for (int x = 0; x < kW; ++x) {
    before += shs[0][x];
    total += shs[1][x];
  }
  const int64_t np = a.Tp * a.Rt * a.HK, U = np + total * a.HK;
  const int C = busy_ctas(a, U);
  const int64_t tb = tiles_of(a, clamped_len(a, b));
  // parts of the prefix (of this row's tile) and of the own cache
  int n_p = 0, n_c = 0;
  int64_t slot_p = 0, slot_c = 0;
  int row_p = 0;
  if (np > 0) {
    const int rt = b / a.nb;
    const int64_t seg = static_cast<int64_t>(hk) * a.Rt + rt;
    const int c0 = cta_of(seg * a.Tp, U, C), c1 = cta_of(seg * a.Tp + a.Tp - 1, U, C);
    n_p = c1 - c0 + 1;
    slot_p = seg + c0;
    row_p = g * a.nb + (b - rt * a.nb);
  }
  if (tb > 0) {
    const int64_t u = np + before * a.HK + hk * tb;
    const int c0 = cta_of(u, U, C), c1 = cta_of(u + tb - 1, U, C);
    n_c = c1 - c0 + 1;
    slot_c = static_cast<int64_t>(b) * a.HK + hk + c0;
  }
  const int nr_p = n_p * a.rep_p, n = nr_p + n_c * a.rep_c;
  float m = -INFINITY, l = 0.f, acc[kD];
#pragma unroll
  for (int e = 0; e < kD; ++e) acc[e] = 0.f;
  for (int i = warp; i < n; i += kW) {
    const float2* ml;
    const float* po;
    if (i < nr_p) {
      const int64_t at = (slot_p * a.rep_p + i) * a.rows_p + row_p;
      ml = a.ml_p + at;
      po = a.po_p + at * DV;
    } else {
      const int64_t at = (slot_c * a.rep_c + (i - nr_p)) * a.rows_c + g;
      ml = a.ml_c + at;
      po = a.po_c + at * DV;
    }
    const float2 v = *ml;
    float x[kD];
#pragma unroll
    for (int e = 0; e < kD; ++e) x[e] = po[e * 32 + lane];
    const float mn = fmaxf(m, v.x);
    if (v.y == 0.f) continue;  // a part without keys
    const float f0 = ex2(m - mn), f1 = ex2(v.x - mn);
    m = mn;
    l = l * f0 + v.y * f1;
#pragma unroll
    for (int e = 0; e < kD; ++e) acc[e] = acc[e] * f0 + x[e] * f1;
  }
#pragma unroll
  for (int e = 0; e < kD; ++e) sh_o[warp][e * 32 + lane] = acc[e];
  if (lane == 0) {
    sh_m[warp] = m;
    sh_l[warp] = l;
  }
  __syncthreads();
  m = -INFINITY;
#pragma unroll
  for (int x = 0; x < kW; ++x) m = fmaxf(m, sh_m[x]);
  const float me = m == -INFINITY ? 0.f : m;
  l = 0.f;
  float f[kW];
#pragma unroll
  for (int x = 0; x < kW; ++x) {
    f[x] = ex2(sh_m[x] - me);
    l += sh_l[x] * f[x];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t row = static_cast<int64_t>(b) * a.HQ + h;
  for (int d = tid; d < DV; d += kJoin) {
    float o = 0.f;
#pragma unroll
    for (int x = 0; x < kW; ++x) o += sh_o[x][d] * f[x];
    a.o[row * DV + d] = __float2bfloat16(o * inv);
  }
  if (tid == 0) a.lse[row] = l == 0.f ? -INFINITY : (me + __log2f(l)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------------------------
// weights: one thread per key of a (sequence, KV head)
// ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) cache_weights_kernel(const Args a) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int hk = blockIdx.y, b = blockIdx.z;
  if (j >= a.S) return;
  const int64_t at = (static_cast<int64_t>(b) * a.HK + hk) * a.S + j;
  const bool live = j < clamped_len(a, b);
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
  cache_part_kernel<DQK, DV><<<a.C, kSimple, 0, st>>>(a);
  int rc = check_launch("cache attention kernel launch");
  if (rc) return rc;
  cache_join_kernel<DV><<<static_cast<unsigned>(a.B * a.HQ), kJoin, 0, st>>>(a);
  rc = check_launch("cache join kernel launch");
  if (rc || !a.w_out) return rc;
  cache_weights_kernel<<<dim3(static_cast<unsigned>((a.S + 255) / 256), a.HK, a.B), 256, 0, st>>>(a);
  return check_launch("cache weights kernel launch");
}

static size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The plan's sizes and the workspace's layout; returns its bytes.
static size_t lay_out(const cache_attn_params* p, Args* a, char* ws) {
  a->B = p->B;
  a->HQ = p->HQ;
  a->HK = p->HK;
  a->G = p->HQ / p->HK;
  a->Dqk = p->Dqk;
  a->Dv = p->Dv;
  a->S = p->S;
  a->P = p->P;
  a->kn = 128;
  a->Sp = (p->S + 127) / 128 * 128;
  a->nb = 128 / a->G;
  if (a->nb > p->B) a->nb = p->B;
  a->Rt = (p->B + a->nb - 1) / a->nb;
  a->Tp = (p->P + a->kn - 1) / a->kn;
  a->rep_p = a->rep_c = 1;
  a->rows_p = a->nb * a->G;
  a->rows_c = a->G;
  const size_t parts_p = p->P ? (static_cast<size_t>(a->HK) * a->Rt + kMaxCtas) * a->rep_p * a->rows_p : 0;
  const size_t parts_c = (static_cast<size_t>(p->B) * p->HK + kMaxCtas) * a->rep_c * a->rows_c;
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
  a->scores = nullptr;
  if (p->weights_out)
    a->scores = reinterpret_cast<float*>(
        take(static_cast<size_t>(p->B) * p->HQ * static_cast<size_t>(a->Sp) * sizeof(float)));
  return off;
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
  if (!(p->softmax_scale > 0.f)) return SA_ERR_INVALID;
  const void* ptrs[] = {p->q, p->k_cache, p->v_cache, p->k_prefix, p->v_prefix, p->o};
  for (const void* x : ptrs)
    if ((reinterpret_cast<uintptr_t>(x) & 15u) != 0) return SA_ERR_ALIGN;
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
