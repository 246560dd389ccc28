// key_weights.cu -- the attention weight every key has received in a forward pass
// (sparse_attn_key_weights): w[b][g][j] = sum over the group's heads h and the queries i that
// see j of P_ij = exp(scale q_i . k_j - lse_i).
//
// Mathematics: with the forward's lse no softmax state is needed; P is recomputed tile by tile
// and summed over its query side.  S^T = K Q^T puts a key on a TMEM lane, so the sum over
// queries is a sum along the columns one thread holds: no exchange between lanes, no atomics,
// one store per key, and a fixed order.
//
// B200 design: a CTA owns 128 keys of one (batch, KV head), its K tile stays in shared memory
// and the query tiles of the key-to-query list stream past it, for every query head of the
// group:
//   warp 0     TMA: K once, then Q tiles of kBN queries, kStages deep;
//   warp 1     tcgen05.mma S^T = K Q^T (128 keys x kBN queries) into one of two TMEM buffers;
//   warps 2-5  thread = key row: exp2(S^T scale log2e - lse log2e) summed over the columns.
//              A step's lse values (one query per thread, fetched a step ahead) pass through
//              shared memory; the presence words of index mode are fetched a step ahead too and
//              transposed across the warp.  Steps are summed on their own before they join the
//              running sum, so that long query ranges do not lose low bits.
// Two CTAs share an SM at head dims up to 192, so that one's prologue and waits overlap the
// other's work.  With fewer key tiles than SMs can hold, the query range is split and the
// parts are added by a second kernel.  Every mbarrier wait is bounded (sa_device.cuh).
#include "sa_device.cuh"
#include "sa_kernels.h"

namespace sa {
namespace kweights {

template <int DQK>
struct Cfg {
  static constexpr int kBN = DQK <= 128 ? 128 : 64;  // queries per step
  static constexpr int kStages = DQK == 64 ? 4 : DQK == 256 ? 4 : 2;
  static constexpr int kCtas = DQK == 256 ? 1 : 2;   // per SM
  static constexpr int kKPanel = 128 * 128;
  static constexpr int kQPanel = kBN * 128;
  static constexpr int kKBytes = 128 * DQK * 2;
  static constexpr int kQBytes = kBN * DQK * 2;
  static constexpr int kQOff = kKBytes;
  static constexpr int kLOff = kQOff + kStages * kQBytes;  // lse of a step, [2][kBN]
  static constexpr int kBarOff = kLOff + 2 * kBN * 4;
  static constexpr int kSmem = kBarOff + 128 + 1024;
  static constexpr uint32_t kTmemCols = 2 * kBN;
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory budget");
};

enum : int { kBK = 0, kBQF = 1, kBQE = 5, kBSF = 9, kBSE = 11, kBDrain = 13, kNumBars = 14 };

struct Args {
  AttnArgs t;
  const float* w_in;
  float* w_out;
  float* part;  // [splits][B * HK][Sk] when splits > 1
  int splits;
};

template <int DQK>
__global__ void __launch_bounds__(192, Cfg<DQK>::kCtas)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k, const Args ka) {
  using C = Cfg<DQK>;
  constexpr int BN = C::kBN;
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
  // the key tiles with the longest lists under causal (the first ones) start first
  const int bgs = a.B * a.HK;
  int lin = static_cast<int>(blockIdx.x);
  const int nt = lin / (bgs * ka.splits);
  lin -= nt * bgs * ka.splits;
  const int sp = lin / bgs, bgi = lin - sp * bgs;
  const int b = bgi / a.HK, g = bgi - b * a.HK;
  const int G = a.HQ / a.HK;
  const int64_t bg = bgi;
  const int64_t trow = bg * a.Tn + nt;
  const int n_full = __ldg(a.tcnt + 2 * trow);
  const int n_mt = n_full + __ldg(a.tcnt + 2 * trow + 1);
  const int32_t* tlist = a.tidx + trow * a.Tm;
  constexpr int kSub = 128 / BN;
  const int64_t n_all = static_cast<int64_t>(G) * n_mt * kSub;  // (head, query tile, part)
  const int64_t it0 = n_all * sp / ka.splits;
  const int n_iter = static_cast<int>(n_all * (sp + 1) / ka.splits - it0);
  int issued = 0;

  if (threadIdx.x == 0) {
    mbar_init(BAR(kBK), 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(BAR(kBQF + s), 1);
      mbar_init(BAR(kBQE + s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(kBSF + s), 1);
      mbar_init(BAR(kBSE + s), 128);
    }
    mbar_init(BAR(kBDrain), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);

  // step -> query head, first query, whether the tile is partial
  auto decode = [&](int it, int& h, int& m0, bool& partial) {
    const int64_t x = it0 + it;
    const int per_head = n_mt * kSub;
    const int hh = static_cast<int>(x / per_head);
    const int rest = static_cast<int>(x - static_cast<int64_t>(hh) * per_head);
    const int k = rest / kSub;
    h = g * G + hh;
    m0 = __ldg(tlist + k) * 128 + (rest % kSub) * BN;
    partial = k >= n_full;
  };

  if (warp == 0) {
    if (n_iter > 0) {
      if (elect_one()) {
        prefetch_tensormap(&tm_q);
        mbar_arrive_expect_tx(BAR(kBK), C::kKBytes);
        for (int c = 0; c < DQK / 64; ++c)
          tma_load_4d(sbase + c * C::kKPanel, &tm_k, BAR(kBK), c * 64, nt * 128, g, b);
      }
      __syncwarp();
      for (int it = 0; it < n_iter; ++it) {
        int h, m0;
        bool partial;
        decode(it, h, m0, partial);
        m0 = __shfl_sync(0xFFFFFFFFu, m0, 0);
        const int st = it % C::kStages, u = it / C::kStages;
        if (!warp_wait(BAR(kBQE + st), (u & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(BAR(kBQF + st), C::kQBytes);
          for (int c = 0; c < DQK / 64; ++c)
            tma_load_4d(sbase + C::kQOff + st * C::kQBytes + c * C::kQPanel, &tm_q, BAR(kBQF + st),
                        c * 64, m0, h, b);
        }
        __syncwarp();
        issued = it + 1;
      }
      // the last arrivals on the stages' barriers have landed before the CTA may leave
      if (issued == n_iter)
        for (int it = max(0, n_iter - C::kStages); it < n_iter; ++it)
          if (!warp_wait(BAR(kBQE + it % C::kStages), (it / C::kStages) & 1, ctl, a.status,
                         a.wait_limit_ns))
            break;
    }
  } else if (warp == 1) {
    if (n_iter > 0) {
      constexpr uint32_t idesc = idesc_bf16(128, BN, 0, 0);
      const uint64_t kd = sw128_desc(sbase, 16, 1024);
      bool ok = warp_wait(BAR(kBK), 0, ctl, a.status, a.wait_limit_ns);
      for (int it = 0; ok && it < n_iter; ++it) {
        const int st = it % C::kStages, u = it / C::kStages, sb = it & 1;
        if (!warp_wait(BAR(kBQF + st), u & 1, ctl, a.status, a.wait_limit_ns)) break;
        if (!warp_wait(BAR(kBSE + sb), ((it >> 1) & 1) ^ 1, ctl, a.status, a.wait_limit_ns)) break;
        tc_fence_after();
        const uint64_t qd = sw128_desc(sbase + C::kQOff + st * C::kQBytes, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < DQK / 16; ++kk)
            umma_ss(tmem + sb * BN, kd + (((kk >> 2) * C::kKPanel + (kk & 3) * 32) >> 4),
                    qd + (((kk >> 2) * C::kQPanel + (kk & 3) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
          umma_commit(BAR(kBSF + sb));
          umma_commit(BAR(kBQE + st));
        }
        __syncwarp();
      }
    }
  } else {
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int64_t j = static_cast<int64_t>(nt) * 128 + r;
    const bool key_ok = j < a.Sk;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* lbuf = reinterpret_cast<float*>(smem + C::kLOff);
    const int tq = threadIdx.x - 64;  // the query of a step whose lse this thread fetches
    constexpr int kWords = BN / 32;
    float l_nxt = 0.f;
    uint32_t w_nxt[kWords];
    auto fetch = [&](int it) {
      if (it >= n_iter) return;
      int h, m0;
      bool partial;
      decode(it, h, m0, partial);
      if (tq < BN) {
        const int64_t i = static_cast<int64_t>(m0) + tq;
        // (a row past Sq, or one that saw no key, adds nothing: exp2(-inf))
        float l = -INFINITY;
        if (i < a.Sq) l = __ldg(a.lse + (static_cast<int64_t>(b) * a.HQ + h) * a.Sq + i);
        l_nxt = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
      }
      if (partial && a.mode == SA_MODE_INDEX) {
        // presence word of query m0 + 32 c + lane over this warp's 32 keys
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
          const int64_t i = static_cast<int64_t>(m0) + 32 * c + lane;
          const int w = nt * 4 + quarter;
          w_nxt[c] = (i < a.Sq && w < a.W) ? __ldg(a.bitmap + (bg * a.Sq + i) * a.W + w) : 0u;
        }
      }
    };
    fetch(0);
    float total = 0.f;
    bool ok = true;
    for (int it = 0; it < n_iter; ++it) {
      int h, m0;
      bool partial;
      decode(it, h, m0, partial);
      const int sb = it & 1;
      float* ls = lbuf + sb * BN;
      if (tq < BN) ls[tq] = l_nxt;
      uint32_t cm[kWords];
#pragma unroll
      for (int c = 0; c < kWords; ++c) cm[c] = 0xFFFFFFFFu;
      if (partial) {
#pragma unroll
        for (int c = 0; c < kWords; ++c) {
          const int64_t q0 = static_cast<int64_t>(m0) + 32 * c;
          uint32_t x = key_ok ? 0xFFFFFFFFu : 0u;
          if (a.causal) {  // i >= j
            const int64_t lo = j - q0;
            x &= lo <= 0 ? 0xFFFFFFFFu : (lo >= 32 ? 0u : (0xFFFFFFFFu << lo));
          }
          if (a.mode == SA_MODE_BLOCK && a.bs == 64 && key_ok) {
            const int64_t mb = q0 / 64;
            const bool m = mb < a.Mb &&
                           __ldg(a.mask + (bg * a.Mb + mb) * static_cast<int64_t>(a.Nb) + j / 64) != 0;
            if (!m) x = 0u;
          } else if (a.mode == SA_MODE_INDEX) {
            x &= warp_transpose32(w_nxt[c], lane);
          }
          cm[c] = x;
        }
      }
      fetch(it + 1);
      // (the four warps meet once a step: the other lse buffer is free, this one is full;
      // they also leave together)
      const bool w_ok = __all_sync(
          0xFFFFFFFFu, mbar_wait(BAR(kBSF + sb), (it >> 1) & 1, ctl, a.status, a.wait_limit_ns));
      if (!named_bar_and(1, 128, w_ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* ls4 = reinterpret_cast<const float4*>(ls);
      const float sc = a.scale_log2;
      float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kWords; ++c) {
        uint32_t s[32];
        tmem_ld32(tl + sb * BN + 32 * c, s);
        tmem_wait_ld();
        if (c == kWords - 1) {  // every column is read: the buffer is free
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
    if (ok && key_ok) {
      if (ka.splits > 1) {
        ka.part[(static_cast<int64_t>(sp) * bgs + bg) * a.Sk + j] = total;
      } else {
        const int64_t at = bg * a.Sk + j;
        ka.w_out[at] = ka.w_in ? ka.w_in[at] + total : total;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // Abort path: no warp issues anything past the barrier above.  Wait (with a limit) for the
  // copies and MMAs in flight before shared and tensor memory are released.
  if (ctl->abort && n_iter > 0) {
    if (warp == 0 && lane == 0) {
      mbar_wait_limited(BAR(kBK), 0);
      for (int it = max(0, issued - C::kStages); it < issued; ++it)
        mbar_wait_limited(BAR(kBQF + it % C::kStages), (it / C::kStages) & 1);
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
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// w_out = w_in + the parts in order
__global__ void __launch_bounds__(256) key_weights_sum_kernel(const float* __restrict__ part,
                                                              const float* w_in, float* w_out,
                                                              int64_t n, int splits) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int k = 0; k < splits; ++k) s += part[k * n + i];
  w_out[i] = w_in ? w_in[i] + s : s;
}

// CTAs over which the queries of one key tile are split: enough to fill the SMs (one wave),
// at least four steps each.
static int splits_of(const sparse_attn_params* p, int sms) {
  const int64_t tn = (p->Sk + 127) / 128, tm = (p->Sq + 127) / 128;
  const int64_t ctas = tn * p->B * p->HK;
  const int64_t room = static_cast<int64_t>(sms) * (p->Dqk == 256 ? 1 : 2);
  const int64_t steps = p->HQ / p->HK * tm * (p->Dqk <= 128 ? 1 : 2);
  const int64_t s = min64(room / ctas, steps / 4);
  return static_cast<int>(max64(1, min64(s, 64)));
}

static int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    (void)cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  (void)cudaGetLastError();
  return sms;
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
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.t.Tn) * a.t.B * a.t.HK * a.splits);
  key_weights_kernel<DQK><<<grid, 192, C::kSmem, st>>>(mq, mk, a);
  return check_launch("key weights kernel launch");
}

}  // namespace kweights
}  // namespace sa

using namespace sa;

extern "C" size_t sparse_attn_key_weights_workspace_size(const sparse_attn_params* p) {
  if (!p || p->B <= 0 || p->HQ <= 0 || p->HK <= 0 || p->Sq <= 0 || p->Sk <= 0 || p->Dqk <= 0)
    return 0;
  const int s = kweights::splits_of(p, kweights::sm_count());
  return s > 1 ? sizeof(float) * static_cast<size_t>(s) * p->B * p->HK * static_cast<size_t>(p->Sk) : 0;
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t need = sparse_attn_key_weights_workspace_size(p);
  if (need && (!workspace || workspace_bytes < need ||
               (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
    return SA_ERR_WORKSPACE;
  rc = check_stream_device(st);
  if (rc) return rc;
  a.w_in = weights;
  a.w_out = weights_out;
  a.splits = kweights::splits_of(p, kweights::sm_count());
  a.part = static_cast<float*>(workspace);
  if (static_cast<int64_t>(a.t.Tn) * p->B * p->HK * a.splits > 0x7FFFFFFF) return SA_ERR_UNSUPPORTED;
  CUtensorMap mq, mk;
  if (!make_map(&mq, p->q, p->Dqk, p->Sq, p->HQ, p->B, p->Dqk <= 128 ? 128 : 64)) return SA_ERR_CUDA;
  if (!make_map(&mk, p->k, p->Dqk, p->Sk, p->HK, p->B, 128)) return SA_ERR_CUDA;
  if (p->Dqk == 64) rc = kweights::launch<64>(a, mq, mk, st);
  else if (p->Dqk == 128) rc = kweights::launch<128>(a, mq, mk, st);
  else if (p->Dqk == 192) rc = kweights::launch<192>(a, mq, mk, st);
  else rc = kweights::launch<256>(a, mq, mk, st);
  if (rc || a.splits == 1) return rc;
  const int64_t n = static_cast<int64_t>(p->B) * p->HK * p->Sk;
  kweights::key_weights_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, st>>>(
      a.part, weights, weights_out, n, a.splits);
  return check_launch("key weights sum kernel launch");
}
