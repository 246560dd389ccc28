// sa_kernels.h -- host-side launch interface shared by the C-ABI layer and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "sparse_attn.h"

namespace sa {

// Everything a forward or backward launch needs besides the TMA tensor maps.
struct AttnArgs {
  void* o;               // bf16 [B][Sq][HQ][Dv]
  float* lse;            // fp32 [B][HQ][Sq]
  const void* dout;      // bf16 [B][Sq][HQ][Dv]
  void* dq;              // bf16 [B][Sq][HQ][Dqk]
  void* dk;              // bf16 [B][Sk][HK][Dqk]
  void* dv;              // bf16 [B][Sk][HK][Dv]
  float* delta;          // fp32 [B][HQ][Sq]   (backward workspace)
  float* dq_acc;         // fp32 [B][Sq][HQ][Dqk] (backward workspace)
  const int32_t* cnt;    // forward lists
  const int32_t* idx;
  const int32_t* tcnt;   // backward (transposed) lists
  const int32_t* tidx;
  const uint8_t* mask;   // block mode, bs = 64 partial tiles
  const uint32_t* bitmap;  // index mode
  int64_t Sq, Sk;
  int B, HQ, HK, Dqk, Dv;
  int Tm, Tn, W;
  int mode, causal, bs, Mb, Nb;
  float scale;       // softmax_scale
  float scale_log2;  // softmax_scale * log2(e)
  int32_t* status;
  // deterministic backward: dQ contributions to each (b, query head, query tile, dQ
  // column part) are added in ascending key-tile order, sequenced by sem
  // [B][HQ][Tm][2] (backward workspace, zeroed by the preprocess)
  int det;
  int32_t* sem;
  // limit of every bounded wait of the launch (ns); kWaitLimitNs unless a test shortened
  // it through sparse_attn_set_wait_limit_ns
  uint64_t wait_limit_ns;
};

// Wait limit for the next launches (0: the default); see sparse_attn_set_wait_limit_ns.
extern std::atomic<uint64_t> g_wait_limit_ns;
// Forward form (SA_FWD_FORM_*); see sparse_attn_set_forward_form.
extern std::atomic<int> g_fwd_form;

struct TensorMaps {
  CUtensorMap q, k, v, dout, dq_acc, dk, dv, o;
  CUtensorMap kh;  // forward: K in 64-row boxes (the half tile of a CTA pair)
};

// Caller-owned events recorded around the launches (see sparse_attn_set_timing_events);
// nullptr when instrumentation is off.
extern cudaEvent_t* g_timing_events;
inline void record_event(int k, cudaStream_t st) {
  if (g_timing_events) cudaEventRecord(g_timing_events[k], st);
}

// Turns a CUDA error into SA_ERR_CUDA; with SA_DEBUG set in the environment it also
// prints which call failed and why.
int cuda_error(cudaError_t e, const char* what);
inline int check_launch(const char* what) { return cuda_error(cudaGetLastError(), what); }

// Launches `kern` so that it may start before the kernel ahead of it in the stream has ended
// (it waits for that kernel itself, wait_previous_kernel()): its launch and set-up overlap
// that kernel's end.  `cluster`: CTAs of a cluster (along x).
template <class... P, class... A>
inline int launch_early(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                        const char* what, int cluster, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cuda_error(cudaLaunchKernelEx(&cfg, kern, args...), what);
}

// Runs `set` (a cudaFuncSetAttribute call and the like) once per device: a flag bit per
// device index (< 64), set only when `set` returns SA_OK, so a failure is retried on
// the next call; thread-safe.  Device = the current device.
struct PerDeviceOnce {
  std::atomic<uint64_t> done{0};
  std::mutex m;
};
template <class F>
inline int once_per_device(PerDeviceOnce& o, F&& set) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SA_ERR_CUDA;
  const uint64_t bit = 1ull << dev;
  if (o.done.load(std::memory_order_acquire) & bit) return SA_OK;
  std::lock_guard<std::mutex> lock(o.m);
  if (o.done.load(std::memory_order_relaxed) & bit) return SA_OK;
  const int rc = set();
  if (rc == SA_OK) o.done.fetch_or(bit, std::memory_order_release);
  return rc;
}

// 4-D tensor map over a [B][S][H][D] bf16 tensor (dimension order D, S, H, B) with
// 64 x box_rows x box_heads (D x S x H) boxes, 128-byte swizzle.  Out-of-range rows (and
// columns) read as zeros.
bool make_map(CUtensorMap* m, const void* base, int D, int64_t S, int H, int B, int box_rows,
              int box_heads = 1);

// Checks an attention call's parameters and fills the launch arguments from them.
int fill_args(const sparse_attn_params* p, AttnArgs* a, bool backward);

// Whether two arrays of n elements share memory without being the same array: a kernel that reads
// one element and writes another of the same index may then read what it has already written.
template <class T>
inline bool partly_overlap(const T* a, const T* b, int64_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x != y && (x < y ? y - x : x - y) / sizeof(T) < static_cast<uint64_t>(n);
}

// Every kernel is launched on the current device.  A stream created on another device
// is refused with SA_ERR_DEVICE before anything is enqueued (the legacy and per-thread
// default streams always belong to the current device).
int check_stream_device(cudaStream_t st);

int launch_fwd(const AttnArgs& a, const TensorMaps& m, cudaStream_t st);
int launch_bwd(const AttnArgs& a, const TensorMaps& m, cudaStream_t st);
int launch_bwd_pair(const AttnArgs& a, const TensorMaps& m, cudaStream_t st);

}  // namespace sa
