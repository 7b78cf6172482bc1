// fp8train.cu — the C ABI declared in include/fp8train.h: host-side validation, launch
// configuration and tensor-map encoding for the four kernels of the FP8 delayed-scaling Linear
// step. Every argument is checked before the first CUDA call, so invalid input returns an error
// status and launches nothing; there is no fallback path.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <functional>
#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "fp8train.h"
#include "cast_transpose_amax.cuh"
#include "current_scaling.cuh"
#include "fp4_cast.cuh"
#include "fused_adamw.cuh"
#include "gemm_tcgen05.cuh"
#include "gemm_mx_wide.cuh"
#include "gemm_fp4.cuh"
#include "fp4_matvec.cuh"
#include "gated.cuh"
#include "gated_rows.cuh"
#include "muon.cuh"
#include "mx_cast.cuh"
#include "rmsnorm.cuh"
#include "scale_update.cuh"

namespace {

thread_local std::string t_last_error;

fp8t_status fail(fp8t_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return s;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  int state = 0;               // 0 unknown, 1 sm_100, 2 other
  int sms = 0;
  int adamw_blocks_per_sm = 0;
  int adamw_cast_blocks_per_sm = 0;
  int gemm_clusters = 0;       // co-resident 2-CTA clusters of the GEMM kernel
  int gemm_wide_clusters = 0;  // ... of its wide-tile form
  int gemm_mx_clusters = 0;    // ... of its MXFP8 variant
  int gemm_mxw_clusters = 0;   // ... of the MXFP8 256 x 384 kernel
  int mx_cast_blocks_per_sm = 0;
  int cast_blocks_per_sm = 0;
  int cast_rowmajor_blocks_per_sm = 0;
  void* noalloc_scratch = nullptr;   // device address of g_adamw_noalloc_scratch
  // set up by their own first calls, so that no other call loads these kernels or fails with them
  std::atomic<bool> fp4_cast_ready{false}, fp4_gemm_ready{false}, norm_backward_ready{false}, pair_ready{false}, gated_rows_ready{false};
  int fp4_cast_blocks_per_sm = 0;
  int fp4_cast_rows_blocks_per_sm = 0;
  int pair_clusters = 0;             // co-resident clusters of the pair-tile products (one CTA per SM)
  int gemm_fp4_clusters = 0;         // co-resident clusters of the 4-bit tile kernel (every form: one CTA per SM)
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mutex;

template <bool NV, int BT>
cudaError_t allow_fp4_split_smem_of() {
  return cudaFuncSetAttribute(fp8t::gemm::k_fp4_gemm_split<NV, BT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fp8t::gemm::SplitShape<NV, BT>::kSmem);
}
template <bool NV, bool WIDE, class G>
cudaError_t allow_fp4_tile_smem_of() {
  return cudaFuncSetAttribute(fp8t::gemm::k_fp4_gemm<NV, WIDE, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fp8t::gemm::kSmemBytes4<NV, WIDE>);
}
template <class G>
cudaError_t allow_fp4_tile_smem() {
  cudaError_t e;
  if ((e = allow_fp4_tile_smem_of<false, false, G>()) != cudaSuccess || (e = allow_fp4_tile_smem_of<true, false, G>()) != cudaSuccess ||
      (e = allow_fp4_tile_smem_of<false, true, G>()) != cudaSuccess)
    return e;
  return allow_fp4_tile_smem_of<true, true, G>();
}
cudaError_t allow_fp4_split_smem() {
  cudaError_t e;
  if ((e = allow_fp4_split_smem_of<false, 16>()) != cudaSuccess || (e = allow_fp4_split_smem_of<true, 16>()) != cudaSuccess ||
      (e = allow_fp4_split_smem_of<false, 32>()) != cudaSuccess || (e = allow_fp4_split_smem_of<true, 32>()) != cudaSuccess ||
      (e = allow_fp4_split_smem_of<false, 64>()) != cudaSuccess || (e = allow_fp4_split_smem_of<true, 64>()) != cudaSuccess ||
      (e = allow_fp4_split_smem_of<false, 128>()) != cudaSuccess)
    return e;
  return allow_fp4_split_smem_of<true, 128>();
}

// Current device must be compute capability 10.0 (sm_100a code runs there only).
fp8t_status current_device(DeviceInfo** out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(FP8T_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(FP8T_ERR_UNSUPPORTED_DEVICE, "device index %d", dev);
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  DeviceInfo& d = g_dev[dev];
  if (d.state == 0) {
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return fail(FP8T_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    d.sms = sms;
    d.state = (major == 10 && minor == 0) ? 1 : 2;
    if (d.state == 1) {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.adamw_blocks_per_sm,
                                                        fp8t::adamw::k_adamw_update<false>,
                                                        fp8t::adamw::kThreads, 0);
      if (e != cudaSuccess || d.adamw_blocks_per_sm < 1) d.adamw_blocks_per_sm = 1;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.adamw_cast_blocks_per_sm,
                                                        fp8t::adamw::k_adamw_update<true>,
                                                        fp8t::adamw::kThreads, 0);
      if (e != cudaSuccess || d.adamw_cast_blocks_per_sm < 1) d.adamw_cast_blocks_per_sm = 1;
      e = cudaFuncSetAttribute(fp8t::gemm::k_fp8_gemm<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               fp8t::gemm::kSmemBytes);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fp8t::gemm::k_fp8_gemm<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 fp8t::gemm::kSmemBytesMX);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fp8t::gemm::k_fp8_gemm_wide, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 fp8t::gemm::kSmemBytesW);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fp8t::mx::k_mx_cast, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 fp8t::mx::kSmemBytes);
      if (e != cudaSuccess) {
        d.state = 0;
        return fail(FP8T_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      }
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
      cfg.blockDim = dim3(fp8t::gemm::kThreads, 1, 1);
      cfg.dynamicSmemBytes = fp8t::gemm::kSmemBytes;
      int clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, fp8t::gemm::k_fp8_gemm<false>, &cfg);
      if (e != cudaSuccess || clusters < 1) {
        (void)cudaGetLastError();
        clusters = sms / 2;
      }
      d.gemm_clusters = clusters;
      cfg.blockDim = dim3(fp8t::gemm::kThreadsW, 1, 1);
      cfg.dynamicSmemBytes = fp8t::gemm::kSmemBytesW;
      clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, fp8t::gemm::k_fp8_gemm_wide, &cfg);
      if (e != cudaSuccess || clusters < 1) {
        (void)cudaGetLastError();
        clusters = sms / 2;
      }
      d.gemm_wide_clusters = clusters;
      cfg.blockDim = dim3(fp8t::gemm::kThreads, 1, 1);
      cfg.dynamicSmemBytes = fp8t::gemm::kSmemBytesMX;
      clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, fp8t::gemm::k_fp8_gemm<true>, &cfg);
      if (e != cudaSuccess || clusters < 1) {
        (void)cudaGetLastError();
        clusters = sms / 2;
      }
      d.gemm_mx_clusters = clusters;
      e = cudaFuncSetAttribute(fp8t::gemm::k_fp8_gemm_mx_wide,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, fp8t::gemm::kSmemBytesX);
      if (e != cudaSuccess) {
        d.state = 0;
        return fail(FP8T_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      }
      cfg.blockDim = dim3(fp8t::gemm::kThreadsX, 1, 1);
      cfg.dynamicSmemBytes = fp8t::gemm::kSmemBytesX;
      clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, fp8t::gemm::k_fp8_gemm_mx_wide, &cfg);
      if (e != cudaSuccess || clusters < 1) {
        (void)cudaGetLastError();
        clusters = sms / 2;
      }
      d.gemm_mxw_clusters = clusters;
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.mx_cast_blocks_per_sm, fp8t::mx::k_mx_cast,
                                                        fp8t::mx::kThreads, fp8t::mx::kSmemBytes);
      if (e != cudaSuccess || d.mx_cast_blocks_per_sm < 1) {
        (void)cudaGetLastError();
        d.mx_cast_blocks_per_sm = 1;
      }
      e = cudaFuncSetAttribute(fp8t::cast::k_cast_transpose_amax<false>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, fp8t::cast::kSmemBytes);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fp8t::cast::k_cast_transpose_amax<true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, fp8t::cast::kSmemBytes);
      if (e != cudaSuccess) {
        d.state = 0;
        return fail(FP8T_ERR_CUDA, "cudaFuncSetAttribute(cast): %s", cudaGetErrorString(e));
      }
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.cast_rowmajor_blocks_per_sm,
                                                        fp8t::cast::k_cast_rowmajor<true>,
                                                        fp8t::cast::kThreads, 0);
      if (e != cudaSuccess || d.cast_rowmajor_blocks_per_sm < 1) {
        (void)cudaGetLastError();
        d.cast_rowmajor_blocks_per_sm = 1;
      }
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.cast_blocks_per_sm,
                                                        fp8t::cast::k_cast_transpose_amax<true>,
                                                        fp8t::cast::kThreads, fp8t::cast::kSmemBytes);
      if (e != cudaSuccess || d.cast_blocks_per_sm < 1) {
        (void)cudaGetLastError();
        d.cast_blocks_per_sm = 1;
      }
    }
  }
  if (d.state != 1) return fail(FP8T_ERR_UNSUPPORTED_DEVICE, "device %d is not sm_100", dev);
  *out = &d;
  return FP8T_OK;
}

// Runs `set_up` (a cudaError_t) once per device for the calls that need it; a failure is tried again by the next call.
template <class F>
fp8t_status once_per_device(std::atomic<bool>& ready, const char* what, F&& set_up) {
  if (ready.load(std::memory_order_acquire)) return FP8T_OK;
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  if (ready.load(std::memory_order_relaxed)) return FP8T_OK;
  const cudaError_t e = set_up();
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(FP8T_ERR_CUDA, "%s: setting up its kernels: %s", what, cudaGetErrorString(e));
  }
  ready.store(true, std::memory_order_release);
  return FP8T_OK;
}
template <class K>
int resident_blocks(K* kernel, int threads, int smem) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) == cudaSuccess && n > 0) return n;
  (void)cudaGetLastError();
  return 1;
}
fp8t_status ready_fp4_cast(DeviceInfo* d) {
  using namespace fp8t::fp4;
  return once_per_device(d->fp4_cast_ready, "fp4_cast", [&] {
    const cudaError_t e = cudaFuncSetAttribute(k_fp4_cast, cudaFuncAttributeMaxDynamicSharedMemorySize, kCastSmemBytes);
    if (e == cudaSuccess) {
      d->fp4_cast_blocks_per_sm = resident_blocks(k_fp4_cast, kCastThreads, kCastSmemBytes);
      d->fp4_cast_rows_blocks_per_sm = resident_blocks(k_fp4_cast_rows, kCastThreads, 0);
    }
    return e;
  });
}
fp8t_status ready_fp4_gemm(DeviceInfo* d) {
  using namespace fp8t::gemm;
  return once_per_device(d->fp4_gemm_ready, "fp4_gemm", [&] {
    cudaError_t e = allow_fp4_tile_smem<SmallGroup4>();
    if (e == cudaSuccess) e = allow_fp4_tile_smem<LargeGroup4>();
    if (e == cudaSuccess) e = allow_fp4_tile_smem<ListGroup4>();
    if (e == cudaSuccess) e = allow_fp4_split_smem();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (d->sms / 2), 1, 1);
    cfg.blockDim = dim3(kThreads4, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes4<true, true>;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, k_fp4_gemm<true, true, ListGroup4>, &cfg) != cudaSuccess || clusters < 1) {
      (void)cudaGetLastError();
      clusters = d->sms / 2;
    }
    d->gemm_fp4_clusters = clusters;
    return cudaSuccess;
  });
}
fp8t_status ready_norm_backward(DeviceInfo* d) {
  using namespace fp8t::norm;
  return once_per_device(d->norm_backward_ready, "fp8_rmsnorm_backward", [] {
    cudaError_t e = cudaSuccess;
    for (auto* k : {k_rmsnorm_backward<1>, k_rmsnorm_backward<2>, k_rmsnorm_backward<3>, k_rmsnorm_backward<4>})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdMaxSmem);
    return e;
  });
}

// A launch that may begin while the kernel before it in the stream still runs (the kernel calls pdl_wait).
template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), int64_t grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                       const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cluster > 0) {                   // a size chosen at launch (kernels without their own)
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

fp8t_status after_launch(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(FP8T_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return FP8T_OK;
}

// ------------------------------------------------------------------ tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// rows x K bytes, row-major: boxes of box_rows rows x 128 bytes, 128-byte swizzle, zero fill.
fp8t_status encode_kmajor(CUtensorMap* map, const void* ptr, int64_t rows, int64_t K,
                          uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(fp8t::gemm::kBK), box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return FP8T_OK;
}

// K rows x N bytes, row-major, read as an MN-major operand in boxes of 64 columns x 128 K rows with
// the 64-byte swizzle, zero fill.
fp8t_status encode_mn64(CUtensorMap* map, const void* ptr, int64_t K, int64_t N) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(K)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(N)};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(fp8t::gemm::kBK)};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (64-column box) failed (%d)", (int)r);
  return FP8T_OK;
}

// ------------------------------------------------------------------ AdamW helpers
struct AdamWPlan {
  int nbatches = 0;
  int64_t nparts = 0;
};

int64_t chunks_of(int64_t numel) { return (numel + fp8t::adamw::kChunk - 1) / fp8t::adamw::kChunk; }

AdamWPlan plan_adamw(const fp8t_adamw_tensor* t, int32_t n) {
  AdamWPlan p;
  for (int32_t b0 = 0; b0 < n; b0 += fp8t::adamw::kMaxTensors) {
    int64_t chunks = 0;
    const int32_t b1 = std::min<int32_t>(n, b0 + fp8t::adamw::kMaxTensors);
    for (int32_t i = b0; i < b1; ++i) chunks += chunks_of(t[i].numel);
    p.nparts += std::min<int64_t>(chunks, fp8t::adamw::kSumsqBlocks);
    ++p.nbatches;
  }
  return p;
}

// One double per norm partial, then one int64 slot for the step a device-counted call performs.
size_t workspace_for(const AdamWPlan& p) {
  return static_cast<size_t>(((p.nparts + 1) * 8 + 255) / 256 * 256);
}

}  // namespace

// Scratch of fused_adamw_multi_tensor_noalloc, for callers that cannot allocate: a file-scope
// device array, present on every GPU that loads the library until the process exits. In host
// code this name is only a stand-in; its device address comes from cudaGetSymbolAddress.
static __device__ __align__(256) unsigned char g_adamw_noalloc_scratch[FP8T_NOALLOC_SCRATCH_BYTES];

extern "C" {

int32_t fp8t_abi_version(void) { return 2; }

const char* fp8t_last_error_message(void) { return t_last_error.c_str(); }

const char* fp8t_status_string(fp8t_status s) {
  switch (s) {
    case FP8T_OK: return "FP8T_OK";
    case FP8T_ERR_INVALID_ARG: return "FP8T_ERR_INVALID_ARG";
    case FP8T_ERR_UNSUPPORTED_SHAPE: return "FP8T_ERR_UNSUPPORTED_SHAPE";
    case FP8T_ERR_MISALIGNED: return "FP8T_ERR_MISALIGNED";
    case FP8T_ERR_UNSUPPORTED_DEVICE: return "FP8T_ERR_UNSUPPORTED_DEVICE";
    case FP8T_ERR_CUDA: return "FP8T_ERR_CUDA";
    case FP8T_ERR_TIMEOUT: return "FP8T_ERR_TIMEOUT";
  }
  return "FP8T_UNKNOWN_STATUS";
}

// ------------------------------------------------------------------ cast / transpose / amax
}  // extern "C"

namespace {

// Casts of n tensors in launches of up to eight; with `updates`, the last CTA of each launch also
// performs the delayed-scaling update of that launch's tensors; with `current_ws`, each launch
// is preceded by the current-scaling amax pass that sets the scales it uses.
fp8t_status cast_multi(const fp8t_cast_tensor* tensors, const fp8t_cast_update* updates,
                       int32_t n_tensors, int32_t history_len, fp8t_amax_algo algo, int32_t margin,
                       unsigned int* d_ticket, unsigned int* current_ws, void* stream) {
  t_last_error.clear();
  if (!tensors || n_tensors < 1 || n_tensors > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax: tensors NULL or n_tensors out of range");
  if (current_ws && (!aligned(current_ws, 4) || margin < 0 || margin > 126))
    return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_current: misaligned workspace or margin outside 0..126");
  if (updates) {
    if (!d_ticket || !aligned(d_ticket, 4))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_update: NULL or misaligned ticket");
    if (history_len < 1 || history_len > 65536)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_update: history_len in 1..65536");
    if (algo != FP8T_AMAX_MAX && algo != FP8T_AMAX_MOST_RECENT)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_update: unknown amax algorithm %d", (int)algo);
    if (margin < 0 || margin > 126)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_update: margin in 0..126");
    for (int32_t i = 0; i < n_tensors; ++i) {
      const fp8t_cast_update& u = updates[i];
      if (!u.d_amax_history || !u.d_scale_inv_next)
        return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_update: tensor %d: NULL history or scale_inv_next", i);
      if (!aligned(u.d_amax_history, 4) || !aligned(u.d_scale_inv_next, 4))
        return fail(FP8T_ERR_MISALIGNED, "fp8_cast_transpose_amax_update: tensor %d: misaligned pointer", i);
      if (u.d_scale_inv_next == tensors[i].d_scale_inv_out)
        return fail(FP8T_ERR_INVALID_ARG,
                    "fp8_cast_transpose_amax_update: tensor %d: scale_inv_next must differ from the cast's scale_inv_out", i);
    }
  }
  for (int32_t i = 0; i < n_tensors; ++i) {
    const fp8t_cast_tensor& t = tensors[i];
    if (updates && !t.x_bf16 && t.rows == 0 && t.cols == 0 && !t.q_rowmajor && !t.q_transposed &&
        !t.d_counters && t.d_scale && t.d_amax_inout && aligned(t.d_scale, 4) &&
        aligned(t.d_amax_inout, 4) && aligned(t.d_scale_inv_out, 4) &&
        (t.fmt == FP8T_E4M3 || t.fmt == FP8T_E5M2))
      continue;                       // scale update only: the amax was accumulated elsewhere
    if (!t.x_bf16 || !t.d_scale || !t.d_amax_inout)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax: tensor %d: NULL input, scale or amax pointer", i);
    if (t.fmt != FP8T_E4M3 && t.fmt != FP8T_E5M2)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax: tensor %d: unknown format %d", i, (int)t.fmt);
    if (t.rows <= 0 || t.cols <= 0)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax: tensor %d: rows and cols must be > 0", i);
    if (t.rows % 16 || t.cols % 16 || t.rows > (int64_t(1) << 31) || t.cols > (int64_t(1) << 31) ||
        t.rows * t.cols >= (int64_t(1) << 40))
      return fail(FP8T_ERR_UNSUPPORTED_SHAPE,
                  "fp8_cast_transpose_amax: tensor %d: rows and cols must be multiples of 16, rows*cols < 2^40", i);
    if (!aligned(t.x_bf16, 16) || !aligned(t.q_rowmajor, 16) || !aligned(t.q_transposed, 16) ||
        !aligned(t.d_scale, 4) || !aligned(t.d_amax_inout, 4) || !aligned(t.d_scale_inv_out, 4) ||
        !aligned(t.d_counters, 8))
      return fail(FP8T_ERR_MISALIGNED, "fp8_cast_transpose_amax: tensor %d: misaligned pointer", i);
  }
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");

  using namespace fp8t::cast;
  static thread_local Group group;
  for (int32_t b0 = 0; b0 < n_tensors; b0 += kMaxTensors) {
    const int32_t b1 = std::min<int32_t>(n_tensors, b0 + kMaxTensors);
    std::memset(&group, 0, sizeof(group));
    group.n = b1 - b0;
    int64_t tiles = 0;
    for (int32_t i = b0; i < b1; ++i) {
      const fp8t_cast_tensor& t = tensors[i];
      Tensor& T = group.t[i - b0];
      if (t.x_bf16) {
        cuuint64_t dims[2] = {static_cast<cuuint64_t>(t.cols), static_cast<cuuint64_t>(t.rows)};
        cuuint64_t strides[1] = {static_cast<cuuint64_t>(t.cols) * 2};
        cuuint32_t box[2] = {kTile, kTile};
        cuuint32_t es[2] = {1, 1};
        CUresult r = fn(&T.x_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(t.x_bf16),
                        dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (cast input) failed (%d)", (int)r);
      }
      if (t.q_transposed) {
        cuuint64_t dims[2] = {static_cast<cuuint64_t>(t.rows), static_cast<cuuint64_t>(t.cols)};
        cuuint64_t strides[1] = {static_cast<cuuint64_t>(t.rows)};
        cuuint32_t box[2] = {kTile, kTile};
        cuuint32_t es[2] = {1, 1};
        CUresult r = fn(&T.qt_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, t.q_transposed, dims, strides,
                        box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (q^T store) failed (%d)", (int)r);
      }
      T.scale = const_cast<float*>(t.d_scale);      // written only by the update
      T.x = static_cast<const uint4*>(t.x_bf16);
      T.amax_bits = reinterpret_cast<unsigned int*>(t.d_amax_inout);
      T.scale_inv = t.d_scale_inv_out;
      if (updates) {
        T.hist = updates[i].d_amax_history;
        T.scale_inv_next = updates[i].d_scale_inv_next;
      }
      T.counters = t.d_counters;
      T.q = static_cast<uint8_t*>(t.q_rowmajor);
      T.rows = t.rows;
      T.cols = t.cols;
      T.tiles_c = (t.cols + kTile - 1) / kTile;
      T.tile_start = tiles;
      T.fmt = t.fmt;
      T.has_qt = t.q_transposed ? 1 : 0;
      tiles += ((t.rows + kTile - 1) / kTile) * T.tiles_c;
    }
    group.total_tiles = tiles;
    if (updates) {
      group.update = 1;
      group.ticket = d_ticket;
      group.H = history_len;
      group.algo_max = algo == FP8T_AMAX_MAX ? 1 : 0;
      group.margin = margin;
    }
    bool count = false, any_qt = false;
    for (int32_t i = b0; i < b1; ++i) {
      count |= tensors[i].d_counters != nullptr;
      any_qt |= tensors[i].q_transposed != nullptr;
    }
    int64_t grid = std::min<int64_t>(tiles, static_cast<int64_t>(dev->sms) * dev->cast_blocks_per_sm);
    if (grid < 1) grid = 1;           // update-only entries: one CTA does the update
    if (current_ws) {                  // the scales of this group, from its own amax
      fp8t::current::Group cg;
      std::memset(&cg, 0, sizeof(cg));
      cg.n = b1 - b0;
      cg.margin = margin;
      cg.ws = current_ws;
      int64_t vecs = 0;
      for (int32_t i = b0; i < b1; ++i) {
        cg.x[i - b0] = static_cast<const uint4*>(tensors[i].x_bf16);
        cg.nvec[i - b0] = tensors[i].rows * tensors[i].cols / 8;
        cg.scale[i - b0] = const_cast<float*>(tensors[i].d_scale);
        cg.fp8_max[i - b0] = tensors[i].fmt == FP8T_E4M3 ? 448.0f : 57344.0f;
        vecs += cg.nvec[i - b0];
      }
      const int64_t cgrid = std::max<int64_t>(1, std::min<int64_t>(
          (vecs + fp8t::current::kThreads - 1) / fp8t::current::kThreads, 4 * static_cast<int64_t>(dev->sms)));
      fp8t::current::k_current_amax<<<static_cast<unsigned>(cgrid), fp8t::current::kThreads, 0,
                                      as_stream(stream)>>>(cg);
      if ((st = after_launch("current-scaling amax launch")) != FP8T_OK) return st;
    }
    if (!any_qt) {                     // row-major codes only: the streaming kernel
      int64_t segs = 0;
      for (int32_t i = b0; i < b1; ++i) segs += tensors[i].rows * tensors[i].cols / 16;
      const int64_t rgrid = std::max<int64_t>(1, std::min<int64_t>(
          (segs + kThreads - 1) / kThreads, static_cast<int64_t>(dev->sms) * dev->cast_rowmajor_blocks_per_sm));
      if (count)
        k_cast_rowmajor<true><<<static_cast<unsigned>(rgrid), kThreads, 0, as_stream(stream)>>>(group);
      else
        k_cast_rowmajor<false><<<static_cast<unsigned>(rgrid), kThreads, 0, as_stream(stream)>>>(group);
    } else if (count) {
      k_cast_transpose_amax<true><<<static_cast<unsigned>(grid), kThreads, kSmemBytes, as_stream(stream)>>>(group);
    } else {
      k_cast_transpose_amax<false><<<static_cast<unsigned>(grid), kThreads, kSmemBytes, as_stream(stream)>>>(group);
    }
    if ((st = after_launch("fp8_cast_transpose_amax launch")) != FP8T_OK) return st;
  }
  return FP8T_OK;
}

}  // namespace

extern "C" {

fp8t_status fp8_cast_transpose_amax_multi(const fp8t_cast_tensor* tensors, int32_t n_tensors,
                                          void* stream) {
  return cast_multi(tensors, nullptr, n_tensors, 0, FP8T_AMAX_MAX, 0, nullptr, nullptr, stream);
}

fp8t_status fp8_cast_transpose_amax_update_multi(const fp8t_cast_tensor* tensors,
                                                 const fp8t_cast_update* updates, int32_t n_tensors,
                                                 int32_t history_len, fp8t_amax_algo algo,
                                                 int32_t margin, unsigned int* d_ticket,
                                                 void* stream) {
  if (!updates) {
    t_last_error.clear();
    return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_update: updates NULL");
  }
  return cast_multi(tensors, updates, n_tensors, history_len, algo, margin, d_ticket, nullptr,
                    stream);
}

fp8t_status fp8_cast_transpose_amax_current_multi(const fp8t_cast_tensor* tensors,
                                                  int32_t n_tensors, int32_t margin,
                                                  unsigned int* d_workspace, void* stream) {
  if (!d_workspace) {
    t_last_error.clear();
    return fail(FP8T_ERR_INVALID_ARG, "fp8_cast_transpose_amax_current: workspace NULL");
  }
  return cast_multi(tensors, nullptr, n_tensors, 0, FP8T_AMAX_MAX, margin, nullptr, d_workspace,
                    stream);
}

fp8t_status fp8_cast_transpose_amax(const void* x_bf16, int64_t rows, int64_t cols, fp8t_format fmt,
                                    const float* d_scale, void* q_rowmajor, void* q_transposed,
                                    float* d_amax_inout, float* d_scale_inv_out,
                                    unsigned long long* d_counters, void* stream) {
  const fp8t_cast_tensor t = {x_bf16, rows, cols, fmt, d_scale, q_rowmajor, q_transposed,
                              d_amax_inout, d_scale_inv_out, d_counters};
  return fp8_cast_transpose_amax_multi(&t, 1, stream);
}

// ------------------------------------------------------------------ GEMM
}  // extern "C"

namespace {

constexpr size_t kSumsqHeader = 256;    // ticket and abort words, then the partial slots

// Tile lists of a grouped GEMM launch: every tile costs its problem's K / 128 k-blocks (twice
// that for a wide tile); tiles are handed out longest first, each to the least-loaded cluster.
// A wide launch then splits tiles into their two 256-column halves, one half moving to the least
// busy cluster, while that lowers the busiest cluster's load. A half tile is costed at 0.58 of a
// whole one, not 0.5: it runs half the MMAs but loads all of A, the operand-starved pattern the
// wide tile avoids. (On the 4096 step this takes the busiest cluster from 704 to 678 k-block
// units with 28 splits, and the launch from ~0.295 to ~0.292 ms; costing halves at 0.5 split
// more and gained less. Timed per cluster, a half tile's k-block costs 0.76 of a whole one's and
// wgrad's k-blocks 8% more than dgrad's; costing the items that way, or running halves last,
// changed the launch by less than its run-to-run spread.) Every cluster then runs its items in
// index order. Items are 3 * tile + part.
// Launches with more tiles than the table holds keep round-robin (with thousands of tiles it is
// balanced already).
void build_schedule(fp8t::gemm::Group& g, int clusters, bool wide, bool mx_wide = false) {
  using namespace fp8t::gemm;
  g.scheduled = 0;
  if (g.total_tiles > kMaxSchedTiles || clusters > kMaxClusters || clusters < 2) return;
  struct Item { int64_t cost; int tile, part; };
  std::vector<Item> items;
  items.reserve(g.total_tiles);
  for (int p = 0; p < g.n; ++p) {
    const int end = p + 1 < g.n ? g.p[p + 1].tile_start : g.total_tiles;
    const int64_t kbs = (g.p[p].K + kBK - 1) / kBK;
    const int64_t cost = kbs * (wide ? 2 : 1);
    for (int t = g.p[p].tile_start; t < end; ++t) {
      // MX 256 x 384 tiles: three 128-column MMAs per k-step, two where N ends within the tile
      const int nt = (t - g.p[p].tile_start) % g.p[p].tiles_n;
      const int64_t c = mx_wide ? kbs * (nt * kBNx + 256 < g.p[p].N ? 3 : 2) : cost;
      items.push_back({c, t, 0});
    }
  }
  std::stable_sort(items.begin(), items.end(),
                   [](const Item& a, const Item& b) { return a.cost > b.cost; });
  std::vector<int64_t> load(clusters, 0);
  std::vector<std::vector<Item>> own(clusters);
  for (const auto& it : items) {
    int best = 0;
    for (int c = 1; c < clusters; ++c)
      if (load[c] < load[best]) best = c;
    load[best] += it.cost;
    own[best].push_back(it);
  }
  // a half tile runs about 0.58 of a whole one: half the MMAs, but all of A's loads
  auto half_cost = [](int64_t whole) { return (whole * 29 + 49) / 50; };
  int n_items = g.total_tiles;
  while (wide && n_items < kMaxSchedTiles) {
    int hi = 0, lo = 0;
    for (int c = 1; c < clusters; ++c) {
      if (load[c] > load[hi]) hi = c;
      if (load[c] < load[lo]) lo = c;
    }
    int pick = -1;                    // the whole tile of `hi` whose split lowers `hi` most
    int64_t best = load[hi];
    for (int k = 0; k < static_cast<int>(own[hi].size()); ++k) {
      const Item& it = own[hi][k];
      if (it.part != 0) continue;
      const int64_t h = half_cost(it.cost);
      const int64_t after = std::max(load[hi] - it.cost + h, load[lo] + h);
      if (after < best) {
        best = after;
        pick = k;
      }
    }
    if (pick < 0) break;
    Item& it = own[hi][pick];
    const int64_t h = half_cost(it.cost);
    load[hi] += h - it.cost;
    load[lo] += h;
    it.cost = h;
    it.part = 1;
    own[lo].push_back({h, it.tile, 2});
    ++n_items;
  }
  int k = 0;
  for (int c = 0; c < clusters; ++c) {
    std::sort(own[c].begin(), own[c].end(), [](const Item& a, const Item& b) {
      return a.tile != b.tile ? a.tile < b.tile : a.part < b.part;
    });
    g.start[c] = static_cast<uint16_t>(k);
    for (const auto& it : own[c]) g.order[k++] = static_cast<uint16_t>(3 * it.tile + it.part);
  }
  g.start[clusters] = static_cast<uint16_t>(k);
  g.scheduled = 1;
}

// Wide tiles (256 x 512 per pair) when every problem of the call is at least 512 wide; the choice
// is made for the whole call, so every launch of it numbers its sum-of-squares slots alike.
bool use_wide(const fp8t_gemm_desc* gemms, int32_t n) {
  for (int32_t i = 0; i < n; ++i)
    if (gemms[i].N < fp8t::gemm::kBNw) return false;
  return true;
}

int64_t gemm_tiles(const fp8t_gemm_desc& d, bool wide) {
  using namespace fp8t::gemm;
  const int64_t bn = wide ? kBNw : kBN;
  return ((d.M + kBM - 1) / kBM) * ((d.N + bn - 1) / bn);
}

int64_t sumsq_slots(const fp8t_gemm_desc* gemms, int32_t n, const int32_t* sumsq_of) {
  const bool wide = use_wide(gemms, n);
  const int64_t per_tile = wide ? fp8t::gemm::kSumsqPerTileW : fp8t::gemm::kSumsqPerTile;
  int64_t slots = 0;
  for (int32_t i = 0; i < n; ++i)
    if (sumsq_of[i]) slots += gemm_tiles(gemms[i], wide) * per_tile;
  return slots;
}

fp8t_status gemm_multi(const fp8t_gemm_desc* gemms, int32_t n_gemms, const int32_t* sumsq_of,
                       double* d_sumsq_out, void* d_workspace, size_t workspace_bytes,
                       void* stream) {
  t_last_error.clear();
  if (!gemms || n_gemms < 1 || n_gemms > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm: gemms NULL or n_gemms out of range");
  const int64_t lim = int64_t(1) << 31;
  for (int32_t i = 0; i < n_gemms; ++i) {
    const fp8t_gemm_desc& d = gemms[i];
    if (!d.A || !d.B || !d.D_bf16 || !d.d_a_scale_inv || !d.d_b_scale_inv)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm: problem %d: NULL pointer", i);
    if ((d.a_fmt != FP8T_E4M3 && d.a_fmt != FP8T_E5M2) || (d.b_fmt != FP8T_E4M3 && d.b_fmt != FP8T_E5M2))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm: problem %d: unknown format", i);
    if ((d.a_layout != FP8T_K_MAJOR && d.a_layout != FP8T_MN_MAJOR) ||
        (d.b_layout != FP8T_K_MAJOR && d.b_layout != FP8T_MN_MAJOR))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm: problem %d: unknown operand layout", i);
    if (d.M <= 0 || d.N <= 0 || d.K <= 0)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm: problem %d: M, N, K must be > 0", i);
    if (d.M % 16 || d.N % 16 || d.K % 16 || d.M >= lim || d.N >= lim || d.K >= lim)
      return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp8_gemm: problem %d: M, N, K must be multiples of 16 below 2^31", i);
    if (!aligned(d.A, 16) || !aligned(d.B, 16) || !aligned(d.D_bf16, 16) ||
        !aligned(d.d_a_scale_inv, 4) || !aligned(d.d_b_scale_inv, 4))
      return fail(FP8T_ERR_MISALIGNED, "fp8_gemm: problem %d: misaligned pointer", i);
  }
  int64_t n_slots = 0;
  if (sumsq_of) {
    if (!d_sumsq_out || !aligned(d_sumsq_out, 8) || !d_workspace || !aligned(d_workspace, 256))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm_multi_sumsq: NULL or misaligned sumsq_out or workspace");
    n_slots = sumsq_slots(gemms, n_gemms, sumsq_of);
    if (n_slots < 1 || n_slots >= (int64_t(1) << 31))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm_multi_sumsq: no problem (or too many tiles) selected");
    const size_t need = kSumsqHeader + static_cast<size_t>(n_slots) * 8;
    if (workspace_bytes < need)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm_multi_sumsq: workspace of %zu bytes needed", need);
  }
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");

  using namespace fp8t::gemm;
  static thread_local Group group;
  int64_t slot = 0;
  const bool wide = use_wide(gemms, n_gemms);
  const int bn = wide ? kBNw : kBN;
  for (int32_t b0 = 0; b0 < n_gemms; b0 += kMaxProblems) {
    const int32_t b1 = std::min<int32_t>(n_gemms, b0 + kMaxProblems);
    std::memset(&group, 0, sizeof(group));
    group.n = b1 - b0;
    if (sumsq_of) {
      group.ticket = static_cast<unsigned int*>(d_workspace);
      group.abort_word = static_cast<unsigned int*>(d_workspace) + 1;
      group.partials = reinterpret_cast<double*>(static_cast<char*>(d_workspace) + kSumsqHeader);
      group.sumsq_out = d_sumsq_out;
      group.n_partials = static_cast<int32_t>(n_slots);
      group.last_launch = b1 == n_gemms ? 1 : 0;
    }
    int64_t tiles = 0;
    for (int32_t i = b0; i < b1; ++i) {
      const fp8t_gemm_desc& d = gemms[i];
      Problem& P = group.p[i - b0];
      // 128 x 128-byte boxes either way: [rows][K] (K-major) or [K][rows] (MN-major)
      const bool a_mn = d.a_layout == FP8T_MN_MAJOR, b_mn = d.b_layout == FP8T_MN_MAJOR;
      if ((st = a_mn ? encode_kmajor(&P.a, d.A, d.K, d.M, kBK)
                     : encode_kmajor(&P.a, d.A, d.M, d.K, kHalf)) != FP8T_OK) return st;
      if ((st = b_mn ? encode_kmajor(&P.b, d.B, d.K, d.N, kBK)
                     : encode_kmajor(&P.b, d.B, d.N, d.K, kHalf)) != FP8T_OK) return st;
      P.a_mn = a_mn ? 1 : 0;
      P.b_mn = b_mn ? 1 : 0;
      // D (BF16 M x N): 32 x 32 boxes, 64-byte swizzle, written by the epilogue's TMA stores
      cuuint64_t dims[2] = {static_cast<cuuint64_t>(d.N), static_cast<cuuint64_t>(d.M)};
      cuuint64_t strides[1] = {static_cast<cuuint64_t>(d.N) * 2};
      cuuint32_t box[2] = {32, 32};
      cuuint32_t es[2] = {1, 1};
      CUresult r = fn(&P.d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d.D_bf16, dims, strides, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                      CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (D) failed (%d)", (int)r);
      P.sa = d.d_a_scale_inv;
      P.sb = d.d_b_scale_inv;
      P.M = static_cast<int32_t>(d.M);
      P.N = static_cast<int32_t>(d.N);
      P.K = static_cast<int32_t>(d.K);
      P.idesc = make_idesc(d.a_fmt, d.b_fmt, P.a_mn, P.b_mn);
      P.tiles_n = static_cast<int32_t>((d.N + bn - 1) / bn);
      P.tile_start = static_cast<int32_t>(tiles);
      P.sumsq_slot = -1;
      if (sumsq_of && sumsq_of[i]) {
        P.sumsq_slot = static_cast<int32_t>(slot);
        slot += gemm_tiles(d, wide) * (wide ? kSumsqPerTileW : kSumsqPerTile);
      }
      tiles += ((d.M + kBM - 1) / kBM) * P.tiles_n;            // one tile per pair
      if (tiles >= (int64_t(1) << 30))
        return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp8_gemm: too many tiles in one launch");
    }
    group.total_tiles = static_cast<int32_t>(tiles);
    // persistent pairs: wide tiles may be split in two, so a wide launch may use up to twice as
    // many clusters as it has tiles
    const int64_t grid = wide ? 2 * std::min<int64_t>(2 * tiles, dev->gemm_wide_clusters)
                              : 2 * std::min<int64_t>(tiles, dev->gemm_clusters);
    build_schedule(group, static_cast<int>(grid / 2), wide);   // round-robin: extra pairs idle
    if (wide)
      k_fp8_gemm_wide<<<static_cast<unsigned>(grid), kThreadsW, kSmemBytesW, as_stream(stream)>>>(group);
    else
      k_fp8_gemm<false><<<static_cast<unsigned>(grid), kThreads, kSmemBytes, as_stream(stream)>>>(group);
    if ((st = after_launch("fp8_gemm launch")) != FP8T_OK) return st;
  }
  return FP8T_OK;
}

}  // namespace

extern "C" {

fp8t_status fp8_gemm_multi(const fp8t_gemm_desc* gemms, int32_t n_gemms, void* stream) {
  return gemm_multi(gemms, n_gemms, nullptr, nullptr, nullptr, 0, stream);
}

size_t fp8_gemm_sumsq_workspace_bytes(const fp8t_gemm_desc* gemms, int32_t n_gemms,
                                      const int32_t* sumsq_of) {
  if (!gemms || !sumsq_of || n_gemms < 1 || n_gemms > 4096) return 0;
  for (int32_t i = 0; i < n_gemms; ++i)
    if (gemms[i].M <= 0 || gemms[i].N <= 0) return 0;
  const int64_t slots = sumsq_slots(gemms, n_gemms, sumsq_of);
  if (slots < 1) return 0;
  return kSumsqHeader + static_cast<size_t>(slots) * 8;
}

fp8t_status fp8_gemm_multi_sumsq(const fp8t_gemm_desc* gemms, int32_t n_gemms,
                                 const int32_t* sumsq_of, double* d_sumsq_out, void* d_workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!sumsq_of) {
    t_last_error.clear();
    return fail(FP8T_ERR_INVALID_ARG, "fp8_gemm_multi_sumsq: sumsq_of NULL");
  }
  return gemm_multi(gemms, n_gemms, sumsq_of, d_sumsq_out, d_workspace, workspace_bytes, stream);
}

// ------------------------------------------------------------------ MXFP8
fp8t_status fp8_mx_cast_multi(const fp8t_mx_cast_tensor* tensors, int32_t n_tensors, void* stream) {
  t_last_error.clear();
  if (!tensors || n_tensors < 1 || n_tensors > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_cast: tensors NULL or n_tensors out of range");
  for (int32_t i = 0; i < n_tensors; ++i) {
    const fp8t_mx_cast_tensor& t = tensors[i];
    if (!t.x_bf16 || (!t.q_row && !t.q_col) || (t.q_row && !t.scales_row) || (t.q_col && !t.scales_col))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_cast: tensor %d: NULL input, or an output without its scales", i);
    if (t.fmt != FP8T_E4M3 && t.fmt != FP8T_E5M2)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_cast: tensor %d: unknown format", i);
    if (t.rows <= 0 || t.cols <= 0 || t.rows % 128 || t.cols % 128 || t.rows >= (int64_t(1) << 31) ||
        t.cols >= (int64_t(1) << 31))
      return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp8_mx_cast: tensor %d: rows and cols must be positive multiples of 128", i);
    if (!aligned(t.x_bf16, 16) || !aligned(t.q_row, 16) || !aligned(t.q_col, 16) ||
        !aligned(t.scales_row, 16) || !aligned(t.scales_col, 16))
      return fail(FP8T_ERR_MISALIGNED, "fp8_mx_cast: tensor %d: pointers must be 16-byte aligned", i);
  }
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  using namespace fp8t::mx;
  static thread_local Group group;
  for (int32_t b0 = 0; b0 < n_tensors; b0 += kMaxTensors) {
    const int32_t b1 = std::min<int32_t>(n_tensors, b0 + kMaxTensors);
    std::memset(&group, 0, sizeof(group));
    group.n = b1 - b0;
    int64_t tiles = 0;
    for (int32_t i = b0; i < b1; ++i) {
      const fp8t_mx_cast_tensor& t = tensors[i];
      Tensor& T = group.t[i - b0];
      // BF16 [rows][cols] read as 128-row x 64-column boxes (128 bytes per row: 128-byte swizzle)
      cuuint64_t dims[2] = {static_cast<cuuint64_t>(t.cols), static_cast<cuuint64_t>(t.rows)};
      cuuint64_t strides[1] = {static_cast<cuuint64_t>(t.cols) * 2};
      cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kTile)};
      cuuint32_t es[2] = {1, 1};
      CUresult r = fn(&T.x_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(t.x_bf16),
                      dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (MX cast input) failed (%d)", (int)r);
      T.q_row = static_cast<uint8_t*>(t.q_row);
      T.sf_row = static_cast<uint8_t*>(t.scales_row);
      T.q_col = static_cast<uint8_t*>(t.q_col);
      T.sf_col = static_cast<uint8_t*>(t.scales_col);
      T.rows = t.rows;
      T.cols = t.cols;
      T.tiles_c = t.cols / kTile;
      T.tile_start = tiles;
      T.fmt = t.fmt;
      tiles += (t.rows / kTile) * T.tiles_c;
    }
    group.total_tiles = tiles;
    const int64_t grid = std::min<int64_t>(tiles, static_cast<int64_t>(dev->sms) * dev->mx_cast_blocks_per_sm);
    k_mx_cast<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, as_stream(stream)>>>(group);
    if ((st = after_launch("fp8_mx_cast launch")) != FP8T_OK) return st;
  }
  return FP8T_OK;
}

}  // extern "C"

namespace {

// MX launches use 256 x 384 tiles when every output is at least 512 wide (for the whole call).
bool mx_use_wide(const fp8t_mx_gemm_desc* gemms, int32_t n) {
  for (int32_t i = 0; i < n; ++i)
    if (gemms[i].N < 512) return false;
  return true;
}

int64_t mx_sumsq_slots(const fp8t_mx_gemm_desc* gemms, int32_t n, const int32_t* sumsq_of) {
  using namespace fp8t::gemm;
  const bool wide = mx_use_wide(gemms, n);
  const int64_t bn = wide ? kBNx : kBN, per_tile = wide ? kSumsqPerTileW : kSumsqPerTile;
  int64_t slots = 0;
  for (int32_t i = 0; i < n; ++i)
    if (sumsq_of[i]) slots += ((gemms[i].M + kBM - 1) / kBM) * ((gemms[i].N + bn - 1) / bn) * per_tile;
  return slots;
}

fp8t_status mx_gemm_multi(const fp8t_mx_gemm_desc* gemms, int32_t n_gemms, const int32_t* sumsq_of,
                          double* d_sumsq_out, void* d_workspace, size_t workspace_bytes,
                          void* stream) {
  t_last_error.clear();
  if (!gemms || n_gemms < 1 || n_gemms > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_gemm: gemms NULL or n_gemms out of range");
  const int64_t lim = int64_t(1) << 31;
  for (int32_t i = 0; i < n_gemms; ++i) {
    const fp8t_mx_gemm_desc& d = gemms[i];
    if (!d.A || !d.B || !d.A_scales || !d.B_scales || !d.D_bf16)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_gemm: problem %d: NULL pointer", i);
    if ((d.a_fmt != FP8T_E4M3 && d.a_fmt != FP8T_E5M2) || (d.b_fmt != FP8T_E4M3 && d.b_fmt != FP8T_E5M2) ||
        (d.a_layout != FP8T_K_MAJOR && d.a_layout != FP8T_MN_MAJOR) ||
        (d.b_layout != FP8T_K_MAJOR && d.b_layout != FP8T_MN_MAJOR))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_gemm: problem %d: unknown format or layout", i);
    if (d.M <= 0 || d.N <= 0 || d.K <= 0 || d.M % 128 || d.N % 128 || d.K % 128 || d.M >= lim ||
        d.N >= lim || d.K >= lim)
      return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp8_mx_gemm: problem %d: M, N, K must be positive multiples of 128", i);
    if (!aligned(d.A, 16) || !aligned(d.B, 16) || !aligned(d.D_bf16, 16) || !aligned(d.A_scales, 16) ||
        !aligned(d.B_scales, 16))
      return fail(FP8T_ERR_MISALIGNED, "fp8_mx_gemm: problem %d: pointers must be 16-byte aligned", i);
  }
  int64_t n_slots = 0;
  if (sumsq_of) {
    if (!d_sumsq_out || !aligned(d_sumsq_out, 8) || !d_workspace || !aligned(d_workspace, 256))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_gemm_multi_sumsq: NULL or misaligned sumsq_out or workspace");
    n_slots = mx_sumsq_slots(gemms, n_gemms, sumsq_of);
    if (n_slots < 1 || n_slots >= (int64_t(1) << 31))
      return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_gemm_multi_sumsq: no problem (or too many tiles) selected");
    const size_t need = kSumsqHeader + static_cast<size_t>(n_slots) * 8;
    if (workspace_bytes < need)
      return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_gemm_multi_sumsq: workspace of %zu bytes needed", need);
  }
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  using namespace fp8t::gemm;
  // 256 x 384 tiles when every output is at least 512 wide (the choice holds for the whole call)
  const bool mxw = mx_use_wide(gemms, n_gemms);
  int64_t slot = 0;
  // scale atoms viewed as [atoms][512] bytes, read one atom at a time
  auto encode_sf = [&](CUtensorMap* map, const void* ptr, int64_t atoms) -> fp8t_status {
    cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(atoms)};
    cuuint64_t strides[1] = {512};
    cuuint32_t box[2] = {128, 1};
    cuuint32_t es[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(ptr), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (scales) failed (%d)", (int)r);
    return FP8T_OK;
  };
  static thread_local Group group;
  for (int32_t b0 = 0; b0 < n_gemms; b0 += kMaxProblems) {
    const int32_t b1 = std::min<int32_t>(n_gemms, b0 + kMaxProblems);
    std::memset(&group, 0, sizeof(group));
    group.n = b1 - b0;
    if (sumsq_of) {
      group.ticket = static_cast<unsigned int*>(d_workspace);
      group.abort_word = static_cast<unsigned int*>(d_workspace) + 1;
      group.partials = reinterpret_cast<double*>(static_cast<char*>(d_workspace) + kSumsqHeader);
      group.sumsq_out = d_sumsq_out;
      group.n_partials = static_cast<int32_t>(n_slots);
      group.last_launch = b1 == n_gemms ? 1 : 0;
    }
    int64_t tiles = 0;
    for (int32_t i = b0; i < b1; ++i) {
      const fp8t_mx_gemm_desc& d = gemms[i];
      Problem& P = group.p[i - b0];
      const bool a_mn = d.a_layout == FP8T_MN_MAJOR, b_mn = d.b_layout == FP8T_MN_MAJOR;
      if ((st = a_mn ? encode_kmajor(&P.a, d.A, d.K, d.M, kBK)
                     : encode_kmajor(&P.a, d.A, d.M, d.K, kHalf)) != FP8T_OK) return st;
      if ((st = b_mn ? encode_kmajor(&P.b, d.B, d.K, d.N, kBK)
                     : encode_kmajor(&P.b, d.B, d.N, d.K, kHalf)) != FP8T_OK) return st;
      if ((st = encode_sf(&P.sfa, d.A_scales, (d.M / 128) * (d.K / 128))) != FP8T_OK) return st;
      if ((st = encode_sf(&P.sfb, d.B_scales, (d.N / 128) * (d.K / 128))) != FP8T_OK) return st;
      cuuint64_t dims[2] = {static_cast<cuuint64_t>(d.N), static_cast<cuuint64_t>(d.M)};
      cuuint64_t strides[1] = {static_cast<cuuint64_t>(d.N) * 2};
      cuuint32_t box[2] = {32, 32};
      cuuint32_t es[2] = {1, 1};
      CUresult r = fn(&P.d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d.D_bf16, dims, strides, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                      CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (D) failed (%d)", (int)r);
      P.sa = nullptr;                          // block scales only: alpha = 1
      P.sb = nullptr;
      P.M = static_cast<int32_t>(d.M);
      P.N = static_cast<int32_t>(d.N);
      P.K = static_cast<int32_t>(d.K);
      P.a_mn = a_mn ? 1 : 0;
      P.b_mn = b_mn ? 1 : 0;
      P.a_fmt = d.a_fmt;
      P.b_fmt = d.b_fmt;
      P.kb128 = static_cast<int32_t>(d.K / 128);
      P.sumsq_slot = -1;
      if (mxw && (st = b_mn ? encode_mn64(&P.b64, d.B, d.K, d.N)
                            : encode_kmajor(&P.b64, d.B, d.N, d.K, kHalf / 2)) != FP8T_OK) return st;
      P.tiles_n = static_cast<int32_t>((d.N + (mxw ? kBNx : kBN) - 1) / (mxw ? kBNx : kBN));
      P.tile_start = static_cast<int32_t>(tiles);
      const int64_t p_tiles = ((d.M + kBM - 1) / kBM) * P.tiles_n;
      if (sumsq_of && sumsq_of[i]) {
        P.sumsq_slot = static_cast<int32_t>(slot);
        slot += p_tiles * (mxw ? kSumsqPerTileW : kSumsqPerTile);
      }
      tiles += p_tiles;
      if (tiles >= (int64_t(1) << 30))
        return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp8_mx_gemm: too many tiles in one launch");
    }
    group.total_tiles = static_cast<int32_t>(tiles);
    const int64_t grid = 2 * std::min<int64_t>(tiles, mxw ? dev->gemm_mxw_clusters : dev->gemm_mx_clusters);
    build_schedule(group, static_cast<int>(grid / 2), false, mxw);
    if (mxw)
      k_fp8_gemm_mx_wide<<<static_cast<unsigned>(grid), kThreadsX, kSmemBytesX, as_stream(stream)>>>(group);
    else
      k_fp8_gemm<true><<<static_cast<unsigned>(grid), kThreads, kSmemBytesMX, as_stream(stream)>>>(group);
    if ((st = after_launch("fp8_mx_gemm launch")) != FP8T_OK) return st;
  }
  return FP8T_OK;
}

}  // namespace

extern "C" {

fp8t_status fp8_mx_gemm_multi(const fp8t_mx_gemm_desc* gemms, int32_t n_gemms, void* stream) {
  return mx_gemm_multi(gemms, n_gemms, nullptr, nullptr, nullptr, 0, stream);
}

size_t fp8_mx_gemm_sumsq_workspace_bytes(const fp8t_mx_gemm_desc* gemms, int32_t n_gemms,
                                         const int32_t* sumsq_of) {
  if (!gemms || !sumsq_of || n_gemms < 1 || n_gemms > 4096) return 0;
  for (int32_t i = 0; i < n_gemms; ++i)
    if (gemms[i].M <= 0 || gemms[i].N <= 0) return 0;
  const int64_t slots = mx_sumsq_slots(gemms, n_gemms, sumsq_of);
  if (slots < 1) return 0;
  return kSumsqHeader + static_cast<size_t>(slots) * 8;
}

fp8t_status fp8_mx_gemm_multi_sumsq(const fp8t_mx_gemm_desc* gemms, int32_t n_gemms,
                                    const int32_t* sumsq_of, double* d_sumsq_out,
                                    void* d_workspace, size_t workspace_bytes, void* stream) {
  if (!sumsq_of) {
    t_last_error.clear();
    return fail(FP8T_ERR_INVALID_ARG, "fp8_mx_gemm_multi_sumsq: sumsq_of NULL");
  }
  return mx_gemm_multi(gemms, n_gemms, sumsq_of, d_sumsq_out, d_workspace, workspace_bytes, stream);
}

fp8t_status fp8_gemm(const void* A, fp8t_format a_fmt, const void* B, fp8t_format b_fmt, int64_t M,
                     int64_t N, int64_t K, const float* d_a_scale_inv, const float* d_b_scale_inv,
                     void* D_bf16, void* stream) {
  const fp8t_gemm_desc d = {A, a_fmt, B, b_fmt, M, N, K, d_a_scale_inv, d_b_scale_inv, D_bf16};
  return fp8_gemm_multi(&d, 1, stream);
}

// ------------------------------------------------------------------ 4-bit cast
size_t fp4_scale_bytes(int64_t mn, int64_t k, fp8t_quant quant) {
  if (mn <= 0 || k <= 0 || mn >= (int64_t(1) << 31) || k >= (int64_t(1) << 31) ||
      (quant != FP8T_Q_MXFP4 && quant != FP8T_Q_NVFP4))
    return 0;
  return static_cast<size_t>((mn + 127) / 128 * fp8t::blk::atoms_per_row(k, quant) * 512);
}

fp8t_status fp4_cast_multi(const fp8t_fp4_cast_tensor* tensors, int32_t n_tensors, void* stream) {
  t_last_error.clear();
  if (!tensors || n_tensors < 1 || n_tensors > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "fp4_cast: tensors NULL or n_tensors out of range");
  const int64_t lim = int64_t(1) << 31;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const fp8t_fp4_cast_tensor& t = tensors[i];
    if (!t.x_bf16 || (!t.q_row && !t.q_col) || (t.q_row && !t.scales_row) || (t.q_col && !t.scales_col))
      return fail(FP8T_ERR_INVALID_ARG, "fp4_cast: tensor %d: NULL input, or an output without its scales", i);
    if (t.quant != FP8T_Q_MXFP4 && t.quant != FP8T_Q_NVFP4)
      return fail(FP8T_ERR_INVALID_ARG, "fp4_cast: tensor %d: quant must be MXFP4 or NVFP4", i);
    if (t.quant == FP8T_Q_NVFP4 ? !t.d_scale : (t.d_scale || t.d_amax_inout || t.d_scale_inv_out))
      return fail(FP8T_ERR_INVALID_ARG, "fp4_cast: tensor %d: NVFP4 needs a scale; MXFP4 has no scale, amax or scale inverse", i);
    if (t.rows <= 0 || t.cols <= 0)
      return fail(FP8T_ERR_INVALID_ARG, "fp4_cast: tensor %d: rows and cols must be > 0", i);
    if (t.cols % 32 || (t.q_col && t.rows % 32) || t.rows >= lim || t.cols >= lim ||
        t.rows * t.cols >= (int64_t(1) << 40))
      return fail(FP8T_ERR_UNSUPPORTED_SHAPE,
                  "fp4_cast: tensor %d: cols (and rows with a column-wise copy) must be multiples of 32, rows*cols < 2^40", i);
    if (!aligned(t.x_bf16, 16) || !aligned(t.q_row, 16) || !aligned(t.q_col, 16) ||
        !aligned(t.scales_row, 16) || !aligned(t.scales_col, 16) || !aligned(t.d_scale, 4) ||
        !aligned(t.d_amax_inout, 4) || !aligned(t.d_scale_inv_out, 4))
      return fail(FP8T_ERR_MISALIGNED, "fp4_cast: tensor %d: misaligned pointer", i);
  }
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK || (st = ready_fp4_cast(dev)) != FP8T_OK) return st;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  using namespace fp8t::fp4;
  static thread_local CastGroup group;
  for (int32_t b0 = 0; b0 < n_tensors; b0 += kCastTensors) {
    const int32_t b1 = std::min<int32_t>(n_tensors, b0 + kCastTensors);
    std::memset(&group, 0, sizeof(group));
    group.n = b1 - b0;
    int64_t tiles = 0;
    bool any_col = false;
    for (int32_t i = b0; i < b1; ++i) any_col |= tensors[i].q_col != nullptr;
    for (int32_t i = b0; i < b1; ++i) {
      const fp8t_fp4_cast_tensor& t = tensors[i];
      CastTensor& T = group.t[i - b0];
      cuuint64_t dims[2] = {static_cast<cuuint64_t>(t.cols), static_cast<cuuint64_t>(t.rows)};
      cuuint64_t strides[1] = {static_cast<cuuint64_t>(t.cols) * 2};
      cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kTile)};
      cuuint32_t es[2] = {1, 1};
      CUresult r = fn(&T.x_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(t.x_bf16),
                      dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
      if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (4-bit cast input) failed (%d)", (int)r);
      if (t.q_col) {
        cuuint64_t qdims[2] = {static_cast<cuuint64_t>(t.rows / 2), static_cast<cuuint64_t>(t.cols)};
        cuuint64_t qstrides[1] = {static_cast<cuuint64_t>(t.rows / 2)};
        cuuint32_t qbox[2] = {static_cast<cuuint32_t>(kTile / 2), static_cast<cuuint32_t>(kTile)};
        r = fn(&T.qc_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, t.q_col, qdims, qstrides, qbox, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (4-bit column codes) failed (%d)", (int)r);
      }
      T.x = t.x_bf16;
      T.q_row = static_cast<uint8_t*>(t.q_row);
      T.sf_row = static_cast<uint8_t*>(t.scales_row);
      T.q_col = static_cast<uint8_t*>(t.q_col);
      T.sf_col = static_cast<uint8_t*>(t.scales_col);
      T.scale = t.d_scale;
      T.amax_bits = reinterpret_cast<unsigned int*>(t.d_amax_inout);
      T.scale_inv = t.d_scale_inv_out;
      T.rows = static_cast<int32_t>(t.rows);
      T.cols = static_cast<int32_t>(t.cols);
      T.tiles_c = static_cast<int32_t>((t.cols + kTile - 1) / kTile);
      T.tile_start = static_cast<int32_t>(tiles);
      T.kind = t.quant;
      tiles += ((t.rows + kTile - 1) / kTile) * T.tiles_c;
    }
    if (tiles >= (int64_t(1) << 30)) return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp4_cast: too many tiles in one launch");
    group.total_tiles = static_cast<int32_t>(tiles);
    // row-wise copies only: the streaming kernel (tiles: 8192 x 4096 16.2 for 14.6 us MXFP4, 18.8 for 16.1 NVFP4)
    if (!any_col) {
      // blocks of 32 values of the largest tensor, or the words that fill up its last atoms (one row of 4096 on
      // the CTAs of its blocks alone: 4.2 and 6.9 us, on those of the words 2.1 and 2.6)
      int64_t most = 0;
      for (int32_t i = b0; i < b1; ++i) {
        const fp8t_fp4_cast_tensor& t = tensors[i];
        const int64_t words = ((t.rows + 127) / 128 * 128 - t.rows) * fp8t::blk::atoms_per_row(t.cols, t.quant);
        most = std::max({most, t.rows * t.cols / 32, words});
      }
      const int64_t rgrid = std::min<int64_t>((most + kCastThreads - 1) / kCastThreads,
                                              static_cast<int64_t>(dev->sms) * dev->fp4_cast_rows_blocks_per_sm);
      (void)launch_pdl(k_fp4_cast_rows, rgrid, kCastThreads, 0, as_stream(stream), 0, group);
      if ((st = after_launch("fp4_cast launch")) != FP8T_OK) return st;
      continue;
    }
    const int64_t grid = std::min<int64_t>(tiles, static_cast<int64_t>(dev->sms) * dev->fp4_cast_blocks_per_sm);
    (void)launch_pdl(k_fp4_cast, grid, kCastThreads, kCastSmemBytes, as_stream(stream), 0, group);
    if ((st = after_launch("fp4_cast launch")) != FP8T_OK) return st;
  }
  return FP8T_OK;
}

// ------------------------------------------------------------------ 4-bit GEMM
}  // extern "C"

namespace {

// Scales of a 4-bit operand: rows of 256 words (1 KB), one (MXFP4) or two (NVFP4) per 128 rows and 256
// values of K, read as one box.
fp8t_status encode_fp4_scales(CUtensorMap* map, const void* ptr, int64_t mn, int64_t K, bool nv) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint32_t per = nv ? 2 : 1;
  cuuint64_t dims[2] = {256, static_cast<cuuint64_t>((mn + 127) / 128 * ((K + 255) / 256) * per)};
  cuuint64_t strides[1] = {1024};
  cuuint32_t box[2] = {256, per};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(ptr), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (4-bit scales) failed (%d)", (int)r);
  return FP8T_OK;
}

// Fills a group's problems (tiles of 256 x tile_n) and returns the number of tiles, or -1 with *st set.
template <class G>
int64_t fill_fp4_group(G& g, const fp8t_fp4_gemm_desc* gemms, int32_t n, int tile_n, fp8t_status* st) {
  using namespace fp8t::gemm;
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    *st = fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    return -1;
  }
  const bool nv = gemms[0].quant == FP8T_Q_NVFP4;
  g.n = n;
  int64_t tiles = 0;
  for (int32_t i = 0; i < n; ++i) {
    const fp8t_fp4_gemm_desc& d = gemms[i];
    Problem4& P = g.p[i];
    if ((*st = encode_kmajor(&P.a, d.A, d.M, d.K / 2, kHalf)) != FP8T_OK ||
        (*st = encode_kmajor(&P.b, d.B, d.N, d.K / 2, kHalf)) != FP8T_OK ||
        (tile_n > kBN && (*st = encode_kmajor(&P.b64, d.B, d.N, d.K / 2, kHalf / 2)) != FP8T_OK) ||
        (*st = encode_fp4_scales(&P.sfa, d.A_scales, d.M, d.K, nv)) != FP8T_OK ||
        (*st = encode_fp4_scales(&P.sfb, d.B_scales, d.N, d.K, nv)) != FP8T_OK)
      return -1;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(d.N), static_cast<cuuint64_t>(d.M)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(d.N) * 2};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t es[2] = {1, 1};
    CUresult r = fn(&P.d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d.D_bf16, dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
      *st = fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled (D) failed (%d)", (int)r);
      return -1;
    }
    P.sa = d.d_a_scale_inv;
    P.sb = d.d_b_scale_inv;
    P.M = static_cast<int32_t>(d.M);
    P.N = static_cast<int32_t>(d.N);
    P.num_kb = static_cast<int32_t>((d.K + 255) / 256);
    P.tiles_n = static_cast<int32_t>((d.N + tile_n - 1) / tile_n);
    P.tile_start = static_cast<int32_t>(tiles);
    tiles += ((d.M + kBM - 1) / kBM) * P.tiles_n;
  }
  g.total_tiles = static_cast<int32_t>(tiles);
  return tiles;
}

// Tiles to clusters, longest (most k-blocks) first, each to the least loaded cluster; every cluster then runs
// its tiles in index order.
void list_fp4_tiles(fp8t::gemm::ListGroup4& g, int clusters) {
  std::vector<std::pair<int, int>> tiles;              // (k-blocks, tile)
  tiles.reserve(g.total_tiles);
  for (int p = 0; p < g.n; ++p) {
    const int end = p + 1 < g.n ? g.p[p + 1].tile_start : g.total_tiles;
    for (int t = g.p[p].tile_start; t < end; ++t) tiles.push_back({g.p[p].num_kb, t});
  }
  std::stable_sort(tiles.begin(), tiles.end(),
                   [](const std::pair<int, int>& a, const std::pair<int, int>& b) { return a.first > b.first; });
  std::vector<std::pair<int64_t, int>> load(clusters); // a heap of (k-blocks, cluster), least first
  for (int c = 0; c < clusters; ++c) load[c] = {0, c};
  std::vector<std::vector<uint16_t>> own(clusters);
  const auto more = std::greater<std::pair<int64_t, int>>();
  for (const auto& t : tiles) {
    std::pop_heap(load.begin(), load.end(), more);
    own[load.back().second].push_back(static_cast<uint16_t>(t.second));
    load.back().first += t.first;
    std::push_heap(load.begin(), load.end(), more);
  }
  int k = 0;
  for (int c = 0; c < clusters; ++c) {
    std::sort(own[c].begin(), own[c].end());
    g.start[c] = static_cast<uint16_t>(k);
    for (uint16_t t : own[c]) g.order[k++] = t;
  }
  g.start[clusters] = static_cast<uint16_t>(k);
}

template <bool WIDE, class G>
fp8t_status launch_fp4_tiles(const G& g, bool nv, const DeviceInfo* dev, cudaStream_t stream) {
  using namespace fp8t::gemm;
  const int grid = 2 * std::min(g.total_tiles, dev->gemm_fp4_clusters);
  if (nv)
    (void)launch_pdl(k_fp4_gemm<true, WIDE, G>, grid, kThreads4, kSmemBytes4<true, WIDE>, stream, 0, g);
  else
    (void)launch_pdl(k_fp4_gemm<false, WIDE, G>, grid, kThreads4, kSmemBytes4<false, WIDE>, stream, 0, g);
  return after_launch("fp4_gemm launch");
}

// n problems of one format on pair tiles. 384 columns need 1.36 times the time of 256 (8.1 against 10.8 us per
// tile of K = 4096 NVFP4, 7.6 and 10.7 MXFP4) for 1.5 times the work, so they are taken where they save
// enough rounds: with fewer tiles than clusters, or an N just past a multiple of 384, they do not.
// Tiles of one length (and launches of at most one tile per cluster) are dealt out in turn; problems of
// different K get a list per cluster, where it fits: the three products of 2048 x 1024 x 4096 27.8 -> 22.7 us (NVFP4), of
// 8192 x 4096 x 11008 398 -> 383 (MXFP4; NVFP4 432 and 437, both at the power cap).
template <bool WIDE>
fp8t_status fp4_gemm_tiles_as(const fp8t_fp4_gemm_desc* gemms, int32_t n, int64_t tiles, bool uneven,
                              const DeviceInfo* dev, cudaStream_t stream) {
  using namespace fp8t::gemm;
  constexpr int tile_n = WIDE ? kBN4w : kBN;
  const bool nv = gemms[0].quant == FP8T_Q_NVFP4;
  fp8t_status st = FP8T_OK;
  if (uneven && tiles > dev->gemm_fp4_clusters && tiles <= kMaxSchedTiles && dev->gemm_fp4_clusters <= kMaxClusters) {
    static thread_local ListGroup4 g;
    if (fill_fp4_group(g, gemms, n, tile_n, &st) < 0) return st;
    list_fp4_tiles(g, dev->gemm_fp4_clusters);
    return launch_fp4_tiles<WIDE>(g, nv, dev, stream);
  }
  if (n <= SmallGroup4::kProblems) {
    static thread_local SmallGroup4 g;
    if (fill_fp4_group(g, gemms, n, tile_n, &st) < 0) return st;
    return launch_fp4_tiles<WIDE>(g, nv, dev, stream);
  }
  static thread_local LargeGroup4 g;
  if (fill_fp4_group(g, gemms, n, tile_n, &st) < 0) return st;
  return launch_fp4_tiles<WIDE>(g, nv, dev, stream);
}

fp8t_status fp4_gemm_tiles(const fp8t_fp4_gemm_desc* gemms, int32_t n, const DeviceInfo* dev, cudaStream_t stream) {
  using namespace fp8t::gemm;
  int64_t narrow = 0, wide = 0, narrow_kb = 0, wide_kb = 0;      // tiles, and k-blocks of all of them
  bool uneven = false;
  for (int32_t i = 0; i < n; ++i) {
    const int64_t m = (gemms[i].M + kBM - 1) / kBM, kb = (gemms[i].K + 255) / 256;
    const int64_t tn = m * ((gemms[i].N + kBN - 1) / kBN), tw = m * ((gemms[i].N + kBN4w - 1) / kBN4w);
    narrow += tn;
    wide += tw;
    narrow_kb += tn * kb;
    wide_kb += tw * kb;
    uneven |= kb != (gemms[0].K + 255) / 256;
  }
  if (narrow >= (int64_t(1) << 30)) return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp4_gemm: too many tiles in one launch");
  // rounds of tiles, or with tiles of different length the clusters' even share of k-blocks
  const int64_t c = dev->gemm_fp4_clusters;
  const double tn = uneven ? double(narrow_kb) / c : double((narrow + c - 1) / c);
  const double tw = uneven ? double(wide_kb) / c : double((wide + c - 1) / c);
  return 1.36 * tw < tn && wide > c ? fp4_gemm_tiles_as<true>(gemms, n, wide, uneven, dev, stream)
                                    : fp4_gemm_tiles_as<false>(gemms, n, narrow, uneven, dev, stream);
}

template <bool NV, int BT>
cudaError_t launch_fp4_split(const fp8t::gemm::SplitGroup& g, int64_t tiles, int ways, cudaStream_t stream) {
  return launch_pdl(fp8t::gemm::k_fp4_gemm_split<NV, BT>, tiles * ways, fp8t::gemm::kSplitThreads,
                    fp8t::gemm::SplitShape<NV, BT>::kSmem, stream, ways, g);
}

// Tokens per tile and CTAs per cluster of the split kernel for up to kMaxSplitProblems problems.
struct SplitPlan {
  int bt, ways;
  int64_t tiles;
};
SplitPlan plan_fp4_split(const fp8t_fp4_gemm_desc* gemms, int32_t n, int sms) {
  int64_t M = 0, kbs = 0;
  for (int32_t i = 0; i < n; ++i) {
    M = std::max(M, gemms[i].M);
    kbs = std::max(kbs, (gemms[i].K + 255) / 256);
  }
  SplitPlan p;
  p.bt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  p.tiles = 0;
  for (int32_t i = 0; i < n; ++i) p.tiles += (gemms[i].N + 127) / 128;
  // the fewest k-blocks for the SM that has most (CTAs per SM x k-blocks per CTA), within two CTAs per SM
  int64_t best = 0;
  p.ways = 1;
  for (int w = 1; w <= 8 && w <= kbs && (w == 1 || p.tiles * w <= 2 * sms); ++w) {
    const int64_t most = (p.tiles * w + sms - 1) / sms * ((kbs + w - 1) / w);
    if (w == 1 || most < best) {
      best = most;
      p.ways = w;
    }
  }
  return p;
}

fp8t_status fp4_gemm_split(const fp8t_fp4_gemm_desc* gemms, int32_t n, const SplitPlan& plan, cudaStream_t stream) {
  using namespace fp8t::gemm;
  const bool nv = gemms[0].quant == FP8T_Q_NVFP4;
  static thread_local SplitGroup group;
  group.n = n;
  int64_t tiles = 0;
  fp8t_status st;
  for (int32_t i = 0; i < n; ++i) {
    const fp8t_fp4_gemm_desc& d = gemms[i];
    SplitProblem& P = group.p[i];
    if ((st = encode_kmajor(&P.w, d.B, d.N, d.K / 2, 128)) != FP8T_OK) return st;
    if ((st = encode_kmajor(&P.t, d.A, d.M, d.K / 2, static_cast<uint32_t>(plan.bt))) != FP8T_OK) return st;
    if ((st = encode_fp4_scales(&P.sfw, d.B_scales, d.N, d.K, nv)) != FP8T_OK) return st;
    if ((st = encode_fp4_scales(&P.sft, d.A_scales, d.M, d.K, nv)) != FP8T_OK) return st;
    P.sa = d.d_a_scale_inv;
    P.sb = d.d_b_scale_inv;
    P.D = static_cast<uint16_t*>(d.D_bf16);
    P.M = static_cast<int32_t>(d.M);
    P.N = static_cast<int32_t>(d.N);
    P.num_kb = static_cast<int32_t>((d.K + 255) / 256);
    P.tile_start = static_cast<int32_t>(tiles);
    tiles += (d.N + 127) / 128;
  }
  cudaError_t e = cudaErrorInvalidValue;
  switch (plan.bt) {
    case 16: e = nv ? launch_fp4_split<true, 16>(group, tiles, plan.ways, stream) : launch_fp4_split<false, 16>(group, tiles, plan.ways, stream); break;
    case 32: e = nv ? launch_fp4_split<true, 32>(group, tiles, plan.ways, stream) : launch_fp4_split<false, 32>(group, tiles, plan.ways, stream); break;
    case 64: e = nv ? launch_fp4_split<true, 64>(group, tiles, plan.ways, stream) : launch_fp4_split<false, 64>(group, tiles, plan.ways, stream); break;
    case 128: e = nv ? launch_fp4_split<true, 128>(group, tiles, plan.ways, stream) : launch_fp4_split<false, 128>(group, tiles, plan.ways, stream); break;
  }
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(FP8T_ERR_CUDA, "fp4_gemm split launch: %s", cudaGetErrorString(e));
  }
  return after_launch("fp4_gemm split launch");
}

}  // namespace

extern "C" {

fp8t_status fp4_gemm_multi(const fp8t_fp4_gemm_desc* gemms, int32_t n_gemms, void* stream) {
  t_last_error.clear();
  if (!gemms || n_gemms < 1 || n_gemms > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "fp4_gemm: gemms NULL or n_gemms out of range");
  const int64_t lim = int64_t(1) << 31;
  for (int32_t i = 0; i < n_gemms; ++i) {
    const fp8t_fp4_gemm_desc& d = gemms[i];
    if (!d.A || !d.B || !d.A_scales || !d.B_scales || !d.D_bf16)
      return fail(FP8T_ERR_INVALID_ARG, "fp4_gemm: problem %d: NULL pointer", i);
    if (d.quant != FP8T_Q_MXFP4 && d.quant != FP8T_Q_NVFP4)
      return fail(FP8T_ERR_INVALID_ARG, "fp4_gemm: problem %d: quant must be MXFP4 or NVFP4", i);
    if (d.M <= 0 || d.N <= 0 || d.K <= 0)
      return fail(FP8T_ERR_INVALID_ARG, "fp4_gemm: problem %d: M, N, K must be > 0", i);
    if (d.N % 8 || d.K % 32 || d.M >= lim || d.N >= lim || d.K >= lim ||
        (std::max(d.M, d.N) + 511) / 128 * ((d.K + 255) / 256) >= (int64_t(1) << 30))
      return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp4_gemm: problem %d: N must be a multiple of 8 and K of 32", i);
    if (!aligned(d.A, 16) || !aligned(d.B, 16) || !aligned(d.D_bf16, 16) || !aligned(d.A_scales, 16) ||
        !aligned(d.B_scales, 16) || !aligned(d.d_a_scale_inv, 4) || !aligned(d.d_b_scale_inv, 4))
      return fail(FP8T_ERR_MISALIGNED, "fp4_gemm: problem %d: misaligned pointer", i);
  }
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK || (st = ready_fp4_gemm(dev)) != FP8T_OK) return st;
  // consecutive problems of one format and size class share a launch: at most 128 rows (the split kernel) or more
  // (pair tiles). Split / tiles, NVFP4: 1 x 4096 x 4096 4.7 / 10.4 us, 128 x 4096 x 4096 7.3 / 11.2, 128 x 11008 x 4096
  // 10.6 / 12.0, 128 x 4096 x 256 4.8 / 6.4. With several tiles of tokens the split kernel took 7.2 to 33 us over 19
  // sizes of 200 to 8000 rows, pair tiles 5.7 to 12.5 (it won at 300 x 1024 x 4096 only)
  for (int32_t b0 = 0, b1 = 0; b0 < n_gemms; b0 = b1) {
    const bool few = gemms[b0].M <= fp8t::gemm::kMaxSplitRows;
    const int most = few ? fp8t::gemm::kMaxSplitProblems : fp8t::gemm::kMaxProblems;
    for (b1 = b0; b1 < n_gemms && b1 - b0 < most && gemms[b1].quant == gemms[b0].quant &&
                  (gemms[b1].M <= fp8t::gemm::kMaxSplitRows) == few; ++b1) {
    }
    st = few ? fp4_gemm_split(gemms + b0, b1 - b0, plan_fp4_split(gemms + b0, b1 - b0, dev->sms), as_stream(stream))
             : fp4_gemm_tiles(gemms + b0, b1 - b0, dev, as_stream(stream));
    if (st != FP8T_OK) return st;
  }
  return FP8T_OK;
}

// ------------------------------------------------------------------ RMSNorm
}  // extern "C"

namespace {

// Threads and vectors per thread of a forward launch. Rows of up to 1024 columns take a warp each, four to a
// CTA (16384 x 1024 to FP8: 21.9 us either way; 1000 x 1024: 3.4 us, on a CTA each 3.6). Wider rows take a CTA: with
// rows enough to fill the GPU two vectors per thread, so that fewer threads are summed over (one / two: 1000 x 4096
// 8.1 / 6.3 us, 8192 x 4096 45.2 / 40.8), else the fewest that 512 threads hold (1 x 2048 2.3 / 2.4, to NVFP4 2.6 / 2.9).
struct NormShape {
  bool warp_row;
  int vpt, threads;
};
NormShape norm_shape(int64_t rows, int64_t cols) {
  using namespace fp8t::norm;
  const int nvec = static_cast<int>(cols / 8);
  NormShape s;
  s.warp_row = cols <= kMaxWarpCols;
  if (s.warp_row) {
    s.vpt = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
    s.threads = 32 * kRowsPerCta;
    return s;
  }
  const int fewest = nvec <= kMaxThreads ? 1 : nvec <= 2 * kMaxThreads ? 2 : 4;
  s.vpt = rows <= 148 ? fewest : std::max(2, fewest);
  s.threads = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  return s;
}

// Backward: vectors per thread, threads per row group, groups per CTA, CTAs (at most one per SM, fewer when
// there are fewer rows; groups only as far as rows fill them).
struct NormBwdShape {
  int vpt, group, groups;
  int64_t ctas;
};
NormBwdShape norm_backward_shape(int64_t rows, int64_t cols) {
  using namespace fp8t::norm;
  const int nvec = static_cast<int>(cols / 8);
  NormBwdShape s;
  // the fewest vectors that 512 threads hold, but two where that leaves a row group a warp or more. 8192 rows, one /
  // two / three vectors: 2048 columns 33 / 27 us, 2816 - / 38 / 46, 5120 - / 73 / 80
  s.vpt = nvec <= 32 ? 1 : nvec <= 2 * kBwdThreads ? 2 : nvec <= 3 * kBwdThreads ? 3 : 4;
  s.group = ((nvec + s.vpt - 1) / s.vpt + 31) / 32 * 32;
  const int most = std::min(kBwdThreads / s.group, s.group == 32 ? 16 : 15);      // barrier ids 1..15
  s.groups = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, (rows + kBwdCtas - 1) / kBwdCtas)));
  s.ctas = std::min<int64_t>(kBwdCtas, (rows + s.groups - 1) / s.groups);
  return s;
}

bool norm_cols_ok(int64_t rows, int64_t cols, int64_t multiple) {
  return cols % multiple == 0 && cols <= fp8t::norm::kMaxCols && rows < (int64_t(1) << 31);
}

// Persistent grid: as many CTAs as are resident at once (looked up once per kernel and size).
template <int VPT, bool WARP_ROW, int Q>
void launch_norm_as(const fp8t::norm::Fwd& p, int threads, int sms, cudaStream_t stream) {
  using namespace fp8t::norm;
  static std::atomic<int> resident[kMaxThreads / 32 + 1];
  int n = resident[threads / 32].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_rmsnorm_cast<VPT, WARP_ROW, Q>, threads, 0) != cudaSuccess ||
        n < 1) {
      (void)cudaGetLastError();
      n = 1;
    }
    resident[threads / 32].store(n, std::memory_order_relaxed);
  }
  const int64_t per_cta = WARP_ROW ? kRowsPerCta : 1;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((p.rows + per_cta - 1) / per_cta, static_cast<int64_t>(sms) * n));
  (void)launch_pdl(k_rmsnorm_cast<VPT, WARP_ROW, Q>, grid, threads, 0, stream, 0, p);
}

template <int Q>
void launch_norm(const fp8t::norm::Fwd& p, const NormShape& s, int sms, cudaStream_t stream) {
  if (s.warp_row) {
    if (s.vpt == 1)      launch_norm_as<1, true, Q>(p, s.threads, sms, stream);
    else if (s.vpt == 2) launch_norm_as<2, true, Q>(p, s.threads, sms, stream);
    else                 launch_norm_as<4, true, Q>(p, s.threads, sms, stream);
  } else {
    if (s.vpt == 1)      launch_norm_as<1, false, Q>(p, s.threads, sms, stream);
    else if (s.vpt == 2) launch_norm_as<2, false, Q>(p, s.threads, sms, stream);
    else                 launch_norm_as<4, false, Q>(p, s.threads, sms, stream);
  }
}

}  // namespace

extern "C" {

fp8t_status fp8_rmsnorm_cast(const fp8t_rmsnorm* desc, void* stream) {
  t_last_error.clear();
  if (!desc) return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: desc NULL");
  const fp8t_rmsnorm& d = *desc;
  if (!d.x_bf16 || !d.gamma_bf16) return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: NULL input or gamma");
  if (d.rows <= 0 || d.cols <= 0) return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: rows and cols must be > 0");
  if (!(d.eps >= 0.0f) || !std::isfinite(d.eps))
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: eps must be finite and >= 0");
  if (d.quant < FP8T_Q_NONE || d.quant > FP8T_Q_NVFP4)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: unknown quant %d", (int)d.quant);
  if (d.h_bf16 && !d.residual_bf16)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: h without a residual (it is x)");
  const bool fp8 = d.quant == FP8T_Q_FP8, nv = d.quant == FP8T_Q_NVFP4, none = d.quant == FP8T_Q_NONE;
  const bool block = !none && !fp8;
  if (none ? !d.y_bf16 || d.q : !d.q)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: neither y nor codes asked for, or codes without a quant");
  if (block != (d.scales != nullptr))
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: scales go with the block formats and only with them");
  if ((fp8 || nv) ? !d.d_scale || (fp8 && !d.d_amax_inout) : d.d_scale || d.d_amax_inout || d.d_scale_inv_out)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: FP8 needs a scale and an amax slot, NVFP4 a scale; the others have none");
  if ((fp8 || d.quant == FP8T_Q_MXFP8) && d.fmt != FP8T_E4M3 && d.fmt != FP8T_E5M2)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_cast: unknown format %d", (int)d.fmt);
  if (!norm_cols_ok(d.rows, d.cols, block ? 32 : 16))
    return fail(FP8T_ERR_UNSUPPORTED_SHAPE,
                "fp8_rmsnorm_cast: cols must be a multiple of 16 (32 with block scales) and at most %d", fp8t::norm::kMaxCols);
  if (!aligned(d.x_bf16, 16) || !aligned(d.residual_bf16, 16) || !aligned(d.gamma_bf16, 16) ||
      !aligned(d.h_bf16, 16) || !aligned(d.y_bf16, 16) || !aligned(d.q, 16) || !aligned(d.scales, 16) ||
      !aligned(d.d_rstd_out, 4) || !aligned(d.d_scale, 4) || !aligned(d.d_amax_inout, 4) ||
      !aligned(d.d_scale_inv_out, 4))
    return fail(FP8T_ERR_MISALIGNED, "fp8_rmsnorm_cast: misaligned pointer");
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  fp8t::norm::Fwd p = {};
  p.x = static_cast<const uint4*>(d.x_bf16);
  p.res = static_cast<const uint4*>(d.residual_bf16);
  p.gamma = static_cast<const uint4*>(d.gamma_bf16);
  p.h = static_cast<uint4*>(d.h_bf16);
  p.rstd = d.d_rstd_out;
  p.y = static_cast<uint4*>(d.y_bf16);
  p.q = static_cast<uint8_t*>(d.q);
  p.sf = static_cast<uint8_t*>(d.scales);
  p.scale = d.d_scale;
  p.amax_bits = reinterpret_cast<unsigned int*>(d.d_amax_inout);
  p.scale_inv = d.d_scale_inv_out;
  p.rows = d.rows;
  p.cols = static_cast<int32_t>(d.cols);
  p.fmt = d.fmt;
  p.eps = d.eps;
  const NormShape s = norm_shape(d.rows, d.cols);
  switch (d.quant) {
    case FP8T_Q_NONE: launch_norm<fp8t::blk::kNone>(p, s, dev->sms, as_stream(stream)); break;
    case FP8T_Q_FP8: launch_norm<fp8t::blk::kFP8>(p, s, dev->sms, as_stream(stream)); break;
    case FP8T_Q_MXFP8: launch_norm<fp8t::blk::kMXFP8>(p, s, dev->sms, as_stream(stream)); break;
    case FP8T_Q_MXFP4: launch_norm<fp8t::blk::kMXFP4>(p, s, dev->sms, as_stream(stream)); break;
    case FP8T_Q_NVFP4: launch_norm<fp8t::blk::kNVFP4>(p, s, dev->sms, as_stream(stream)); break;
  }
  return after_launch("fp8_rmsnorm_cast launch");
}

size_t fp8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || !norm_cols_ok(rows, cols, 16)) return 0;
  return static_cast<size_t>(norm_backward_shape(rows, cols).ctas * cols * 4);
}

fp8t_status fp8_rmsnorm_backward(const fp8t_rmsnorm_grad* desc, void* d_workspace,
                                 size_t workspace_bytes, void* stream) {
  t_last_error.clear();
  if (!desc) return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_backward: desc NULL");
  const fp8t_rmsnorm_grad& d = *desc;
  if (!d.dy_bf16 || !d.h_bf16 || !d.gamma_bf16 || !d.d_rstd || !d.dh_bf16)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_backward: NULL pointer");
  if (d.rows <= 0 || d.cols <= 0) return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_backward: rows and cols must be > 0");
  if (!norm_cols_ok(d.rows, d.cols, 16))
    return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp8_rmsnorm_backward: cols must be a multiple of 16 and at most %d",
                fp8t::norm::kMaxCols);
  if (!aligned(d.dy_bf16, 16) || !aligned(d.h_bf16, 16) || !aligned(d.gamma_bf16, 16) || !aligned(d.d_rstd, 4) ||
      !aligned(d.dres_bf16, 16) || !aligned(d.dh_bf16, 16) || !aligned(d.dgamma_f32, 4) ||
      !aligned(d.dgamma_bf16, 2) || !aligned(d_workspace, 16))
    return fail(FP8T_ERR_MISALIGNED, "fp8_rmsnorm_backward: misaligned pointer");
  const bool want = d.dgamma_f32 || d.dgamma_bf16;
  const NormBwdShape s = norm_backward_shape(d.rows, d.cols);
  const int64_t ctas = s.ctas;
  if (want && (!d_workspace || workspace_bytes < static_cast<size_t>(ctas * d.cols * 4)))
    return fail(FP8T_ERR_INVALID_ARG, "fp8_rmsnorm_backward: workspace of %zu bytes needed",
                static_cast<size_t>(ctas * d.cols * 4));
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK || (st = ready_norm_backward(dev)) != FP8T_OK) return st;
  using namespace fp8t::norm;
  Bwd p = {};
  p.dy = static_cast<const uint4*>(d.dy_bf16);
  p.h = static_cast<const uint4*>(d.h_bf16);
  p.gamma = static_cast<const uint4*>(d.gamma_bf16);
  p.rstd = d.d_rstd;
  p.dres = static_cast<const uint4*>(d.dres_bf16);
  p.dh = static_cast<uint4*>(d.dh_bf16);
  p.partials = want ? static_cast<float*>(d_workspace) : nullptr;
  p.rows = d.rows;
  p.cols = static_cast<int32_t>(d.cols);
  p.group = s.group;
  const size_t smem = want ? static_cast<size_t>(s.groups - 1) * d.cols * 4 : 0;
  (void)launch_pdl(s.vpt == 1 ? k_rmsnorm_backward<1> : s.vpt == 2 ? k_rmsnorm_backward<2>
             : s.vpt == 3 ? k_rmsnorm_backward<3> : k_rmsnorm_backward<4>,
                   ctas, s.group * s.groups, smem, as_stream(stream), 0, p);
  if ((st = after_launch("fp8_rmsnorm_backward launch")) != FP8T_OK) return st;
  if (want) {
    (void)launch_pdl(k_rmsnorm_dgamma, (d.cols + 31) / 32, 32 * kReduceWarps, 0, as_stream(stream), 0,
                     static_cast<const float*>(p.partials), static_cast<int>(ctas), p.cols, d.dgamma_f32,
                     static_cast<uint16_t*>(d.dgamma_bf16));
    st = after_launch("fp8_rmsnorm_backward dgamma launch");
  }
  return st;
}

}  // extern "C"

// ------------------------------------------------------------------ gated feed-forward
namespace {

template <class Op>
cudaError_t allow_pair_smem() {
  return cudaFuncSetAttribute(fp8t::pair::k_pair_gemm<Op>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fp8t::pair::kPairSmemBytes<Op>);
}
using fp8t::gated::kGelu;
using fp8t::gated::kSilu;
template <int MODE>
cudaError_t muon_small_smem() {
  return cudaFuncSetAttribute(fp8t::muon::k_muon_small<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, fp8t::muon::kSmallSmemBytes);
}
fp8t_status ready_pair(DeviceInfo* d) {
  using namespace fp8t;
  return once_per_device(d->pair_ready, "pair products", [&] {
    cudaError_t e;
    if ((e = allow_pair_smem<gated::Forward<kSilu>>()) != cudaSuccess || (e = allow_pair_smem<gated::Forward<kGelu>>()) != cudaSuccess ||
        (e = allow_pair_smem<gated::Backward<kSilu>>()) != cudaSuccess || (e = allow_pair_smem<gated::Backward<kGelu>>()) != cudaSuccess ||
        (e = allow_pair_smem<muon::Steps<4>>()) != cudaSuccess ||
        (e = allow_pair_smem<muon::Steps<muon::kMaxMatrices>>()) != cudaSuccess ||
        (e = muon_small_smem<muon::kMuon>()) != cudaSuccess || (e = muon_small_smem<muon::kOrthBf16>()) != cudaSuccess ||
        (e = muon_small_smem<muon::kOrthF32>()) != cudaSuccess)
      return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (d->sms / 2), 1, 1);
    cfg.blockDim = dim3(pair::kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = pair::kPairSmemBytes<gated::Forward<kSilu>>;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, pair::k_pair_gemm<gated::Forward<kSilu>>, &cfg) != cudaSuccess || clusters < 1) {
      (void)cudaGetLastError();
      clusters = d->sms / 2;
    }
    // and of the grid-wide steps, whose CTAs all have to be resident
    int together = 0;
    if (cudaOccupancyMaxActiveClusters(&together, pair::k_pair_gemm<muon::Steps<muon::kMaxMatrices>>, &cfg) == cudaSuccess && together > 0)
      clusters = std::min(clusters, together);
    else
      (void)cudaGetLastError();
    d->pair_clusters = clusters;
    return cudaSuccess;
  });
}

// rows x cols elements of `bytes` each, row pitch in elements: boxes of box_rows x box_cols, zero fill.
fp8t_status encode_2d(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, int64_t pitch, int bytes,
                      uint32_t box_rows, uint32_t box_cols, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch * bytes)};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(map, bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(ptr),
                  dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FP8T_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return FP8T_OK;
}

// What the forward and the backward call share; `width`: rows of B as [rows][K], columns of the codes.
struct GatedCall {
  const char* name;
  const void *A, *B;
  fp8t_format a_fmt, b_fmt;
  fp8t_layout b_layout;
  int64_t M, N, K, b_rows;
  const float *sa, *sb;
  fp8t_act act;
  const void *gu, *out16, *q;      // out16, q: M x (N or 2N)
  fp8t_format q_fmt;
  const float* scale;
  float *amax, *scale_inv;
};
fp8t_status check_gated(const GatedCall& c) {
  if (!c.A || !c.B || !c.sa || !c.sb) return fail(FP8T_ERR_INVALID_ARG, "%s: NULL operand or scale inverse", c.name);
  for (int f : {c.a_fmt, c.b_fmt, c.q ? c.q_fmt : FP8T_E4M3})
    if (f != FP8T_E4M3 && f != FP8T_E5M2) return fail(FP8T_ERR_INVALID_ARG, "%s: unknown format %d", c.name, f);
  if (c.b_layout != FP8T_K_MAJOR && c.b_layout != FP8T_MN_MAJOR)
    return fail(FP8T_ERR_INVALID_ARG, "%s: unknown operand layout", c.name);
  if (c.act != FP8T_ACT_SILU && c.act != FP8T_ACT_GELU)
    return fail(FP8T_ERR_INVALID_ARG, "%s: act must be SILU or GELU", c.name);
  if ((c.q != nullptr) != (c.scale != nullptr) || (c.scale_inv && !c.q))
    return fail(FP8T_ERR_INVALID_ARG, "%s: codes need a scale, and scale and scale_inv go with codes", c.name);
  if (c.M <= 0 || c.N <= 0 || c.K <= 0) return fail(FP8T_ERR_INVALID_ARG, "%s: M, N, K must be > 0", c.name);
  const int64_t lim = int64_t(1) << 30;
  if (c.N % 16 || c.K % 16 || c.M >= lim || c.N >= lim || c.K >= lim ||
      (c.M + 255) / 256 * ((c.N + 127) / 128) >= lim)
    return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "%s: N and K must be multiples of 16, all sizes below 2^30", c.name);
  if (!aligned(c.A, 16) || !aligned(c.B, 16) || !aligned(c.gu, 16) || !aligned(c.out16, 16) || !aligned(c.q, 16) ||
      !aligned(c.sa, 4) || !aligned(c.sb, 4) || !aligned(c.scale, 4) || !aligned(c.amax, 4) || !aligned(c.scale_inv, 4))
    return fail(FP8T_ERR_MISALIGNED, "%s: misaligned pointer", c.name);
  return FP8T_OK;
}
// Operands, sizes and scalars.
// outputs: of a tile of 256 columns.
fp8t_status fill_gated(fp8t::gated::Params& p, const GatedCall& c, int outputs, const DeviceInfo* dev) {
  using namespace fp8t::gemm;
  const bool mn = c.b_layout == FP8T_MN_MAJOR;
  p.sa = c.sa;
  p.sb = c.sb;
  p.scale = c.scale;
  p.amax_bits = reinterpret_cast<unsigned int*>(c.amax);
  p.scale_inv = c.scale_inv;
  p.M = static_cast<int32_t>(c.M);
  p.N = static_cast<int32_t>(c.N);
  p.tiles_m = static_cast<int32_t>((c.M + kBM - 1) / kBM);
  // Tiles of half the columns where all of them run at once: half an epilogue at the end (back 512 x 256 x 688 10.1 / 7.1 us). Tiles
  // of three quarters where the rounds of tiles on the clusters get at least a tenth shorter by them (back 1000 x 2048 x 5504 25.2 / 20.4,
  // gated 40 x 4096 -> 2 x 11008 27.3 / 24.9, 1237 x 1024 -> 2 x 2752 with G and U 13.0 / 12.4, without 10.7 / 10.9).
  auto tiles_n = [&](int h) { return (c.N * 128 + outputs * h - 1) / (outputs * h); };
  auto rounds = [&](int h) { return (p.tiles_m * tiles_n(h) + dev->pair_clusters - 1) / dev->pair_clusters; };
  p.half_n = mn ? 128 : rounds(64) == 1 ? 64 : rounds(96) * 96 * 10 <= rounds(128) * 128 * 9 ? 96 : 128;
  // Rows that A does not have are left out of its boxes: what the stage holds there reaches no output. Boxes that begin inside A and
  // are mostly past it are slow to land (9 x 4096 -> 2 x 11008 33.0 / 24.8 us, 16 rows 31.4 / 24.8).
  p.a_rows = static_cast<int32_t>(std::min<int64_t>(kHalf, (c.M + 7) / 8 * 8));
  fp8t_status st = encode_kmajor(&p.a, c.A, c.M, c.K, static_cast<uint32_t>(p.a_rows));
  if (st == FP8T_OK)
    st = mn ? encode_kmajor(&p.b, c.B, c.K, c.b_rows, kBK) : encode_kmajor(&p.b, c.B, c.b_rows, c.K, static_cast<uint32_t>(p.half_n));
  p.tiles_n = static_cast<int32_t>(tiles_n(p.half_n));
  p.total_tiles = p.tiles_m * p.tiles_n;
  p.num_kb = static_cast<int32_t>((c.K + kBK - 1) / kBK);
  p.b_mn = mn ? 1 : 0;
  p.idesc = make_idesc(c.a_fmt, c.b_fmt, 0, p.b_mn) - (static_cast<uint32_t>((128 - p.half_n) / 4) << 17);
  p.act = c.act;
  p.fmt = c.q_fmt;
  p.has_q = c.q != nullptr;
  return st;
}
// Few rows: always up to eight, and up to 32 while the weights, read once for every eight rows, are small. Few-rows kernel / pair
// tiles, graph replays, cold weights. W out x in: 8 x 4096 -> 2 x 11008 21.7 / 26.3 us; 16 x 4096 -> 2 x 2048 (34 MB for two eights)
// 7.8 / 13.4, 16 x 11008 -> 2 x 1024 (45 MB) 14.0 / 27.7, 24 x 2048 -> 2 x 2752 (34 MB) 9.5 / 9.2, 32 x 2048 -> 2 x 2752 (45 MB) 9.9 / 9.2,
// 32 x 1024 -> 2 x 2752 6.9 / 6.9; past the limit 16 x 4096 -> 2 x 11008 34.4 / 24.5. W in x out: 8 x 4096 -> 2 x 11008 21.0 / 27.3;
// 16 x 4096 -> 2 x 2048 12.7 / 14.6, 32 x 2048 -> 2 x 1376 (23 MB) 9.8 / 9.9, 24 x 2048 -> 2 x 2752 10.3 / 10.1, 16 x 256 -> 2 x 688 3.3 / 5.6; past
// the limit 32 x 2048 -> 2 x 2752 11.6 / 10.1. The rule goes by bytes alone: where k is small and n large pair tiles would be faster
// (32 x 512 -> 2 x 5504 8.1 / 6.9 and 11.4 / 7.2), and in x out long k past the limit would be faster here (16 x 11008 -> 2 x 1024 26.1 / 29.6).
bool gated_few_rows(const fp8t_gated& d) {
  const int64_t groups = (d.M + 7) / 8, most = d.b_layout == FP8T_MN_MAJOR ? int64_t(36) << 20 : int64_t(48) << 20;
  return groups == 1 || (d.M <= 32 && groups * 2 * d.N * d.K <= most);
}
// Chunks of a warp's ring for tiles of 32 G outputs: 144 to 192 KB of a CTA.
constexpr int gated_ring(int g) { return g == 1 ? 9 : g == 2 ? 5 : 3; }
template <int WF, int AF, int G>
fp8t_status launch_gated_rows_mn(const fp8t::gated::RowParams& p, cudaLaunchConfig_t& cfg) {
  using namespace fp8t::gated;
  RowMnParams P = {};
  P.p = p;
  P.ring = gated_ring(G);
  const int warps = std::min(kRowWarps, (p.K + 31) / 32);
  cfg.gridDim.x = static_cast<unsigned>((p.N + 32 * G - 1) / (32 * G));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps), 1, 1);
  cfg.dynamicSmemBytes = row_smem_bytes(G, P.ring, warps);
  const fp8t_status st = encode_2d(&P.w, p.w, p.K, 2 * static_cast<int64_t>(p.N), 2 * static_cast<int64_t>(p.N), 1, 32, 32 * G,
                                   G == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st == FP8T_OK) (void)cudaLaunchKernelEx(&cfg, k_gated_rows_mn<WF, AF, G>, P);
  return st;
}
template <int WF, int AF>
fp8t_status launch_gated_rows_as(const fp8t::gated::RowParams& p, bool mn, int sms, cudaStream_t stream) {
  using namespace fp8t::gated;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + 15) / 16), static_cast<unsigned>((p.M + kRowTokens - 1) / kRowTokens), 1);
  cfg.blockDim = dim3(static_cast<unsigned>(32 * std::min(kRowWarps, (p.K + 63) / 64)), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  if (!mn) {
    // two CTAs an SM, two chunks ahead, where the SMs' rounds are fewer for it and there are chunks to be ahead (1 x 4096 -> 2 x 9472
    // 20.0 / 17.4 us, 1 x 11008 -> 2 x 4096 24.9 / 18.4; otherwise 1 x 4096 -> 2 x 11008 20.8 / 21.8)
    const int64_t ctas = static_cast<int64_t>(cfg.gridDim.x) * cfg.gridDim.y;
    const bool ahead = p.K >= 2048 && (ctas + 2 * sms - 1) / (2 * sms) * 2 < (ctas + 3 * sms - 1) / (3 * sms) * 3;
    (void)(ahead ? cudaLaunchKernelEx(&cfg, k_gated_rows<WF, AF, 2>, p) : cudaLaunchKernelEx(&cfg, k_gated_rows<WF, AF, 1>, p));
    return FP8T_OK;
  }
  // Tiles for which the SMs' rounds take the least time, a CTA an SM: its time goes with the width, and something for its start.
  // The ring keeps a second CTA out: it would be the next call's, and take a place that the scheduler then fills unevenly (1 x 4096
  // -> 2 x 11008 in 172 tiles of 64, two an SM, 23.0 us; in 115 of 96 18.3, now 19.4 with slots filled behind their reads).
  const int64_t groups = cfg.gridDim.y;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int g = 1; g <= 4; ++g) {
    const int64_t cost = ((p.N + 32 * g - 1) / (32 * g) * groups + sms - 1) / sms * (2 * g + 1);
    if (cost < least) least = cost, best = g;
  }
  switch (best) {
    case 1: return launch_gated_rows_mn<WF, AF, 1>(p, cfg);
    case 2: return launch_gated_rows_mn<WF, AF, 2>(p, cfg);
    case 3: return launch_gated_rows_mn<WF, AF, 3>(p, cfg);
    default: return launch_gated_rows_mn<WF, AF, 4>(p, cfg);
  }
}
template <int WF, int AF, int G>
cudaError_t allow_gated_rows_smem_of() {
  using namespace fp8t::gated;
  return cudaFuncSetAttribute(k_gated_rows_mn<WF, AF, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              row_smem_bytes(G, gated_ring(G), kRowWarps));
}
template <int WF, int AF>
cudaError_t allow_gated_rows_smem() {
  cudaError_t e;
  if ((e = allow_gated_rows_smem_of<WF, AF, 1>()) != cudaSuccess || (e = allow_gated_rows_smem_of<WF, AF, 2>()) != cudaSuccess ||
      (e = allow_gated_rows_smem_of<WF, AF, 3>()) != cudaSuccess)
    return e;
  return allow_gated_rows_smem_of<WF, AF, 4>();
}
fp8t_status ready_gated_rows(DeviceInfo* d) {
  return once_per_device(d->gated_rows_ready, "fp8_gated_gemm", [] {
    cudaError_t e;
    if ((e = allow_gated_rows_smem<0, 0>()) != cudaSuccess || (e = allow_gated_rows_smem<0, 1>()) != cudaSuccess ||
        (e = allow_gated_rows_smem<1, 0>()) != cudaSuccess)
      return e;
    return allow_gated_rows_smem<1, 1>();
  });
}
fp8t_status launch_gated_rows(const fp8t_gated& d, int sms, cudaStream_t stream) {
  fp8t::gated::RowParams p = {};
  p.a = static_cast<const uint8_t*>(d.A);
  p.w = static_cast<const uint8_t*>(d.B);
  p.gu = static_cast<uint16_t*>(d.gu_bf16);
  p.h = static_cast<uint16_t*>(d.h_bf16);
  p.q = static_cast<uint8_t*>(d.q);
  p.sa = d.d_a_scale_inv;
  p.sb = d.d_b_scale_inv;
  p.scale = d.d_scale;
  p.amax_bits = reinterpret_cast<unsigned int*>(d.d_amax_inout);
  p.scale_inv = d.d_scale_inv_out;
  p.M = static_cast<int32_t>(d.M);
  p.N = static_cast<int32_t>(d.N);
  p.K = static_cast<int32_t>(d.K);
  p.act = d.act;
  p.fmt = d.q_fmt;
  const bool mn = d.b_layout == FP8T_MN_MAJOR, w5 = d.b_fmt == FP8T_E5M2, a5 = d.a_fmt == FP8T_E5M2;
  const fp8t_status st = w5 ? (a5 ? launch_gated_rows_as<1, 1>(p, mn, sms, stream) : launch_gated_rows_as<1, 0>(p, mn, sms, stream))
                            : (a5 ? launch_gated_rows_as<0, 1>(p, mn, sms, stream) : launch_gated_rows_as<0, 0>(p, mn, sms, stream));
  return st != FP8T_OK ? st : after_launch("fp8_gated_gemm launch");
}

template <class Op, class P>
fp8t_status launch_pair(const P& p, const DeviceInfo* dev, const char* what, cudaStream_t stream) {
  const int64_t grid = 2 * std::min<int64_t>(p.total_tiles, dev->pair_clusters);
  (void)launch_pdl(fp8t::pair::k_pair_gemm<Op>, grid, fp8t::pair::kPairThreads, fp8t::pair::kPairSmemBytes<Op>, stream, 0, p);
  return after_launch(what);
}
// Most warps, CTAs per SM and loads ahead of a matrix-vector launch.
template <bool NV, int W, int B, bool AHEAD>
void launch_matvec_as(const fp8t::mv::Params& p, int64_t ctas, cudaStream_t stream) {
  const int warps = std::min(W, (p.K + 127) / 128);
  (void)launch_pdl(fp8t::mv::k_fp4_matvec<NV, W, B, AHEAD>, ctas, 32 * warps, 0, stream, 0, p);
}
// As many CTAs as SMs or fewer: 16 warps each, the next chunk on its way during a chunk's arithmetic. More: 8 warps, three CTAs on
// an SM in each other's shadow. First / second, graph replays with cold weights: 1 x 4096 x 4096 4.6 / 8.4 us, 8 x 11008 x 4096
// 9.9 / 21.8, 4 x 4096 x 2 x 11008 25.8 / 18.3.
template <bool NV>
void launch_matvec_of(const fp8t::mv::Params& p, int sms, cudaStream_t stream) {
  const int64_t per = fp8t::mv::kGroups * (p.act ? 8 : 16), ctas = (p.N + per - 1) / per;
  if (ctas <= sms) launch_matvec_as<NV, 16, 1, true>(p, ctas, stream);
  else launch_matvec_as<NV, 8, 3, false>(p, ctas, stream);
}
void launch_matvec(const fp8t::mv::Params& p, bool nv, int sms, cudaStream_t stream) {
  nv ? launch_matvec_of<true>(p, sms, stream) : launch_matvec_of<false>(p, sms, stream);
}

constexpr CUtensorMapSwizzle kSwizzle16 = CU_TENSOR_MAP_SWIZZLE_64B, kSwizzle8 = CU_TENSOR_MAP_SWIZZLE_32B;

}  // namespace

extern "C" {

fp8t_status fp8_gated_gemm(const fp8t_gated* desc, void* stream) {
  t_last_error.clear();
  if (!desc) return fail(FP8T_ERR_INVALID_ARG, "fp8_gated_gemm: desc NULL");
  const fp8t_gated& d = *desc;
  const GatedCall c = {"fp8_gated_gemm", d.A, d.B, d.a_fmt, d.b_fmt, d.b_layout, d.M, d.N, d.K, 2 * d.N, d.d_a_scale_inv,
                       d.d_b_scale_inv, d.act, d.gu_bf16, d.h_bf16, d.q, d.q_fmt, d.d_scale, d.d_amax_inout, d.d_scale_inv_out};
  fp8t_status st = check_gated(c);
  if (st != FP8T_OK) return st;
  if (!d.gu_bf16 && !d.h_bf16 && !d.q) return fail(FP8T_ERR_INVALID_ARG, "fp8_gated_gemm: no output asked for");
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != FP8T_OK) return st;
  if (gated_few_rows(d)) return (st = ready_gated_rows(dev)) != FP8T_OK ? st : launch_gated_rows(d, dev->sms, as_stream(stream));
  if ((st = ready_pair(dev)) != FP8T_OK) return st;
  fp8t::gated::Params p = {};
  if ((st = fill_gated(p, c, 128, dev)) != FP8T_OK) return st;
  p.keep = d.gu_bf16 != nullptr;
  p.has_h = d.h_bf16 != nullptr;
  if (p.keep && ((st = encode_2d(&p.o0, d.gu_bf16, d.M, d.N, 2 * d.N, 2, 32, 32, kSwizzle16)) != FP8T_OK ||
                 (st = encode_2d(&p.o1, static_cast<const uint16_t*>(d.gu_bf16) + d.N, d.M, d.N, 2 * d.N, 2, 32, 32, kSwizzle16)) != FP8T_OK))
    return st;
  if (p.has_h && (st = encode_2d(&p.h, d.h_bf16, d.M, d.N, d.N, 2, 32, 32, kSwizzle16)) != FP8T_OK) return st;
  if (p.has_q && (st = encode_2d(&p.q0, d.q, d.M, d.N, d.N, 1, 32, 32, kSwizzle8)) != FP8T_OK) return st;
  using namespace fp8t::gated;
  return d.act == FP8T_ACT_SILU ? launch_pair<Forward<kSilu>>(p, dev, "fp8_gated_gemm launch", as_stream(stream))
                                : launch_pair<Forward<kGelu>>(p, dev, "fp8_gated_gemm launch", as_stream(stream));
}

fp8t_status fp8_gated_gemm_backward(const fp8t_gated_grad* desc, void* stream) {
  t_last_error.clear();
  if (!desc) return fail(FP8T_ERR_INVALID_ARG, "fp8_gated_gemm_backward: desc NULL");
  const fp8t_gated_grad& d = *desc;
  const GatedCall c = {"fp8_gated_gemm_backward", d.A, d.B, d.a_fmt, d.b_fmt, d.b_layout, d.M, d.N, d.K, d.N, d.d_a_scale_inv,
                       d.d_b_scale_inv, d.act, d.gu_bf16, d.dgu_bf16, d.q, d.q_fmt, d.d_scale, d.d_amax_inout, d.d_scale_inv_out};
  fp8t_status st = check_gated(c);
  if (st != FP8T_OK) return st;
  if (!d.gu_bf16) return fail(FP8T_ERR_INVALID_ARG, "fp8_gated_gemm_backward: gu NULL");
  if (!d.dgu_bf16 && !d.q) return fail(FP8T_ERR_INVALID_ARG, "fp8_gated_gemm_backward: no output asked for");
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != FP8T_OK || (st = ready_pair(dev)) != FP8T_OK) return st;
  fp8t::gated::Params p = {};
  if ((st = fill_gated(p, c, fp8t::gemm::kBN, dev)) != FP8T_OK) return st;
  if ((st = encode_2d(&p.g, d.gu_bf16, d.M, d.N, 2 * d.N, 2, 32, 32, kSwizzle16)) != FP8T_OK ||
      (st = encode_2d(&p.u, static_cast<const uint16_t*>(d.gu_bf16) + d.N, d.M, d.N, 2 * d.N, 2, 32, 32, kSwizzle16)) != FP8T_OK)
    return st;
  p.keep = d.dgu_bf16 != nullptr;
  if (p.keep && ((st = encode_2d(&p.o0, d.dgu_bf16, d.M, d.N, 2 * d.N, 2, 32, 32, kSwizzle16)) != FP8T_OK ||
                 (st = encode_2d(&p.o1, static_cast<const uint16_t*>(d.dgu_bf16) + d.N, d.M, d.N, 2 * d.N, 2, 32, 32, kSwizzle16)) != FP8T_OK))
    return st;
  if (p.has_q && ((st = encode_2d(&p.q0, d.q, d.M, d.N, 2 * d.N, 1, 32, 32, kSwizzle8)) != FP8T_OK ||
                  (st = encode_2d(&p.q1, static_cast<const uint8_t*>(d.q) + d.N, d.M, d.N, 2 * d.N, 1, 32, 32, kSwizzle8)) != FP8T_OK))
    return st;
  using namespace fp8t::gated;
  return d.act == FP8T_ACT_SILU ? launch_pair<Backward<kSilu>>(p, dev, "fp8_gated_gemm_backward launch", as_stream(stream))
                                : launch_pair<Backward<kGelu>>(p, dev, "fp8_gated_gemm_backward launch", as_stream(stream));
}

// ------------------------------------------------------------------ 4-bit weights times a few tokens
fp8t_status fp4_matvec(const fp8t_fp4_matvec* desc, void* stream) {
  t_last_error.clear();
  if (!desc) return fail(FP8T_ERR_INVALID_ARG, "fp4_matvec: desc NULL");
  const fp8t_fp4_matvec& d = *desc;
  if (!d.x_bf16 || !d.q || !d.scales || !d.y_bf16) return fail(FP8T_ERR_INVALID_ARG, "fp4_matvec: NULL pointer");
  if (d.quant != FP8T_Q_MXFP4 && d.quant != FP8T_Q_NVFP4)
    return fail(FP8T_ERR_INVALID_ARG, "fp4_matvec: quant must be MXFP4 or NVFP4");
  if (d.act < FP8T_ACT_NONE || d.act > FP8T_ACT_GELU) return fail(FP8T_ERR_INVALID_ARG, "fp4_matvec: unknown act %d", (int)d.act);
  if (d.rows <= 0 || d.N <= 0 || d.K <= 0) return fail(FP8T_ERR_INVALID_ARG, "fp4_matvec: rows, N, K must be > 0");
  const int64_t lim = int64_t(1) << 30;
  if (d.rows > fp8t::mv::kMaxRows || d.N % 8 || d.K % 32 || d.N >= lim || d.K >= lim)
    return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "fp4_matvec: at most 8 rows, N a multiple of 8 and K of 32, both below 2^30");
  if (!aligned(d.x_bf16, 16) || !aligned(d.q, 16) || !aligned(d.scales, 16) || !aligned(d.y_bf16, 16) ||
      !aligned(d.d_w_scale_inv, 4))
    return fail(FP8T_ERR_MISALIGNED, "fp4_matvec: misaligned pointer");
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  fp8t::mv::Params p = {};
  p.x = static_cast<const uint16_t*>(d.x_bf16);
  p.q = static_cast<const uint8_t*>(d.q);
  p.sf = static_cast<const uint8_t*>(d.scales);
  p.factor = d.d_w_scale_inv;
  p.y = static_cast<uint16_t*>(d.y_bf16);
  p.rows = static_cast<int32_t>(d.rows);
  p.N = static_cast<int32_t>(d.N);
  p.K = static_cast<int32_t>(d.K);
  const bool nv = d.quant == FP8T_Q_NVFP4;
  p.words = static_cast<int32_t>(fp8t::blk::atoms_per_row(d.K, nv ? fp8t::blk::kNVFP4 : fp8t::blk::kMXFP4));
  p.act = d.act;
  launch_matvec(p, nv, dev->sms, as_stream(stream));
  return after_launch("fp4_matvec launch");
}

}  // extern "C"

// ------------------------------------------------------------------ Newton-Schulz and Muon
namespace {

constexpr int64_t kMaxMuonSide = 65536;
int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Where a matrix's FP16 copies lie in a batch's part of the workspace: X twice, A and B.
struct MuonSizes {
  int64_t rows, cols, side, pitch_x, pitch_s;
  size_t x, s;                     // bytes of X, of A
  MuonSizes(int64_t r, int64_t c) : rows(r), cols(c), side(std::min(r, c)), pitch_x(round_up(c, 8)), pitch_s(round_up(side, 8)) {
    x = static_cast<size_t>(round_up(rows * pitch_x * 2, 256));
    s = static_cast<size_t>(round_up(side * pitch_s * 2, 256));
  }
  size_t bytes() const { return 2 * x + 2 * s; }
  int64_t chunks() const { return (rows * cols + fp8t::muon::kChunk - 1) / fp8t::muon::kChunk; }
};
// The workspace: a norm per matrix, the partial sums of the largest batch, the copies of the largest batch.
struct MuonPlan {
  size_t norms = 0, partials = 0, copies = 0;
  bool ok = true;
  template <class Shape>
  MuonPlan(int32_t n, Shape&& shape) {
    for (int32_t b0 = 0; b0 < n && ok; b0 += fp8t::muon::kMaxMatrices) {
      size_t copy = 0;
      int64_t chunks = 0;
      for (int32_t i = b0; i < std::min<int32_t>(n, b0 + fp8t::muon::kMaxMatrices); ++i) {
        const std::pair<int64_t, int64_t> v = shape(i);
        if (v.first <= 0 || v.second <= 0 || v.first > kMaxMuonSide || v.second > kMaxMuonSide) {
          ok = false;
          return;
        }
        const MuonSizes s(v.first, v.second);
        copy += s.bytes();
        chunks += s.chunks();
      }
      copies = std::max(copies, copy);
      partials = std::max(partials, static_cast<size_t>(round_up(chunks * 8, 256)));
    }
    norms = static_cast<size_t>(round_up(static_cast<int64_t>(n) * sizeof(fp8t::muon::Norm) + 12, 256));   // and three words
  }
  size_t bytes() const { return norms + partials + copies; }
};

// Tiles of A and of X in columns of tile_n; half: only those of A on and above the diagonal.
int64_t muon_sym_tiles(const MuonSizes& z, int tile_n, bool half) {
  const int64_t m = (z.side + 255) / 256;
  return half ? m * (m + 1) / 2 : m * ((z.side + tile_n - 1) / tile_n);
}
int64_t muon_x_tiles(const MuonSizes& z, int tile_n) { return (z.rows + 255) / 256 * ((z.cols + tile_n - 1) / tile_n); }
// A matrix's tensor maps and tiles.
fp8t_status fill_muon_matrix(fp8t::muon::Matrix& m, const MuonSizes& z, char* at, int tile_n, bool half, int32_t& sym_tiles,
                             int32_t& x_tiles) {
  fp8t_status st = FP8T_OK;
  for (int i = 0; i < 2; ++i) {
    char *x = at + i * z.x, *s = at + 2 * z.x + i * z.s;
    if ((st = encode_2d(&m.x[i], x, z.rows, z.cols, z.pitch_x, 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)) != FP8T_OK ||
        (st = encode_2d(&m.s[i], s, z.side, z.side, z.pitch_s, 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)) != FP8T_OK ||
        (st = encode_2d(&m.xd[i], x, z.rows, z.cols, z.pitch_x, 2, 32, 32, kSwizzle16)) != FP8T_OK ||
        (st = encode_2d(&m.sd[i], s, z.side, z.side, z.pitch_s, 2, 32, 32, kSwizzle16)) != FP8T_OK)
      return st;
  }
  m.rows = static_cast<int32_t>(z.rows);
  m.cols = static_cast<int32_t>(z.cols);
  m.sym_start = sym_tiles;
  m.x_start = x_tiles;
  sym_tiles += static_cast<int32_t>(muon_sym_tiles(z, tile_n, half));
  x_tiles += static_cast<int32_t>(muon_x_tiles(z, tile_n));
  return st;
}
// The steps of a table's matrices `which`, grid-wide: their launch's parameters, then the launch.
template <class G>
G& muon_group() {
  static thread_local G g;
  return g;
}
template <int NP>
fp8t_status prepare_newton_schulz(const std::vector<MuonSizes>& z, const std::vector<char*>& at, const std::vector<int32_t>& which,
                                  int32_t steps, const fp8t::pair::Grid& grid, const DeviceInfo* dev) {
  fp8t::muon::Group<NP>& g = muon_group<fp8t::muon::Group<NP>>();
  g.n = static_cast<int32_t>(which.size());
  g.steps = steps;
  g.sym_tiles = g.x_tiles = 0;
  g.grid = grid;
  // Where all tiles of A fit the clusters at once, computing both halves spares the transposed stores; where tiles half as wide
  // do, a phase has half the columns to compute and to store (1237 x 611 190 / 151 us).
  int64_t whole = 0, narrow = 0;
  for (int32_t k : which) {
    whole += muon_sym_tiles(z[k], 256, false);
    narrow += std::max(muon_sym_tiles(z[k], 128, false), muon_x_tiles(z[k], 128));
  }
  g.tile_n = narrow <= dev->pair_clusters ? 128 : 256;
  g.whole = whole <= dev->pair_clusters ? 1 : 0;
  for (int32_t k = 0; k < g.n; ++k) {
    const fp8t_status st = fill_muon_matrix(g.m[k], z[which[k]], at[which[k]], g.tile_n, !g.whole, g.sym_tiles, g.x_tiles);
    if (st != FP8T_OK) return st;
  }
  return FP8T_OK;
}
template <int NP>
fp8t_status newton_schulz(const DeviceInfo* dev, cudaStream_t stream) {
  using Op = fp8t::muon::Steps<NP>;
  const fp8t::muon::Group<NP>& g = muon_group<fp8t::muon::Group<NP>>();
  // its CTAs wait for one another: a cooperative launch has them all resident or fails
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(std::max(g.sym_tiles, g.x_tiles), dev->pair_clusters)), 1, 1);
  cfg.blockDim = dim3(fp8t::pair::kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = fp8t::pair::kPairSmemBytes<Op>;
  cfg.stream = stream;
  cudaLaunchAttribute together[1];
  together[0].id = cudaLaunchAttributeCooperative;
  together[0].val.cooperative = 1;
  cfg.attrs = together;
  cfg.numAttrs = 1;
  (void)cudaLaunchKernelEx(&cfg, fp8t::pair::k_pair_gemm<Op>, g);
  return after_launch("Newton-Schulz products launch");
}
bool muon_small(const MuonSizes& z) { return std::max(z.rows, z.cols) <= fp8t::muon::kSmallSide; }
// The same for matrices of at most 256 x 256, a CTA pair each.
fp8t_status prepare_newton_schulz_small(const std::vector<MuonSizes>& z, const std::vector<char*>& at,
                                        const std::vector<int32_t>& which, int32_t steps, int32_t* expired) {
  using namespace fp8t::muon;
  SmallGroup& g = muon_group<SmallGroup>();
  g.steps = steps;
  g.expired = expired;
  for (size_t k = 0; k < which.size(); ++k) {
    const MuonSizes& s = z[which[k]];
    SmallMatrix& m = g.m[k];
    char* x = at[which[k]];
    const fp8t_status st = encode_2d(&m.x, x, s.rows, s.cols, s.pitch_x, 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != FP8T_OK) return st;
    m.out = reinterpret_cast<uint16_t*>(x + (steps & 1 ? s.x : 0));
    m.rows = static_cast<int32_t>(s.rows);
    m.cols = static_cast<int32_t>(s.cols);
    m.pitch = static_cast<int32_t>(s.pitch_x);
  }
  return FP8T_OK;
}
// A table's steps: the longest matrices first, for a cluster takes every n-th tile and the phase of A should end with the
// shortest (its K is the longer side). large, small: how many of each form.
fp8t_status prepare_table(const std::vector<MuonSizes>& z, char* copies, int32_t steps, const fp8t::pair::Grid& grid,
                          const DeviceInfo* dev, size_t& n_large, size_t& n_small) {
  std::vector<char*> at(z.size());
  std::vector<int32_t> large, small;
  for (size_t k = 0; k < z.size(); copies += z[k].bytes(), ++k) {
    at[k] = copies;
    (muon_small(z[k]) ? small : large).push_back(static_cast<int32_t>(k));
  }
  std::stable_sort(large.begin(), large.end(), [&](int32_t a, int32_t b) { return std::max(z[a].rows, z[a].cols) > std::max(z[b].rows, z[b].cols); });
  n_large = large.size();
  n_small = small.size();
  fp8t_status st = FP8T_OK;
  if (n_large > 0)
    st = n_large <= 4 ? prepare_newton_schulz<4>(z, at, large, steps, grid, dev)
                      : prepare_newton_schulz<fp8t::muon::kMaxMatrices>(z, at, large, steps, grid, dev);
  if (st == FP8T_OK && n_small > 0) st = prepare_newton_schulz_small(z, at, small, steps, grid.expired);
  return st;
}
fp8t_status launch_table(size_t n_large, size_t n_small, const DeviceInfo* dev, cudaStream_t stream) {
  using namespace fp8t::muon;
  fp8t_status st = FP8T_OK;
  if (n_large > 0) st = n_large <= 4 ? newton_schulz<4>(dev, stream) : newton_schulz<kMaxMatrices>(dev, stream);
  if (st != FP8T_OK || n_small == 0) return st;
  (void)launch_pdl(k_muon_small<kMuon>, 2 * static_cast<int64_t>(n_small), kSmallThreads, kSmallSmemBytes, stream, 0,
                   muon_group<SmallGroup>());
  return after_launch("Newton-Schulz products launch");
}

// Of the batch's matrices [b0, b1), those of at most 256 x 256, orthogonalised by one kernel.
template <int MODE, class Get>
fp8t_status orthogonalize_small(const char* name, int32_t b0, int32_t b1, int32_t steps, cudaStream_t stream, Get&& get) {
  using namespace fp8t::muon;
  static thread_local SmallGroup g;
  g.steps = steps;
  g.expired = nullptr;
  int32_t k = 0;
  for (int32_t i = b0; i < b1; ++i) {
    int64_t r, c;
    Tensor T;
    get(i, T, r, c);
    if (!muon_small(MuonSizes(r, c))) continue;
    SmallMatrix& m = g.m[k++];
    m.g = T.g;
    m.out = T.w;
    m.rows = static_cast<int32_t>(r);
    m.cols = static_cast<int32_t>(c);
  }
  if (k == 0) return FP8T_OK;
  (void)launch_pdl(k_muon_small<MODE>, 2 * static_cast<int64_t>(k), kSmallThreads, kSmallSmemBytes, stream, 0, g);
  return after_launch(name);
}

// Both calls; `get(i)` gives the kernels' view of matrix i (x, chunk_start and pitch are filled here).
template <int MODE, class Get>
fp8t_status muon_call(const char* name, int32_t n, int32_t steps, fp8t::muon::Table& t, void* d_workspace, size_t workspace_bytes,
                      cudaStream_t stream, Get&& get) {
  using namespace fp8t::muon;
  auto shape = [&](int32_t i) {
    int64_t r, c;
    Tensor T;
    get(i, T, r, c);
    return std::make_pair(r, c);
  };
  const MuonPlan plan(n, shape);
  if (!plan.ok) return fail(FP8T_ERR_UNSUPPORTED_SHAPE, "%s: rows and cols must be 1 to 65536", name);
  if (!d_workspace || workspace_bytes < plan.bytes())
    return fail(FP8T_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed", name, plan.bytes());
  if (!aligned(d_workspace, 256)) return fail(FP8T_ERR_MISALIGNED, "%s: misaligned workspace", name);
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK || (st = ready_pair(dev)) != FP8T_OK) return st;
  char* ws = static_cast<char*>(d_workspace);
  t.norms = reinterpret_cast<Norm*>(ws);
  t.grid.counter = reinterpret_cast<unsigned int*>(t.norms + n);
  t.grid.expired = reinterpret_cast<int32_t*>(t.norms + n) + 1;
  t.gave_up = t.grid.expired + 1;
  t.partials = reinterpret_cast<double*>(ws + plan.norms);
  char* copies = ws + plan.norms + plan.partials;
  t.all = n;
  std::vector<MuonSizes> sizes;
  auto table = [&](int32_t b0) {
    const int32_t b1 = std::min<int32_t>(n, b0 + kMaxMatrices);
    sizes.clear();
    t.n = 0;
    t.first = b0;
    t.chunks = 0;
    char* at = copies;
    for (int32_t i = b0; i < b1; ++i) {
      Tensor& T = t.t[t.n];
      int64_t r, c;
      get(i, T, r, c);
      if (MODE != kMuon && muon_small(MuonSizes(r, c))) continue;
      ++t.n;
      sizes.emplace_back(r, c);
      T.x = reinterpret_cast<uint16_t*>(at);
      T.numel = r * c;
      T.cols = static_cast<int32_t>(c);
      T.pitch = static_cast<int32_t>(sizes.back().pitch_x);
      T.chunk_start = t.chunks;
      t.chunks += static_cast<int32_t>(sizes.back().chunks());
      at += sizes.back().bytes();
    }
  };
  // every norm before the first write: a non-finite one anywhere leaves all matrices as they are
  for (int32_t b0 = 0; b0 < n; b0 += kMaxMatrices) {
    table(b0);
    if (t.n == 0) continue;
    (void)launch_pdl(k_muon_sumsq<MODE>, t.chunks, kPassThreads, 0, stream, 0, t);
    if ((st = after_launch(name)) != FP8T_OK) return st;
    (void)launch_pdl(k_muon_norms, t.n, kPassThreads, 0, stream, 0, t);
    if ((st = after_launch(name)) != FP8T_OK) return st;
  }
  for (int32_t b0 = 0; b0 < n; b0 += kMaxMatrices) {
    if (MODE != kMuon && (st = orthogonalize_small<MODE>(name, b0, std::min<int32_t>(n, b0 + kMaxMatrices), steps, stream, get)) != FP8T_OK)
      return st;
    if (n > kMaxMatrices) table(b0);
    if (t.n == 0) continue;
    // what can fail on the host comes before the first kernel that changes a tensor, but for the launches themselves
    size_t large = 0, small = 0;
    if ((st = prepare_table(sizes, copies, steps, t.grid, dev, large, small)) != FP8T_OK) return st;
    t.last = b0 + kMaxMatrices >= n;
    (void)launch_pdl(k_muon_scale<MODE>, t.chunks, kPassThreads, 0, stream, 0, t);
    if ((st = after_launch(name)) != FP8T_OK) return st;
    if ((st = launch_table(large, small, dev, stream)) != FP8T_OK) return st;
    if (steps & 1)                 // the result is in the second copy
      for (int32_t i = 0; i < t.n; ++i) t.t[i].x += sizes[i].x / 2;
    (void)launch_pdl(k_muon_apply<MODE>, t.chunks, kPassThreads, 0, stream, 0, t);
    if ((st = after_launch(name)) != FP8T_OK) return st;
  }
  return FP8T_OK;
}

// What a call reads and writes, by address and matrix; `own`: a matrix's output may be its own input.
struct MuonBuffer {
  const void* p;
  int32_t matrix;
  bool own;
};
bool by_address(const MuonBuffer& a, const MuonBuffer& b) { return std::less<const void*>()(a.p, b.p); }
// Whether an address is written twice, or written for one matrix and read for another (the tables of a long list run one after
// the other).
bool muon_conflict(std::vector<MuonBuffer>& outs, std::vector<MuonBuffer>& ins) {
  std::sort(outs.begin(), outs.end(), by_address);
  std::sort(ins.begin(), ins.end(), by_address);
  for (size_t i = 0; i + 1 < outs.size(); ++i)
    if (outs[i].p == outs[i + 1].p) return true;
  for (const MuonBuffer& o : outs)
    for (auto it = std::lower_bound(ins.begin(), ins.end(), o, by_address); it != ins.end() && it->p == o.p; ++it)
      if (!o.own || it->matrix != o.matrix) return true;
  return false;
}
// No exception leaves a C entry: the lists above are the only ones that allocate.
template <class F>
fp8t_status without_exceptions(const char* name, F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(FP8T_ERR_CUDA, "%s: %s", name, e.what());
  }
}

}  // namespace

extern "C" {

size_t muon_workspace_bytes(const int64_t* rows, const int64_t* cols, int32_t n_matrices) {
  if (!rows || !cols || n_matrices < 1 || n_matrices > 4096) return 0;
  const MuonPlan plan(n_matrices, [&](int32_t i) { return std::make_pair(rows[i], cols[i]); });
  return plan.ok ? plan.bytes() : 0;
}

fp8t_status muon_orthogonalize(const fp8t_orth_matrix* matrices, int32_t n_matrices, int32_t x_f32, int32_t steps,
                               void* d_workspace, size_t workspace_bytes, void* stream) {
  t_last_error.clear();
  if (!matrices || n_matrices < 1 || n_matrices > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "muon_orthogonalize: matrices NULL or n_matrices out of range");
  if (steps < 1 || steps > 16) return fail(FP8T_ERR_INVALID_ARG, "muon_orthogonalize: steps in 1..16");
  return without_exceptions("muon_orthogonalize", [&]() -> fp8t_status {
    std::vector<MuonBuffer> outs, ins;
    for (int32_t i = 0; i < n_matrices; ++i) {
      const fp8t_orth_matrix& m = matrices[i];
      if (!m.x || !m.out_bf16) return fail(FP8T_ERR_INVALID_ARG, "muon_orthogonalize: matrix %d: NULL pointer", i);
      if (x_f32 && m.x == m.out_bf16) return fail(FP8T_ERR_INVALID_ARG, "muon_orthogonalize: matrix %d: out is the f32 input", i);
      if (!aligned(m.x, 16) || !aligned(m.out_bf16, 16))
        return fail(FP8T_ERR_MISALIGNED, "muon_orthogonalize: matrix %d: misaligned pointer", i);
      outs.push_back({m.out_bf16, i, true});
      ins.push_back({m.x, i, true});
    }
    if (muon_conflict(outs, ins)) return fail(FP8T_ERR_INVALID_ARG, "muon_orthogonalize: a result twice, or in another matrix");
    fp8t::muon::Table t = {};
    auto get = [&](int32_t i, fp8t::muon::Tensor& T, int64_t& r, int64_t& c) {
      T = {};
      T.g = matrices[i].x;
      T.w = static_cast<uint16_t*>(matrices[i].out_bf16);
      r = matrices[i].rows;
      c = matrices[i].cols;
    };
    return x_f32 ? muon_call<fp8t::muon::kOrthF32>("muon_orthogonalize", n_matrices, steps, t, d_workspace, workspace_bytes, as_stream(stream), get)
                 : muon_call<fp8t::muon::kOrthBf16>("muon_orthogonalize", n_matrices, steps, t, d_workspace, workspace_bytes, as_stream(stream), get);
  });
}

fp8t_status fused_muon_multi_tensor(const fp8t_muon_tensor* tensors, int32_t n_tensors, float lr, float beta,
                                    float weight_decay, float update_rms, float loss_scale, int32_t nesterov,
                                    int32_t steps, int32_t* d_skipped_out, void* d_workspace, size_t workspace_bytes,
                                    void* stream) {
  t_last_error.clear();
  if (!tensors || n_tensors < 1 || n_tensors > 4096)
    return fail(FP8T_ERR_INVALID_ARG, "fused_muon_multi_tensor: tensors NULL or n_tensors out of range");
  if (steps < 1 || steps > 16) return fail(FP8T_ERR_INVALID_ARG, "fused_muon_multi_tensor: steps in 1..16");
  if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale) || !std::isfinite(lr) || !std::isfinite(beta) ||
      !std::isfinite(weight_decay) || !std::isfinite(update_rms))
    return fail(FP8T_ERR_INVALID_ARG, "fused_muon_multi_tensor: non-finite hyperparameter or loss_scale <= 0");
  return without_exceptions("fused_muon_multi_tensor", [&]() -> fp8t_status {
    std::vector<MuonBuffer> outs, ins;
    for (int32_t i = 0; i < n_tensors; ++i) {
      const fp8t_muon_tensor& m = tensors[i];
      if (!m.master || !m.momentum || !m.grad_bf16 || !m.weight_bf16)
        return fail(FP8T_ERR_INVALID_ARG, "fused_muon_multi_tensor: tensor %d: NULL pointer", i);
      if (!aligned(m.master, 16) || !aligned(m.momentum, 16) || !aligned(m.grad_bf16, 16) || !aligned(m.weight_bf16, 16))
        return fail(FP8T_ERR_MISALIGNED, "fused_muon_multi_tensor: tensor %d: misaligned pointer", i);
      outs.push_back({m.master, i, false});
      outs.push_back({m.momentum, i, false});
      outs.push_back({m.weight_bf16, i, true});
      ins.push_back({m.grad_bf16, i, true});
    }
    if (muon_conflict(outs, ins)) return fail(FP8T_ERR_INVALID_ARG, "fused_muon_multi_tensor: a tensor is written twice or read elsewhere");
    if (!aligned(d_skipped_out, 4)) return fail(FP8T_ERR_MISALIGNED, "fused_muon_multi_tensor: misaligned skipped");
    fp8t::muon::Table t = {};
    t.beta = beta;
    t.inv_scale = static_cast<float>(1.0 / static_cast<double>(loss_scale));
    t.keep = static_cast<float>(1.0 - static_cast<double>(lr) * static_cast<double>(weight_decay));
    t.nesterov = nesterov ? 1 : 0;
    t.skipped = d_skipped_out;
    auto get = [&](int32_t i, fp8t::muon::Tensor& T, int64_t& r, int64_t& c) {
      const fp8t_muon_tensor& m = tensors[i];
      T = {};
      T.p = m.master;
      T.m = m.momentum;
      T.g = m.grad_bf16;
      T.w = static_cast<uint16_t*>(m.weight_bf16);
      r = m.rows;
      c = m.cols;
      T.rate = static_cast<float>(static_cast<double>(lr) * static_cast<double>(update_rms) *
                                  std::sqrt(static_cast<double>(std::max(r, c))));
    };
    return muon_call<fp8t::muon::kMuon>("fused_muon_multi_tensor", n_tensors, steps, t, d_workspace, workspace_bytes, as_stream(stream), get);
  });
}

// ------------------------------------------------------------------ scale update
fp8t_status fp8_scale_update(int32_t n_tensors, float* d_amax, float* d_amax_history,
                             int32_t history_len, const float* d_fp8_max, fp8t_amax_algo algo,
                             int32_t margin, float* d_scale, float* d_scale_inv, void* stream) {
  t_last_error.clear();
  if (!d_amax || !d_amax_history || !d_fp8_max || !d_scale || !d_scale_inv)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_scale_update: NULL pointer");
  if (n_tensors < 1 || n_tensors > 65535 || history_len < 1 || history_len > 65536)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_scale_update: n_tensors in 1..65535, history_len in 1..65536");
  if (algo != FP8T_AMAX_MAX && algo != FP8T_AMAX_MOST_RECENT)
    return fail(FP8T_ERR_INVALID_ARG, "fp8_scale_update: unknown amax algorithm %d", (int)algo);
  if (margin < 0 || margin > 126) return fail(FP8T_ERR_INVALID_ARG, "fp8_scale_update: margin in 0..126");
  if (!aligned(d_amax, 4) || !aligned(d_amax_history, 4) || !aligned(d_fp8_max, 4) ||
      !aligned(d_scale, 4) || !aligned(d_scale_inv, 4))
    return fail(FP8T_ERR_MISALIGNED, "fp8_scale_update: misaligned pointer");
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  fp8t::scale::k_scale_update<<<n_tensors, fp8t::scale::kThreads, 0, as_stream(stream)>>>(
      d_amax, d_amax_history, history_len, d_fp8_max, algo == FP8T_AMAX_MAX ? 1 : 0, margin,
      d_scale, d_scale_inv);
  return after_launch("fp8_scale_update launch");
}

// ------------------------------------------------------------------ fused AdamW
size_t fused_adamw_workspace_bytes(const fp8t_adamw_tensor* tensors, int32_t n_tensors) {
  if (!tensors || n_tensors < 1 || n_tensors > (1 << 20)) return 0;
  for (int32_t i = 0; i < n_tensors; ++i)
    if (tensors[i].numel <= 0) return 0;
  return workspace_for(plan_adamw(tensors, n_tensors));
}

}  // extern "C"

namespace {

// The AdamW call; with d_presummed the norm pass is skipped and its sum of squares read there.
fp8t_status adamw_call(const fp8t_adamw_tensor* tensors, const fp8t_adamw_cast* casts,
                       int32_t n_tensors, float lr, float beta1,
                       float beta2, float eps, float weight_decay, int64_t step,
                       int64_t* d_step_inout, float loss_scale, float max_grad_norm,
                       float* d_grad_norm_out, int32_t* d_skipped_out, void* d_workspace,
                       size_t workspace_bytes, const double* d_presummed, unsigned int* d_ticket,
                       void* stream) {
  t_last_error.clear();
  if (!tensors || n_tensors < 1 || n_tensors > (1 << 20))
    return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor: tensors NULL or n_tensors out of range");
  for (int32_t i = 0; i < n_tensors; ++i) {
    const fp8t_adamw_tensor& t = tensors[i];
    if (!t.master || !t.m || !t.v || !t.grad_bf16 || !t.weight_bf16 || t.numel <= 0)
      return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor: tensor %d has a NULL pointer or numel <= 0", i);
    if (!aligned(t.master, 16) || !aligned(t.m, 16) || !aligned(t.v, 16) ||
        !aligned(t.grad_bf16, 16) || !aligned(t.weight_bf16, 16))
      return fail(FP8T_ERR_MISALIGNED, "fused_adamw_multi_tensor: tensor %d is not 16-byte aligned", i);
  }
  if (casts) {
    for (int32_t i = 0; i < n_tensors; ++i) {
      const fp8t_adamw_cast& c = casts[i];
      if (c.rows == 0 && c.cols == 0) continue;                     // no cast for this tensor
      if (c.rows <= 0 || c.cols <= 0 || c.rows % 16 || c.cols % 16 || c.rows >= (int64_t(1) << 31) ||
          c.cols >= (int64_t(1) << 31) || c.rows * c.cols != tensors[i].numel)
        return fail(FP8T_ERR_UNSUPPORTED_SHAPE,
                    "fused_adamw_multi_tensor_presummed: cast %d: rows x cols must equal numel, multiples of 16", i);
      if (c.fmt != FP8T_E4M3 && c.fmt != FP8T_E5M2)
        return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor_presummed: cast %d: unknown format", i);
      if (!c.d_scale || !c.d_amax_inout)
        return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor_presummed: cast %d: NULL scale or amax", i);
      if (!aligned(c.d_scale, 4) || !aligned(c.d_amax_inout, 4) || !aligned(c.d_scale_inv_out, 4) ||
          !aligned(c.q_rowmajor, 16))
        return fail(FP8T_ERR_MISALIGNED, "fused_adamw_multi_tensor_presummed: cast %d: misaligned pointer", i);
    }
  }
  if (!d_step_inout && step < 1)
    return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor: step must be >= 1");
  if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale) || !std::isfinite(lr) ||
      !std::isfinite(beta1) || !std::isfinite(beta2) || !std::isfinite(eps) ||
      !std::isfinite(weight_decay) || !std::isfinite(max_grad_norm))
    return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor: non-finite hyperparameter or loss_scale <= 0");
  if (!aligned(d_grad_norm_out, 4) || !aligned(d_skipped_out, 4) || !aligned(d_workspace, 16) ||
      !aligned(d_step_inout, 8))
    return fail(FP8T_ERR_MISALIGNED, "fused_adamw_multi_tensor: misaligned output or workspace");
  const AdamWPlan plan = plan_adamw(tensors, n_tensors);
  const size_t need = workspace_for(plan);
  if (d_presummed) {
    if (!aligned(d_presummed, 8))
      return fail(FP8T_ERR_MISALIGNED, "fused_adamw_multi_tensor_presummed: misaligned sum of squares");
    if (d_step_inout && (!d_ticket || !aligned(d_ticket, 4)))
      return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor_presummed: a device step counter needs a ticket");
  } else if (!d_workspace || workspace_bytes < need) {
    return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor: workspace of %zu bytes needed", need);
  }
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;

  using namespace fp8t::adamw;
  Scalars k;
  k.beta1 = beta1;
  k.beta2 = beta2;
  k.omb1 = static_cast<float>(1.0 - static_cast<double>(beta1));
  k.omb2 = static_cast<float>(1.0 - static_cast<double>(beta2));
  k.decay = static_cast<float>(1.0 - static_cast<double>(lr) * static_cast<double>(weight_decay));
  k.d_step = d_step_inout;
  k.step_slot = d_presummed ? nullptr
                            : reinterpret_cast<const int64_t*>(static_cast<double*>(d_workspace) + plan.nparts);
  k.step_ticket = d_ticket;
  k.lr_d = lr;
  k.beta1_d = beta1;
  k.beta2_d = beta2;
  if (!d_step_inout) {
    k.step_size = static_cast<float>(static_cast<double>(lr) /
                                     (1.0 - std::pow(static_cast<double>(beta1), static_cast<double>(step))));
    k.bc2_sqrt = static_cast<float>(std::sqrt(1.0 - std::pow(static_cast<double>(beta2), static_cast<double>(step))));
  } else {
    k.step_size = 0.0f;      // formed on the device from the counter
    k.bc2_sqrt = 0.0f;
  }
  k.eps = eps;
  k.inv_s_d = 1.0 / static_cast<double>(loss_scale);
  k.inv_s = static_cast<float>(k.inv_s_d);
  k.max_norm = max_grad_norm;

  cudaStream_t s = as_stream(stream);
  double* partials = static_cast<double*>(d_workspace);
  static thread_local Batch batch;   // ~17 KB: kept off the stack
  // a batch ends at kMaxTensors tensors or kMaxCasts casts
  auto has_cast = [&](int32_t i) { return casts && casts[i].rows > 0; };
  auto batch_end = [&](int32_t b0) {
    int32_t b1 = b0, nc = 0;
    while (b1 < n_tensors && b1 - b0 < kMaxTensors) {
      if (has_cast(b1)) {
        if (nc == kMaxCasts) break;
        ++nc;
      }
      ++b1;
    }
    return b1;
  };
  int64_t off = 0;
  for (int pass = d_presummed ? 1 : 0; pass < 2; ++pass) {
    off = 0;
    for (int32_t b0 = 0, bi = 0, b1 = 0; b0 < n_tensors; b0 = b1, ++bi) {
      b1 = batch_end(b0);
      batch.n = b1 - b0;
      batch.first = bi == 0 ? 1 : 0;
      batch.last = b1 == n_tensors ? 1 : 0;
      int64_t acc = 0;
      int32_t nc = 0;
      for (int32_t i = b0; i < b1; ++i) {
        const int j = i - b0;
        batch.chunk_start[j] = acc;
        batch.cast_of[j] = -1;
        if (has_cast(i)) {
          const fp8t_adamw_cast& c = casts[i];
          CastInfo& ci = batch.cast[nc];
          ci.scale = c.d_scale;
          ci.amax_bits = reinterpret_cast<unsigned int*>(c.d_amax_inout);
          ci.scale_inv = c.d_scale_inv_out;
          ci.q = static_cast<uint8_t*>(c.q_rowmajor);
          ci.fmt = c.fmt;
          batch.cast_of[j] = static_cast<int8_t>(nc++);
        }
        acc += chunks_of(tensors[i].numel);
        batch.numel[j] = tensors[i].numel;
        batch.master[j] = tensors[i].master;
        batch.m[j] = tensors[i].m;
        batch.v[j] = tensors[i].v;
        batch.g[j] = static_cast<const uint16_t*>(tensors[i].grad_bf16);
        batch.w[j] = static_cast<uint16_t*>(tensors[i].weight_bf16);
      }
      batch.chunk_start[batch.n] = acc;
      if (pass == 0) {
        const int64_t grid = std::min<int64_t>(acc, kSumsqBlocks);
        k_adamw_sumsq<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(
            batch, partials + off, bi == 0 ? d_step_inout : nullptr,
            reinterpret_cast<int64_t*>(partials + plan.nparts));
        off += grid;
        if ((st = after_launch("adamw norm pass launch")) != FP8T_OK) return st;
      } else {
        const double* parts = d_presummed ? d_presummed : partials;
        const int np = d_presummed ? 1 : static_cast<int>(plan.nparts);
        if (nc) {
          const int64_t grid = std::min<int64_t>(acc, static_cast<int64_t>(dev->sms) * dev->adamw_cast_blocks_per_sm);
          k_adamw_update<true><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(
              batch, k, parts, np, d_grad_norm_out, d_skipped_out);
        } else {
          const int64_t grid = std::min<int64_t>(acc, static_cast<int64_t>(dev->sms) * dev->adamw_blocks_per_sm);
          k_adamw_update<false><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(
              batch, k, parts, np, d_grad_norm_out, d_skipped_out);
        }
        if ((st = after_launch("adamw update launch")) != FP8T_OK) return st;
      }
    }
  }
  return FP8T_OK;
}

}  // namespace

extern "C" {

fp8t_status fused_adamw_multi_tensor(const fp8t_adamw_tensor* tensors, int32_t n_tensors, float lr,
                                     float beta1, float beta2, float eps, float weight_decay,
                                     int64_t step, int64_t* d_step_inout, float loss_scale,
                                     float max_grad_norm, float* d_grad_norm_out,
                                     int32_t* d_skipped_out, void* d_workspace,
                                     size_t workspace_bytes, void* stream) {
  return adamw_call(tensors, nullptr, n_tensors, lr, beta1, beta2, eps, weight_decay, step,
                    d_step_inout, loss_scale, max_grad_norm, d_grad_norm_out, d_skipped_out,
                    d_workspace, workspace_bytes, nullptr, nullptr, stream);
}

fp8t_status fused_adamw_multi_tensor_presummed(const fp8t_adamw_tensor* tensors,
                                               const fp8t_adamw_cast* casts, int32_t n_tensors,
                                               float lr, float beta1, float beta2, float eps,
                                               float weight_decay, int64_t step,
                                               int64_t* d_step_inout, float loss_scale,
                                               float max_grad_norm, const double* d_grad_sumsq,
                                               float* d_grad_norm_out, int32_t* d_skipped_out,
                                               unsigned int* d_ticket, void* stream) {
  if (!d_grad_sumsq) {
    t_last_error.clear();
    return fail(FP8T_ERR_INVALID_ARG, "fused_adamw_multi_tensor_presummed: d_grad_sumsq NULL");
  }
  return adamw_call(tensors, casts, n_tensors, lr, beta1, beta2, eps, weight_decay, step,
                    d_step_inout, loss_scale, max_grad_norm, d_grad_norm_out, d_skipped_out,
                    nullptr, 0, d_grad_sumsq, d_ticket, stream);
}

// Same step as fused_adamw_multi_tensor, with the built-in scratch array as its workspace.
fp8t_status fused_adamw_multi_tensor_noalloc(const fp8t_adamw_tensor* tensors, int32_t n_tensors,
                                             float lr, float beta1, float beta2, float eps,
                                             float weight_decay, int64_t step,
                                             int64_t* d_step_inout, float loss_scale,
                                             float max_grad_norm, float* d_grad_norm_out,
                                             int32_t* d_skipped_out, void* stream) {
  t_last_error.clear();
  const size_t need = fused_adamw_workspace_bytes(tensors, n_tensors);
  if (need == 0)   // invalid tensor table: the regular entry point reports it, launching nothing
    return fused_adamw_multi_tensor(tensors, n_tensors, lr, beta1, beta2, eps, weight_decay, step,
                                    d_step_inout, loss_scale, max_grad_norm, d_grad_norm_out,
                                    d_skipped_out, nullptr, 0, stream);
  if (need > FP8T_NOALLOC_SCRATCH_BYTES)
    return fail(FP8T_ERR_UNSUPPORTED_SHAPE,
                "fused_adamw_multi_tensor_noalloc: needs %zu bytes of scratch, the built-in array "
                "holds %d; split the tensors over several calls or use fused_adamw_multi_tensor",
                need, FP8T_NOALLOC_SCRATCH_BYTES);
  DeviceInfo* dev = nullptr;
  fp8t_status st = current_device(&dev);
  if (st != FP8T_OK) return st;
  void* scratch = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (!dev->noalloc_scratch) {       // once per device, with that device current
      void* p = nullptr;
      cudaError_t e = cudaGetSymbolAddress(&p, g_adamw_noalloc_scratch);
      if (e != cudaSuccess || !p)
        return fail(FP8T_ERR_CUDA, "cudaGetSymbolAddress(noalloc scratch): %s", cudaGetErrorString(e));
      dev->noalloc_scratch = p;
    }
    scratch = dev->noalloc_scratch;
  }
  return fused_adamw_multi_tensor(tensors, n_tensors, lr, beta1, beta2, eps, weight_decay, step,
                                  d_step_inout, loss_scale, max_grad_norm, d_grad_norm_out,
                                  d_skipped_out, scratch, FP8T_NOALLOC_SCRATCH_BYTES, stream);
}

// ------------------------------------------------------------------ device error word
fp8t_status fp8t_check_device_error(void* stream) {
  t_last_error.clear();
  cudaError_t e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return fail(FP8T_ERR_CUDA, "stream: %s", cudaGetErrorString(e));
  unsigned int word = 0;
  e = cudaMemcpyFromSymbol(&word, fp8t::g_error_word, sizeof(word));
  if (e != cudaSuccess) return fail(FP8T_ERR_CUDA, "reading the error word: %s", cudaGetErrorString(e));
  if (word) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(fp8t::g_error_word, &zero, sizeof(zero));
    if (e != cudaSuccess) return fail(FP8T_ERR_CUDA, "clearing the error word: %s", cudaGetErrorString(e));
    if (word & fp8t::kErrTimeout) return fail(FP8T_ERR_TIMEOUT, "a bounded wait in a kernel expired");
  }
  return FP8T_OK;
}

fp8t_status fp8t_debug_expire_waits(int32_t mode) {
  t_last_error.clear();
  if (mode < 0 || mode > 2) return fail(FP8T_ERR_INVALID_ARG, "fp8t_debug_expire_waits: mode in 0..2");
  cudaError_t e = cudaMemcpyToSymbol(fp8t::g_expire_waits, &mode, sizeof(mode));
  if (e != cudaSuccess) return fail(FP8T_ERR_CUDA, "setting the test hook: %s", cudaGetErrorString(e));
  return FP8T_OK;
}

fp8t_status fp8t_set_wait_timeout_ns(uint64_t ns) {
  t_last_error.clear();
  const unsigned long long v = ns;
  cudaError_t e = cudaMemcpyToSymbol(fp8t::g_wait_timeout_ns, &v, sizeof(v));
  if (e != cudaSuccess) return fail(FP8T_ERR_CUDA, "setting the wait limit: %s", cudaGetErrorString(e));
  return FP8T_OK;
}

}  // extern "C"
