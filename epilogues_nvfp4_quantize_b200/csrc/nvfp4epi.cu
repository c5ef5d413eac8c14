// C-ABI entry points of libnvfp4epi: argument validation, tensor-map encoding and
// kernel launches. All device code is in the included headers, built as one
// translation unit for sm_100a.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "nvfp4epi.h"
#include "ptx.cuh"
#include "codec.cuh"
#include "quantize.cuh"
#include "unfused.cuh"
#include "gemm.cuh"
#include "gemv.cuh"
#include "residual_norm.cuh"
#include "rope.cuh"

#define NVFP4_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per wait
constexpr int kMaxDevices = 64;

std::atomic<int64_t> g_launches{0};
constexpr int kEpiKinds = nvfp4::EPI_REDUCE + 1;

struct DeviceInfo {
  bool probed = false;
  bool supported = false;
  int sm_count = 0;
  // per kernel instance: index epilogue kind + kEpiKinds * (MXFP4 scales)
  bool gemm_attr_set[2 * kEpiKinds] = {};
  bool pair_attr_set[2 * kEpiKinds] = {};
  int pair_clusters[2 * kEpiKinds] = {};
  // resident CTAs of quantize_rows_kernel<V8 = false>, <V8 = true>, quantize_flat_kernel<Y =
  // false>, <Y = true>
  int quant_ctas_per_sm[4] = {0, 0, 0, 0};
  int mx_ctas_per_sm[2] = {0, 0};  // resident CTAs of mx_quantize_kernel<V8 = false, true>
  // clusters of gemv_nvfp4_kernel that fit at once, by log2 of the cluster size (all instances take
  // one CTA per SM)
  int gemv_clusters[4] = {};
  bool gemv_attr_set[24] = {};     // gemv_nvfp4_kernel, by NT, PAIR and SILU
  int norm_regs[8] = {};             // registers of residual_norm_ring_kernel, by stream type, NV and POST
  bool norm_grad_attr_set[8] = {};   // residual_norm_grad_kernel, by stream type, POST and CLUSTER
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_mutex;

nvfp4_status current_device(int* dev_out, DeviceInfo** info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return NVFP4_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceInfo& d = g_dev[dev];
  if (!d.probed) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    d.supported = (major == 10 && minor == 0);
    d.sm_count = sms;
    d.probed = true;
  }
  if (!d.supported) return NVFP4_ERR_UNSUPPORTED_DEVICE;
  *dev_out = dev;
  *info = &d;
  return NVFP4_OK;
}

nvfp4_status launch_status() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The GEMM kernels split their registers between warpgroups at run time (setmaxnreg): the
// epilogue warpgroups can only grow if the block was launched with enough registers for
// the whole split, otherwise they would wait forever. Checked once per kernel, before its
// first launch.
template <class Kernel>
bool register_split_fits(Kernel kern) {
  using namespace nvfp4::gemm_cfg;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return false;
  const long long launched = static_cast<long long>(fa.numRegs) * NUM_THREADS;
  const long long needed = static_cast<long long>(EPI_THREADS) * EPI_REGS + 32ll * ROLE_WARPS * ROLE_REGS;
  return launched >= needed;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool make_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                 uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_stride_bytes};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

nvfp4_status check_operand(const nvfp4_tensor& t) {
  if (t.codes == nullptr || t.sf == nullptr || t.gscale == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (t.rows <= 0 || t.cols <= 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(t.codes) || !aligned16(t.sf)) return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// Common checks and launch of the GEMM kernels: the CTA-pair kernel from M = 256 on (for
// M % 256 == 128 its last tile's second CTA computes rows past M, which are zeros and are
// not stored), the single-CTA kernel for M = 128.
template <int EPI, bool MX = false>
nvfp4_status run_gemm(const nvfp4_tensor& A, const nvfp4_tensor& B, void* D, int64_t ldd, int64_t n_out,
                      nvfp4::GemmArgs args, cudaStream_t stream) {
  using namespace nvfp4::gemm_cfg;
  nvfp4_status st;
  if ((st = check_operand(A)) != NVFP4_OK) return st;
  if ((st = check_operand(B)) != NVFP4_OK) return st;
  const int64_t M = A.rows, K = A.cols, N = B.rows;
  if (B.cols != K) return NVFP4_ERR_INVALID_ARG;
  if (M % BM || N % BN || K % BK) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (M > (1ll << 30) || N > (1ll << 30) || K > (1ll << 30)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int out_kind = EPI == nvfp4::EPI_POINTWISE ? args.out_kind : nvfp4::OUT_BF16;
  const int esize = out_kind == nvfp4::OUT_F32 ? 4 : 2;
  if (D != nullptr) {
    if (ldd < n_out) return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(D) || (ldd * esize) % 16 != 0) return NVFP4_ERR_MISALIGNED;
  }
  int dev;
  DeviceInfo* info;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;

  const bool pair = M > BM;
  CUtensorMap tmA, tmB, tmD, tmSFA, tmSFB;
  std::memset(&tmD, 0, sizeof(tmD));
  if (!make_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, A.codes, K / 2, M, K / 2, BK_BYTES, BM,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, B.codes, K / 2, N, K / 2, BK_BYTES, pair ? 128 : BN,
                   CU_TENSOR_MAP_SWIZZLE_128B))
    return NVFP4_ERR_CUDA;
  if (pair) {
    // the block scales seen as rows of 256 bytes; one 128-row x 256-K group = 8 rows
    // (NVFP4, a scale per 16 values) or 4 rows (MXFP4, a scale per 32)
    const int64_t per_scale = MX ? 32 : 16;
    const uint32_t box_rows = MX ? 4 : 8;
    if (!make_map_2d(&tmSFA, CU_TENSOR_MAP_DATA_TYPE_UINT8, A.sf, 256, M * (K / per_scale) / 256, 256, 256, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_NONE) ||
        !make_map_2d(&tmSFB, CU_TENSOR_MAP_DATA_TYPE_UINT8, B.sf, 256, N * (K / per_scale) / 256, 256, 256, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_NONE))
      return NVFP4_ERR_CUDA;
  }
  // D staged by 32 rows x 128 bytes and stored by TMA: 64 columns of bf16/f16 or 32 of f32
  const CUtensorMapDataType d_type = out_kind == nvfp4::OUT_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : out_kind == nvfp4::OUT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (D != nullptr && !make_map_2d(&tmD, d_type, D, n_out, M, ldd * esize, 128 / esize, 32,
                                   CU_TENSOR_MAP_SWIZZLE_128B))
    return NVFP4_ERR_CUDA;

  args.sfa = static_cast<const uint8_t*>(A.sf);
  args.sfb = static_cast<const uint8_t*>(B.sf);
  args.ga = A.gscale;
  args.gb = B.gscale;
  args.M = static_cast<int>(M);
  args.N = static_cast<int>(N);
  args.K = static_cast<int>(K);
  args.tiles_m = static_cast<int>(pair ? (M + 255) / 256 : M / BM);
  args.tiles_n = static_cast<int>(N / BN);
  args.num_tiles = args.tiles_m * args.tiles_n;
  // keep the smaller operand resident in L2 while the larger one streams through once
  args.n_fastest = N <= M ? 1 : 0;
  args.write_d = D != nullptr;
  args.wait_limit_ns = kWaitLimitNs;

  if (!pair) {
    using P = nvfp4::PlanSingleT<MX>;
    auto kern = nvfp4::gemm_nvfp4_kernel<EPI, MX>;
    {
      std::lock_guard<std::mutex> lock(g_mutex);
      if (!info->gemm_attr_set[EPI + kEpiKinds * MX]) {
        if (!register_split_fits(kern)) return NVFP4_ERR_CUDA;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM_BYTES) != cudaSuccess)
          return NVFP4_ERR_CUDA;
        info->gemm_attr_set[EPI + kEpiKinds * MX] = true;
      }
    }
    const int grid = args.num_tiles < info->sm_count ? args.num_tiles : info->sm_count;
    kern<<<grid, NUM_THREADS, P::SMEM_BYTES, stream>>>(tmA, tmB, tmD, args);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return launch_status();
  }

  using P = nvfp4::PlanPairT<MX>;
  auto kern = nvfp4::gemm_nvfp4_pair_kernel<EPI, MX>;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = P::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int max_clusters;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!info->pair_attr_set[EPI + kEpiKinds * MX]) {
      if (!register_split_fits(kern)) return NVFP4_ERR_CUDA;
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM_BYTES) != cudaSuccess)
        return NVFP4_ERR_CUDA;
      cfg.gridDim = dim3(2 * (info->sm_count / 2), 1, 1);
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return NVFP4_ERR_CUDA;
      info->pair_clusters[EPI + kEpiKinds * MX] = n;
      info->pair_attr_set[EPI + kEpiKinds * MX] = true;
    }
    max_clusters = info->pair_clusters[EPI + kEpiKinds * MX];
  }
  const int clusters = args.num_tiles < max_clusters ? args.num_tiles : max_clusters;
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  if (cudaLaunchKernelEx(&cfg, kern, tmA, tmB, tmSFA, tmSFB, tmD, args) != cudaSuccess) return NVFP4_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

}  // namespace

// Launch of the two-kernel quantiser (quantize.cuh) for nvfp4_quantize and
// nvfp4_fake_quantize: with compute_amax, the amax partials kernel then the quantise kernel
// (programmatic dependent launch); with a static scale, the quantise kernel alone.
static nvfp4_status launch_quantize2(DeviceInfo* info, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                                     int compute_amax, bool inter, float* gscale, uint8_t* codes, uint8_t* sf,
                                     uint16_t* y, int64_t ldy, void* workspace, cudaStream_t stream) {
  using namespace nvfp4::q2cfg;
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  // 256-bit accesses need every row of x (and of y) to start on a 32-byte boundary
  const bool x_v8 = (reinterpret_cast<uintptr_t>(x) & 31u) == 0 && (ldx % 16) == 0;
  const bool y_v8 = y == nullptr || ((reinterpret_cast<uintptr_t>(y) & 31u) == 0 && (ldy % 16) == 0);
  nvfp4::Quant2Args qa{};
  qa.x = xp;
  qa.rows = rows;
  qa.cols = cols;
  qa.ldx = ldx;
  qa.interleave = inter ? 1 : 0;
  qa.gscale = gscale;
  qa.codes = codes;
  qa.sf = sf;
  qa.y = y;
  qa.ldy = ldy;
  if (compute_amax) {
    const int64_t chunks = rows * (cols / 16);
    int64_t parts = (chunks + 4 * AMAX_THREADS - 1) / (4 * AMAX_THREADS);
    const int64_t cap = 2ll * info->sm_count < MAX_PARTIALS ? 2ll * info->sm_count : MAX_PARTIALS;
    if (parts > cap) parts = cap;
    if (parts < 1) parts = 1;
    float* partials = static_cast<float*>(workspace);
    const dim3 grid(static_cast<unsigned>(parts));
    if (ldx == cols && x_v8) {
      nvfp4::amax_partial_kernel<true, true><<<grid, AMAX_THREADS, 0, stream>>>(xp, rows, cols, ldx, partials);
    } else if (ldx == cols) {
      nvfp4::amax_partial_kernel<true, false><<<grid, AMAX_THREADS, 0, stream>>>(xp, rows, cols, ldx, partials);
    } else if (x_v8) {
      nvfp4::amax_partial_kernel<false, true><<<grid, AMAX_THREADS, 0, stream>>>(xp, rows, cols, ldx, partials);
    } else {
      nvfp4::amax_partial_kernel<false, false><<<grid, AMAX_THREADS, 0, stream>>>(xp, rows, cols, ldx, partials);
    }
    g_launches.fetch_add(1, std::memory_order_relaxed);
    nvfp4_status st;
    if ((st = launch_status()) != NVFP4_OK) return st;
    qa.partials = partials;
    qa.nparts = static_cast<int>(parts);
  }
  const bool v8 = x_v8 && y_v8;
  // the flat kernel: x (and y) contiguous and 32-byte aligned, no interleave
  const bool flat = v8 && !inter && ldx == cols && (y == nullptr || ldy == cols);
  const int kind = flat ? (y != nullptr ? 3 : 2) : (v8 ? 1 : 0);
  {
    // CTAs that fit on an SM at once: the kernel's warps stride over the whole tensor, so a
    // grid larger than one wave would only queue CTAs behind it
    std::lock_guard<std::mutex> lock(g_mutex);
    int& per_sm = info->quant_ctas_per_sm[kind];
    if (per_sm == 0) {
      int n = 0;
      const cudaError_t e =
          kind == 3   ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4::quantize_flat_kernel<true>,
                                                                      QUANT_THREADS, 0)
          : kind == 2 ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4::quantize_flat_kernel<false>,
                                                                      QUANT_THREADS, 0)
          : kind == 1
              ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4::quantize_rows_kernel<true>, QUANT_THREADS, 0)
              : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4::quantize_rows_kernel<false>, QUANT_THREADS, 0);
      if (e != cudaSuccess || n < 1) return NVFP4_ERR_CUDA;
      per_sm = n;
    }
  }
  const int64_t rows_pad = (rows + 127) / 128 * 128;
  // warp tasks: 128 blocks of 16 (flat), or 512 columns of one row (row kernel)
  const int64_t tasks = flat ? (rows * (cols / 16) + 127) / 128 : rows_pad * ((cols / 64 + 7) / 8);
  int64_t grid = (tasks + QUANT_WARPS - 1) / QUANT_WARPS;
  const int64_t full = static_cast<int64_t>(info->quant_ctas_per_sm[kind]) * info->sm_count;
  if (grid > full) grid = full;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(QUANT_THREADS, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = kind == 3   ? cudaLaunchKernelEx(&cfg, nvfp4::quantize_flat_kernel<true>, qa)
                        : kind == 2 ? cudaLaunchKernelEx(&cfg, nvfp4::quantize_flat_kernel<false>, qa)
                        : kind == 1 ? cudaLaunchKernelEx(&cfg, nvfp4::quantize_rows_kernel<true>, qa)
                                    : cudaLaunchKernelEx(&cfg, nvfp4::quantize_rows_kernel<false>, qa);
  if (e != cudaSuccess) return NVFP4_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

NVFP4_API int64_t nvfp4_sf_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return -1;
  return ((rows + 127) / 128) * 128 * ((cols / 16 + 3) / 4) * 4;
}

NVFP4_API int64_t nvfp4_quantize_workspace_bytes(void) {
  return nvfp4::q2cfg::MAX_PARTIALS * static_cast<int64_t>(sizeof(float));
}

NVFP4_API nvfp4_status nvfp4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx, int compute_amax,
                                      int flags, nvfp4_tensor out, void* workspace, cudaStream_t stream) {
  if (x == nullptr || out.codes == nullptr || out.sf == nullptr || out.gscale == nullptr)
    return NVFP4_ERR_INVALID_ARG;
  if (compute_amax != 0 && compute_amax != 1) return NVFP4_ERR_INVALID_ARG;
  if (compute_amax && workspace == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (flags & ~NVFP4_SWIGLU_INTERLEAVE) return NVFP4_ERR_INVALID_ARG;
  if (out.rows != rows || out.cols != cols) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || cols <= 0 || cols % 64 != 0 || ldx < cols) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if ((flags & NVFP4_SWIGLU_INTERLEAVE) && (rows % 2) != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (rows > (1ll << 31) || cols > (1ll << 31)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || (ldx % 8) != 0 || !aligned16(out.codes) ||
      (reinterpret_cast<uintptr_t>(out.sf) & 3u) != 0 ||
      (compute_amax && (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0))
    return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;

  return launch_quantize2(info, x, rows, cols, ldx, compute_amax, (flags & NVFP4_SWIGLU_INTERLEAVE) != 0,
                          out.gscale, static_cast<uint8_t*>(out.codes), static_cast<uint8_t*>(out.sf), nullptr, 0,
                          workspace, stream);
}

NVFP4_API nvfp4_status nvfp4_fake_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx, int compute_amax,
                                           float* gscale, void* y, int64_t ldy, void* workspace,
                                           cudaStream_t stream) {
  if (x == nullptr || y == nullptr || gscale == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (compute_amax != 0 && compute_amax != 1) return NVFP4_ERR_INVALID_ARG;
  if (compute_amax && workspace == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || cols <= 0 || cols % 64 != 0 || ldx < cols || ldy < cols) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (rows > (1ll << 31) || cols > (1ll << 31)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || (ldx % 8) != 0 || !aligned16(y) || (ldy % 8) != 0 ||
      (reinterpret_cast<uintptr_t>(gscale) & 3u) != 0 ||
      (compute_amax && (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0))
    return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  return launch_quantize2(info, x, rows, cols, ldx, compute_amax, false, gscale, nullptr, nullptr,
                          static_cast<uint16_t*>(y), ldy, workspace, stream);
}

NVFP4_API nvfp4_status gemm_nvfp4_plain(nvfp4_tensor A, nvfp4_tensor B, void* D, int64_t ldd,
                                        cudaStream_t stream) {
  if (D == nullptr) return NVFP4_ERR_INVALID_ARG;
  nvfp4::GemmArgs args{};
  return run_gemm<nvfp4::EPI_PLAIN>(A, B, D, ldd, B.rows, args, stream);
}

NVFP4_API nvfp4_status gemm_nvfp4_pointwise(nvfp4_tensor A, nvfp4_tensor B, const float* bias, int act,
                                            int out_dtype, void* D, int64_t ldd, const nvfp4_tensor* Dq,
                                            cudaStream_t stream) {
  if (D == nullptr && Dq == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_RELU) return NVFP4_ERR_INVALID_ARG;
  if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_F16 && out_dtype != NVFP4_OUT_F32)
    return NVFP4_ERR_INVALID_ARG;
  if (bias != nullptr && !aligned16(bias)) return NVFP4_ERR_MISALIGNED;
  nvfp4::GemmArgs args{};
  args.bias = bias;
  args.act = act;
  args.out_kind = out_dtype;
  if (Dq != nullptr) {
    if (Dq->codes == nullptr || Dq->sf == nullptr || Dq->gscale == nullptr) return NVFP4_ERR_INVALID_ARG;
    if (Dq->rows != A.rows || Dq->cols != B.rows) return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(Dq->codes) || !aligned16(Dq->sf)) return NVFP4_ERR_MISALIGNED;
    args.q_codes = static_cast<uint8_t*>(Dq->codes);
    args.q_sf = static_cast<uint8_t*>(Dq->sf);
    args.q_gscale = Dq->gscale;
    args.q_cols = static_cast<int>(B.rows);
  }
  return run_gemm<nvfp4::EPI_POINTWISE>(A, B, D, ldd, B.rows, args, stream);
}

NVFP4_API nvfp4_status gemm_nvfp4_reduce_rows_f32(nvfp4_tensor A, nvfp4_tensor B, float* const* dst, int world,
                                                  int64_t rows_per_rank, int64_t ldd, cudaStream_t stream) {
  if (dst == nullptr || (reinterpret_cast<uintptr_t>(dst) & 7u) != 0) return NVFP4_ERR_INVALID_ARG;
  if (world < 1 || rows_per_rank <= 0) return NVFP4_ERR_INVALID_ARG;
  if (rows_per_rank % 128 != 0 || A.rows != static_cast<int64_t>(world) * rows_per_rank)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ldd < B.rows) return NVFP4_ERR_INVALID_ARG;
  if (ldd % 4 != 0) return NVFP4_ERR_MISALIGNED;
  nvfp4::GemmArgs args{};
  args.red_dst = dst;
  args.red_rows = rows_per_rank;
  args.red_ldd = ldd;
  return run_gemm<nvfp4::EPI_REDUCE>(A, B, nullptr, 0, B.rows, args, stream);
}

NVFP4_API int64_t mxfp4_sf_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return -1;
  return ((rows + 127) / 128) * 128 * ((cols / 32 + 3) / 4) * 4;
}

NVFP4_API nvfp4_status mxfp4_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx, int flags,
                                      nvfp4_tensor out, cudaStream_t stream) {
  if (x == nullptr || out.codes == nullptr || out.sf == nullptr || out.gscale == nullptr)
    return NVFP4_ERR_INVALID_ARG;
  if (flags & ~(MXFP4_HADAMARD32 | NVFP4_SWIGLU_INTERLEAVE)) return NVFP4_ERR_INVALID_ARG;
  if ((flags & NVFP4_SWIGLU_INTERLEAVE) && (rows % 2) != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (out.rows != rows || out.cols != cols) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || cols <= 0 || cols % 128 != 0 || ldx < cols) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (rows > (1ll << 31) || cols > (1ll << 31)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || (ldx % 8) != 0 || !aligned16(out.codes) || (reinterpret_cast<uintptr_t>(out.sf) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(out.gscale) & 3u) != 0)
    return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  // the per-tensor factor a GEMM applies: 1, or 1/sqrt(32) per transformed operand
  // (x H)(w H)^T = 32 x w^T
  const float g = (flags & MXFP4_HADAMARD32) ? 0.17677669529663689f : 1.0f;
  const int64_t rows_pad = (rows + 127) / 128 * 128;
  const int64_t threads = rows_pad * (cols / 32);
  // 256-bit loads when every row of x starts on a 32-byte boundary; one wave of CTAs at the
  // occupancy the runtime reports, walking the blocks with the grid's stride
  const bool v8 = (reinterpret_cast<uintptr_t>(x) & 31u) == 0 && (ldx % 16) == 0;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    int& per_sm = info->mx_ctas_per_sm[v8 ? 1 : 0];
    if (per_sm == 0) {
      int n = 0;
      const cudaError_t e = v8 ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4::mx_quantize_kernel<true>, 256, 0)
                               : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4::mx_quantize_kernel<false>, 256, 0);
      if (e != cudaSuccess || n < 1) return NVFP4_ERR_CUDA;
      per_sm = n;
    }
  }
  int64_t grid = (threads + 255) / 256;
  const int64_t full = static_cast<int64_t>(info->mx_ctas_per_sm[v8 ? 1 : 0]) * info->sm_count;
  if (grid > full) grid = full;
  const int had = (flags & MXFP4_HADAMARD32) ? 1 : 0, inter = (flags & NVFP4_SWIGLU_INTERLEAVE) ? 1 : 0;
  if (v8) {
    nvfp4::mx_quantize_kernel<true><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
        static_cast<const uint16_t*>(x), rows, cols, ldx, had, inter, static_cast<uint8_t*>(out.codes),
        static_cast<uint8_t*>(out.sf), out.gscale, g);
  } else {
    nvfp4::mx_quantize_kernel<false><<<static_cast<unsigned>(grid), 256, 0, stream>>>(
        static_cast<const uint16_t*>(x), rows, cols, ldx, had, inter, static_cast<uint8_t*>(out.codes),
        static_cast<uint8_t*>(out.sf), out.gscale, g);
  }
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

NVFP4_API nvfp4_status gemm_mxfp4_pointwise(nvfp4_tensor A, nvfp4_tensor B, const float* bias, int act,
                                            int out_dtype, void* D, int64_t ldd, cudaStream_t stream) {
  if (D == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_RELU) return NVFP4_ERR_INVALID_ARG;
  if (out_dtype != NVFP4_OUT_BF16 && out_dtype != NVFP4_OUT_F16 && out_dtype != NVFP4_OUT_F32)
    return NVFP4_ERR_INVALID_ARG;
  if (bias != nullptr && !aligned16(bias)) return NVFP4_ERR_MISALIGNED;
  nvfp4::GemmArgs args{};
  args.bias = bias;
  args.act = act;
  args.out_kind = out_dtype;
  return run_gemm<nvfp4::EPI_POINTWISE, true>(A, B, D, ldd, B.rows, args, stream);
}

NVFP4_API nvfp4_status gemm_mxfp4_plain(nvfp4_tensor A, nvfp4_tensor B, void* D, int64_t ldd, cudaStream_t stream) {
  return gemm_mxfp4_pointwise(A, B, nullptr, NVFP4_ACT_NONE, NVFP4_OUT_BF16, D, ldd, stream);
}

template <bool MX>
static nvfp4_status rmsnorm_entry(nvfp4_tensor A, nvfp4_tensor B, const float* w, int head_dim, int64_t n_norm_cols,
                                  float eps, void* D, int64_t ldd, cudaStream_t stream) {
  if (D == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (head_dim != 128 && head_dim != 256) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (n_norm_cols < 0 || n_norm_cols > B.rows || n_norm_cols % head_dim != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (n_norm_cols > 0 && w == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (w != nullptr && !aligned16(w)) return NVFP4_ERR_MISALIGNED;
  if (!(eps >= 0.0f)) return NVFP4_ERR_INVALID_ARG;
  nvfp4::GemmArgs args{};
  args.w = w;
  args.head_dim = head_dim;
  args.n_norm_cols = static_cast<int>(n_norm_cols);
  args.eps = eps;
  return run_gemm<nvfp4::EPI_RMSNORM, MX>(A, B, D, ldd, B.rows, args, stream);
}

NVFP4_API nvfp4_status gemm_nvfp4_rmsnorm(nvfp4_tensor A, nvfp4_tensor B, const float* w, int head_dim,
                                          int64_t n_norm_cols, float eps, void* D, int64_t ldd,
                                          cudaStream_t stream) {
  return rmsnorm_entry<false>(A, B, w, head_dim, n_norm_cols, eps, D, ldd, stream);
}

NVFP4_API nvfp4_status gemm_mxfp4_rmsnorm(nvfp4_tensor A, nvfp4_tensor B, const float* w, int head_dim,
                                          int64_t n_norm_cols, float eps, void* D, int64_t ldd,
                                          cudaStream_t stream) {
  return rmsnorm_entry<true>(A, B, w, head_dim, n_norm_cols, eps, D, ldd, stream);
}

template <bool MX>
static nvfp4_status swiglu_entry(nvfp4_tensor A, nvfp4_tensor B, void* D, int64_t ldd, const nvfp4_tensor* Dq,
                                 cudaStream_t stream) {
  if (D == nullptr && Dq == nullptr) return NVFP4_ERR_INVALID_ARG;
  const int64_t nh = B.rows / 2;
  nvfp4::GemmArgs args{};
  if (Dq != nullptr) {
    if (Dq->codes == nullptr || Dq->sf == nullptr || Dq->gscale == nullptr) return NVFP4_ERR_INVALID_ARG;
    if (Dq->rows != A.rows || Dq->cols != nh) return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(Dq->codes) || !aligned16(Dq->sf)) return NVFP4_ERR_MISALIGNED;
    args.q_codes = static_cast<uint8_t*>(Dq->codes);
    args.q_sf = static_cast<uint8_t*>(Dq->sf);
    args.q_gscale = Dq->gscale;
    args.q_cols = static_cast<int>(nh);
  }
  return run_gemm<nvfp4::EPI_SWIGLU, MX>(A, B, D, ldd, nh, args, stream);
}

NVFP4_API nvfp4_status gemm_nvfp4_swiglu(nvfp4_tensor A, nvfp4_tensor B, void* D, int64_t ldd,
                                         const nvfp4_tensor* Dq, cudaStream_t stream) {
  return swiglu_entry<false>(A, B, D, ldd, Dq, stream);
}

NVFP4_API nvfp4_status gemm_mxfp4_swiglu(nvfp4_tensor A, nvfp4_tensor B, void* D, int64_t ldd,
                                         const nvfp4_tensor* Dq, cudaStream_t stream) {
  return swiglu_entry<true>(A, B, D, ldd, Dq, stream);
}

NVFP4_API nvfp4_status rmsnorm_heads_bf16(const void* x, int64_t rows, int64_t ldx, const float* w, int head_dim,
                                          int64_t n_norm_cols, float eps, void* y, int64_t ldy,
                                          cudaStream_t stream) {
  if (x == nullptr || y == nullptr || w == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (head_dim != 128 && head_dim != 256) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (rows <= 0 || n_norm_cols <= 0 || n_norm_cols % head_dim != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ldx < n_norm_cols || ldy < n_norm_cols) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(w) || ldx % 8 || ldy % 8) return NVFP4_ERR_MISALIGNED;
  if (!(eps >= 0.0f)) return NVFP4_ERR_INVALID_ARG;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  const int64_t warps = rows * (n_norm_cols / head_dim);
  const int64_t blocks = (warps * 32 + 255) / 256;
  if (head_dim == 256)
    nvfp4::rmsnorm_heads_kernel<256><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        static_cast<const uint16_t*>(x), rows, ldx, w, n_norm_cols, eps, static_cast<uint16_t*>(y), ldy);
  else
    nvfp4::rmsnorm_heads_kernel<128><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        static_cast<const uint16_t*>(x), rows, ldx, w, n_norm_cols, eps, static_cast<uint16_t*>(y), ldy);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

NVFP4_API nvfp4_status swiglu_bf16(const void* c, int64_t rows, int64_t nh, int64_t ldc, void* y, int64_t ldy,
                                   cudaStream_t stream) {
  if (c == nullptr || y == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || nh <= 0 || nh % 8 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ldc < 2 * nh || ldy < nh) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(c) || !aligned16(y) || ldc % 8 || ldy % 8) return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  const int64_t threads = rows * (nh / 8);
  const int64_t blocks = (threads + 255) / 256;
  nvfp4::swiglu_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
      static_cast<const uint16_t*>(c), rows, nh, ldc, static_cast<uint16_t*>(y), ldy);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

NVFP4_API const char* nvfp4_status_string(nvfp4_status s) {
  switch (s) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case NVFP4_ERR_MISALIGNED: return "misaligned pointer or leading dimension";
    case NVFP4_ERR_UNSUPPORTED_DEVICE: return "unsupported device (needs compute capability 10.0)";
    case NVFP4_ERR_CUDA: return "CUDA error";
    case NVFP4_ERR_DEVICE_TIMEOUT: return "a bounded wait inside a kernel ran out";
  }
  return "unknown status";
}

NVFP4_API int nvfp4_read_device_status(cudaStream_t stream) {
  if (cudaStreamSynchronize(stream) != cudaSuccess) return -1;
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, nvfp4::g_device_status, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyToSymbol(nvfp4::g_device_status, &zero, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

NVFP4_API nvfp4_status nvfp4_selftest_bounded_wait(int64_t limit_ns, cudaStream_t stream) {
  if (limit_ns < 1 || limit_ns > 1000000000ll) return NVFP4_ERR_INVALID_ARG;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  nvfp4::selftest_wait_kernel<<<1, 32, 0, stream>>>(static_cast<uint64_t>(limit_ns));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

NVFP4_API int64_t nvfp4_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

// -------------------------------------------------------------------------------------
// Stream-ordered barrier over peer-mapped signal words (one process per GPU), for the
// row-parallel GEMM whose epilogue adds into the other ranks' output blocks.
// -------------------------------------------------------------------------------------
namespace {

__device__ __forceinline__ void st_release_sys(uint32_t* p, uint32_t v) {
  asm volatile("st.release.sys.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_acquire_sys(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.sys.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Thread q < world publishes `epoch` in slot [rank] of rank q's signal words (after a
// system-scope fence, so everything this GPU wrote before, the previous kernels' additions
// into peer blocks included, is visible to q first), then waits until slot [q] of this
// rank's words has reached `epoch`. A wait that runs past limit_ns records
// NVFP4_ERR_DEVICE_TIMEOUT in the device status word and returns.
__global__ void __launch_bounds__(64) signal_barrier_kernel(uint32_t* const* __restrict__ signals, int world,
                                                            int rank, uint32_t epoch, uint64_t limit_ns) {
  const int q = threadIdx.x;
  if (q < world) {
    __threadfence_system();
    st_release_sys(signals[q] + rank, epoch);
  }
  __syncthreads();
  if (q < world) {
    const uint32_t* mine = signals[rank] + q;
    const uint64_t t0 = nvfp4::globaltimer_ns();
    while (static_cast<int32_t>(ld_acquire_sys(mine) - epoch) < 0) {
      if (nvfp4::globaltimer_ns() - t0 > limit_ns) {
        nvfp4::record_status(NVFP4_ERR_DEVICE_TIMEOUT, 70);
        break;
      }
      __nanosleep(64);
    }
  }
}

}  // namespace

NVFP4_API nvfp4_status nvfp4_signal_barrier(uint32_t* const* signals, int world, int rank, uint32_t epoch,
                                            int64_t limit_ns, cudaStream_t stream) {
  if (signals == nullptr || epoch == 0) return NVFP4_ERR_INVALID_ARG;
  if (world < 1 || world > 64 || rank < 0 || rank >= world) return NVFP4_ERR_INVALID_ARG;
  if (limit_ns < 1 || limit_ns > 60000000000ll) return NVFP4_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(signals) & 7u) != 0) return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  signal_barrier_kernel<<<1, 64, 0, stream>>>(signals, world, rank, epoch, static_cast<uint64_t>(limit_ns));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

// -------------------------------------------------------------------------------------
// Allocation-free quantiser: nvfp4_quantize with compute_amax = 1, whose scratch (one
// partial maximum per block of 16384 input values, then the tensor's amax) lives in a
// file-scope device array instead of a caller workspace.
// -------------------------------------------------------------------------------------
namespace {

constexpr int kNoAllocPartials = 16384;                     // partial maxima the array holds
constexpr int64_t kNoAllocUnitsPerBlock = 256 * 8;          // 16-byte units per partial (16384 values)
constexpr int64_t kNoAllocMaxValues = static_cast<int64_t>(kNoAllocPartials) * kNoAllocUnitsPerBlock * 8;
static_assert(kNoAllocMaxValues == NVFP4_NOALLOC_MAX_VALUES, "limit stated in the header");

// [0, kNoAllocPartials): partial maxima; [kNoAllocPartials]: the tensor's amax (float bits).
// Every GPU that loads the library holds these 64 KB until the process exits.
static __device__ __align__(256) float g_noalloc_scratch[kNoAllocPartials + 64];

float* g_noalloc_ptr[kMaxDevices] = {nullptr};

// One partial maximum of |x| per block: block b covers 16-byte units
// [b * 2048, (b + 1) * 2048) of the row-major rows x cols view. Written, not accumulated.
__global__ void __launch_bounds__(256) noalloc_amax_partial_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                   int64_t cols, int64_t ldx,
                                                                   float* __restrict__ partials) {
  const int64_t upr = cols >> 3;
  const int64_t total = rows * upr;
  const int64_t base = blockIdx.x * kNoAllocUnitsPerBlock;
  float m = 0.0f;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t u = base + i * 256 + threadIdx.x;
    if (u < total) {
      const int64_t r = u / upr, c = u - r * upr;
      v[i] = __ldg(reinterpret_cast<const uint4*>(x + r * ldx + c * 8));
    } else {
      v[i] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu, v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu};
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(nvfp4::bf16_lo(w[k]), nvfp4::bf16_hi(w[k])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  __shared__ float wmax[8];
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    float b = 0.0f;
    for (int i = 0; i < 8; ++i) b = fmaxf(b, wmax[i]);
    partials[blockIdx.x] = b;
  }
}

// Maximum of the n partials, written as float bits to *amax_bits.
__global__ void __launch_bounds__(256) noalloc_amax_reduce_kernel(const float* __restrict__ partials, int n,
                                                                  unsigned int* __restrict__ amax_bits) {
  float m = 0.0f;
  for (int i = threadIdx.x; i < n; i += 256) m = fmaxf(m, partials[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  __shared__ float wmax[8];
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    float b = 0.0f;
    for (int i = 0; i < 8; ++i) b = fmaxf(b, wmax[i]);
    *amax_bits = __float_as_uint(b);
  }
}

// Device address of the scratch array on device `dev` (looked up once per device, with
// that device current).
nvfp4_status noalloc_scratch(int dev, float** out) {
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || p == nullptr) return NVFP4_ERR_CUDA;
    g_noalloc_ptr[dev] = static_cast<float*>(p);
  }
  *out = g_noalloc_ptr[dev];
  return NVFP4_OK;
}

}  // namespace

NVFP4_API nvfp4_status nvfp4_quantize_noalloc(const void* x, int64_t rows, int64_t cols, int64_t ldx, int flags,
                                              nvfp4_tensor out, cudaStream_t stream) {
  if (x == nullptr || out.codes == nullptr || out.sf == nullptr || out.gscale == nullptr)
    return NVFP4_ERR_INVALID_ARG;
  if (flags & ~NVFP4_SWIGLU_INTERLEAVE) return NVFP4_ERR_INVALID_ARG;
  if (out.rows != rows || out.cols != cols) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || cols <= 0 || cols % 64 != 0 || ldx < cols) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if ((flags & NVFP4_SWIGLU_INTERLEAVE) && (rows % 2) != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  // the scratch array holds one partial maximum per 16384 values
  if (rows > kNoAllocMaxValues / cols) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(x) || (ldx % 8) != 0 || !aligned16(out.codes) || (reinterpret_cast<uintptr_t>(out.sf) & 3u) != 0)
    return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  float* scratch;
  if ((st = noalloc_scratch(dev, &scratch)) != NVFP4_OK) return st;

  const uint16_t* xp = static_cast<const uint16_t*>(x);
  const int64_t units = rows * (cols / 8);
  const int blocks = static_cast<int>((units + kNoAllocUnitsPerBlock - 1) / kNoAllocUnitsPerBlock);
  unsigned int* amax_bits = reinterpret_cast<unsigned int*>(scratch + kNoAllocPartials);
  noalloc_amax_partial_kernel<<<blocks, 256, 0, stream>>>(xp, rows, cols, ldx, scratch);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if ((st = launch_status()) != NVFP4_OK) return st;
  noalloc_amax_reduce_kernel<<<1, 256, 0, stream>>>(scratch, blocks, amax_bits);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if ((st = launch_status()) != NVFP4_OK) return st;
  const int64_t rows_pad = (rows + 127) / 128 * 128;
  const int64_t threads = rows_pad * (cols / 64);
  nvfp4::quantize_kernel<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(
      xp, rows, cols, ldx, (flags & NVFP4_SWIGLU_INTERLEAVE) ? 1 : 0, amax_bits, out.gscale,
      static_cast<uint8_t*>(out.codes), static_cast<uint8_t*>(out.sf));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_status();
}

// -------------------------------------------------------------------------------------
// Operators between the GEMMs of a layer: few-row products, residual norm, rotary positions.
// -------------------------------------------------------------------------------------
namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t out_size(int dtype) { return dtype == NVFP4_OUT_F32 ? 4 : 2; }
// Launch with programmatic dependent launch: the kernels of this section let the next kernel start
// launching at once and wait (griddepcontrol.wait) for the previous one before they touch memory, so
// in a run of them the launch of each overlaps the end of the one before.
template <class Args>
nvfp4_status launch_dependent(void (*kern)(Args), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                              const Args& args, int cluster = 1) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, args) != cudaSuccess) {
    (void)cudaGetLastError();
    return NVFP4_ERR_CUDA;
  }
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return NVFP4_OK;
}

bool is_dtype(int d) { return d == NVFP4_OUT_BF16 || d == NVFP4_OUT_F16 || d == NVFP4_OUT_F32; }

// a.tile rows of x per CTA: at most 8 NT, 2 with PAIR, half as many with SILU_ROWS.
template <int NT, int PAIR, int SILU>
nvfp4_status launch_gemv(DeviceInfo* info, nvfp4::GemvArgs a, cudaStream_t stream) {
  using namespace nvfp4::gemvcfg;
  void (*const kerns[2])(nvfp4::GemvArgs) = {nvfp4::gemv_nvfp4_kernel<NT, 4, PAIR, SILU>,
                                             nvfp4::gemv_nvfp4_kernel<NT, 2, PAIR, SILU>};
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  int clusters[4];
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    bool& set = info->gemv_attr_set[NT + 2 * PAIR + 6 * SILU];
    if (!set) {
      for (auto kern : kerns) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM) != cudaSuccess)
          return NVFP4_ERR_CUDA;
      }
      cfg.numAttrs = 2;
      cfg.dynamicSmemBytes = MAX_SMEM;
      for (int i = 0; i < 4; ++i) {
        attr[1].val.clusterDim.x = 1u << i;
        cfg.gridDim = dim3(static_cast<unsigned>(info->sm_count >> i << i), 1, 1);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kerns[0], &cfg) != cudaSuccess || n <= 0) return NVFP4_ERR_CUDA;
        info->gemv_clusters[i] = n;
      }
      set = true;
    }
    std::memcpy(clusters, info->gemv_clusters, sizeof(clusters));
  }
  // How K is cut: over the CTAs of a cluster and over the warps of a CTA. A larger cluster leaves each CTA
  // less of x to copy and to convert, and a shorter start; what it costs is the joins. In hundredths of a
  // step of all warps (0.4 us): the steps of the longest warp, 100 for each join of warps, 75 for each
  // CTA in each join of a cluster, 8 for each 128 columns of a row of x (12 with SiLU). Over 12 shapes of 1 to
  // 16 rows (all 20 cuts of each measured) the cut so chosen is 2.2 % behind the best on average and 16 % at
  // most; with x left out and 400 for any join of a cluster it was 18 and 55 %: 1024 x 1024 takes one CTA and 8 warps, the
  // others mostly 4 CTAs (2 x 4096 x 6144: 6.7 us against 9.0 in one CTA each, 8 x 4096 x 12288: 12.5 against
  // 17.1). Four chunks of weights in flight per warp where they fit beside x, else two.
  const int groups = static_cast<int>((a.K + GROUP - 1) / GROUP);
  const int tokens = static_cast<int>(a.M < a.tile ? a.M : a.tile);
  auto smem = [&](int buffers, int kslice, int cluster) {
    return nvfp4::gemv_smem(NT, buffers, tokens, SILU ? 2 : 1, kslice, cluster);
  };
  int64_t best = -1;
  int buffers_i = 0;
  for (int i = 0; i < 4; ++i) {
    const int slice = (groups + (1 << i) - 1) >> i;  // groups per CTA
    const int d = smem(4, slice * GROUP, 1 << i) <= MAX_SMEM ? 0 : 1;
    if (d == 1 && smem(2, slice * GROUP, 1 << i) > MAX_SMEM) continue;
    if (i > 0 && slice * ((1 << i) - 1) >= groups) continue;  // a CTA without columns
    for (int kw = 0; 1 << kw <= WARPS; ++kw) {
      const int per_iter = clusters[i] * (WARPS >> kw);
      const int iters = (a.strips + per_iter - 1) / per_iter;
      const int per = (slice + (1 << kw) - 1) >> kw;
      const int64_t rounds = i == 0 ? 0 : (static_cast<int64_t>(iters) * (WARPS >> kw) + ROUND - 1) / ROUND;
      const int64_t cost = 100ll * iters * (per + (kw > 0 ? 1 : 0)) + (rounds * 75 << i) + (SILU ? 12ll : 8ll) * tokens * slice;
      if (best < 0 || cost < best) {
        best = cost;
        buffers_i = d;
        a.cluster_log2 = i;
        a.kwarps_log2 = kw;
        a.per = per;
        a.iters = iters;
        a.kslice = slice * GROUP;
      }
    }
  }
  if (best < 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int per_cluster = WARPS >> a.kwarps_log2;
  int n = (a.strips + per_cluster - 1) / per_cluster;
  if (n > clusters[a.cluster_log2]) n = clusters[a.cluster_log2];
  a.strips_at_once = n * per_cluster;
  attr[1].val.clusterDim.x = 1u << a.cluster_log2;
  cfg.numAttrs = a.cluster_log2 > 0 ? 2 : 1;
  const int64_t tiles = (a.M + a.tile - 1) / a.tile, layers = (tiles + 65534) / 65535;
  cfg.gridDim = dim3(static_cast<unsigned>(n << a.cluster_log2), static_cast<unsigned>((tiles + layers - 1) / layers),
                     static_cast<unsigned>(layers));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem(buffers_i == 0 ? 4 : 2, a.kslice, 1 << a.cluster_log2));
  if (cudaLaunchKernelEx(&cfg, kerns[buffers_i], a) != cudaSuccess) {
    (void)cudaGetLastError();
    return NVFP4_ERR_CUDA;
  }
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return NVFP4_OK;
}

nvfp4_status launch_gemv(DeviceInfo* info, nvfp4::GemvArgs a, bool silu, cudaStream_t stream) {
  using namespace nvfp4;
  if (a.M <= gemvcfg::PAIR_TOKENS) {
    a.tile = static_cast<int>(a.M);
    return !silu      ? launch_gemv<1, PAIR_LANES, SILU_NO>(info, a, stream)
           : a.M == 1 ? launch_gemv<1, PAIR_LANES, SILU_ROWS>(info, a, stream)
                      : launch_gemv<1, PAIR_HALVES, SILU_ROWS>(info, a, stream);
  }
  // 16 rows at a time, or 8 (with SiLU then 4) where so many of a very long K do not fit in a cluster's shared memory
  nvfp4_status st = NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (a.M > 8) {
    a.tile = 16;
    st = silu ? launch_gemv<2, PAIR_NO, SILU_PARTS>(info, a, stream) : launch_gemv<2, PAIR_NO, SILU_NO>(info, a, stream);
  }
  if (st == NVFP4_ERR_UNSUPPORTED_SHAPE && (!silu || a.M > 4)) {
    a.tile = 8;
    st = silu ? launch_gemv<1, PAIR_NO, SILU_PARTS>(info, a, stream) : launch_gemv<1, PAIR_NO, SILU_NO>(info, a, stream);
  }
  if (st == NVFP4_ERR_UNSUPPORTED_SHAPE && silu) {
    a.tile = 4;
    st = launch_gemv<1, PAIR_NO, SILU_ROWS>(info, a, stream);
  }
  return st;
}

}  // namespace

NVFP4_API nvfp4_status gemv_nvfp4(const void* x, int x_dtype, int64_t M, int64_t ldx, int act, nvfp4_tensor B,
                                  const float* bias, int out_dtype, void* D, int64_t ldd, cudaStream_t stream) {
  if (x == nullptr || D == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (x_dtype != NVFP4_OUT_BF16 && x_dtype != NVFP4_OUT_F16) return NVFP4_ERR_INVALID_ARG;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_SILU) return NVFP4_ERR_INVALID_ARG;
  if (!is_dtype(out_dtype)) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st;
  if ((st = check_operand(B)) != NVFP4_OK) return st;
  if (M <= 0 || M > 524280 || B.rows > (1ll << 31) || B.cols % 64 != 0 || B.cols > 32768)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ldx < B.cols || ldd < B.rows) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(x) || ldx % 8 != 0 || !aligned_to(D, static_cast<uintptr_t>(out_size(out_dtype))) ||
      !aligned_to(bias, 4) || !aligned_to(B.gscale, 4))
    return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  nvfp4::GemvArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.x_f16 = x_dtype == NVFP4_OUT_F16;
  a.ldx = ldx;
  a.M = M;
  a.N = B.rows;
  a.K = B.cols;
  a.codes = static_cast<const uint8_t*>(B.codes);
  a.sf = static_cast<const uint8_t*>(B.sf);
  a.gscale = B.gscale;
  a.bias = bias;
  a.D = D;
  a.ldd = ldd;
  a.out_kind = out_dtype;
  a.strips = static_cast<int>((B.rows + 127) / 128 * 8);
  return launch_gemv(info, a, act == NVFP4_ACT_SILU, stream);
}

namespace {

// Checks that the forward call and the gradient share. `branch` and `norm` say which parts are used.
nvfp4_status check_norm(const nvfp4_norm_inputs* in) {
  if (in == nullptr || in->x == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (in->stream_dtype != NVFP4_OUT_BF16 && in->stream_dtype != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (in->mod_dtype != NVFP4_OUT_BF16 && in->mod_dtype != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (in->norm < NVFP4_NORM_NONE || in->norm > NVFP4_NORM_RMS) return NVFP4_ERR_INVALID_ARG;
  if (in->post_norm != 0 && in->post_norm != 1) return NVFP4_ERR_INVALID_ARG;
  if (!(in->eps > 0.0f) || !(in->eps <= 3.4028234663852886e38f)) return NVFP4_ERR_INVALID_ARG;
  if (in->y == nullptr &&
      (in->gate != nullptr || in->post_norm || in->w_post != nullptr || in->residual_scale != 1.0f))
    return NVFP4_ERR_INVALID_ARG;
  if (in->w_post != nullptr && !in->post_norm) return NVFP4_ERR_INVALID_ARG;
  if (in->norm == NVFP4_NORM_NONE && (in->w != nullptr || in->scale != nullptr || in->shift != nullptr))
    return NVFP4_ERR_INVALID_ARG;
  if (in->rows <= 0 || in->rows > (1ll << 31) - 256 || in->cols <= 0 || in->cols % 8 != 0 || in->cols > 16384 ||
      in->batches <= 0 || in->batches > (1ll << 31))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (in->offsets == nullptr && in->rows % in->batches != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t st = out_size(in->stream_dtype), md = out_size(in->mod_dtype);
  if (in->ldx < in->cols || (in->y != nullptr && in->ldy < in->cols)) return NVFP4_ERR_INVALID_ARG;
  const struct {
    const void* p;
    int64_t ld;
  } mods[3] = {{in->gate, in->ldgate}, {in->scale, in->ldscale}, {in->shift, in->ldshift}};
  for (const auto& m : mods) {
    if (m.p == nullptr) continue;
    if (m.ld < in->cols) return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(m.p) || (m.ld * md) % 16 != 0) return NVFP4_ERR_MISALIGNED;
  }
  if (!aligned16(in->x) || (in->ldx * st) % 16 != 0 || !aligned16(in->y) || (in->y != nullptr && in->ldy % 8 != 0) ||
      !aligned16(in->w) || !aligned16(in->w_post) || !aligned_to(in->offsets, 4))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// The ring kernel for many rows: as many CTAs per SM as its registers allow, as long as each has a few
// row buffers, and a piece of rows for each. NVFP4_ERR_UNSUPPORTED_SHAPE: too few rows for it.
template <class ST, int NV, bool POST>
nvfp4_status launch_norm_ring(DeviceInfo* info, nvfp4::NormArgs a, cudaStream_t stream) {
  using namespace nvfp4::normcfg;
  auto kern = nvfp4::residual_norm_ring_kernel<ST, NV, POST>;
  int regs;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    int& known = info->norm_regs[(sizeof(ST) == 4) + 2 * (NV == 4) + 4 * POST];
    if (known == 0) {
      cudaFuncAttributes fa;
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess ||
          cudaFuncGetAttributes(&fa, kern) != cudaSuccess)
        return NVFP4_ERR_CUDA;
      known = (fa.numRegs + 7) / 8 * 8;
    }
    regs = known;
  }
  const int64_t vecs = a.cols / 8;
  const int threads = static_cast<int>((vecs + 32 * NV - 1) / (32 * NV) * 32);
  const int64_t vectors =
      NV == 2 ? nvfp4::norm_vector_bytes(a.cols, a.mod_f32,
                                         (a.gate != nullptr) + (a.scale != nullptr) + (a.shift != nullptr),
                                         (a.w_post != nullptr) + (a.w != nullptr))
              : 0;
  const int64_t stage = nvfp4::norm_stage(a.cols, sizeof(ST), a.y != nullptr);
  int per_sm = 65536 / (regs * threads);
  if (per_sm > 16) per_sm = 16;
  int64_t stages = 0;
  for (; per_sm >= 1; --per_sm) {
    stages = (SMEM / per_sm - SMEM_OTHER - vectors) / stage;
    if (stages >= 3 || per_sm == 1) break;
  }
  const int64_t chunks = static_cast<int64_t>(info->sm_count) * per_sm;
  if (per_sm < 1 || stages < 1 || a.rows < RING_ROWS * chunks) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (stages > FWD_MAX_STAGES) stages = FWD_MAX_STAGES;
  a.chunks = static_cast<int>(chunks);
  a.chunk_rows = a.rows / chunks;
  a.chunk_extra = static_cast<int>(a.rows % chunks);
  a.stages = static_cast<int>(stages);
  return launch_dependent(kern, dim3(static_cast<unsigned>(chunks)), threads,
                          static_cast<size_t>(stages * stage + vectors), stream, a);
}

// `rows`: with the rows that pad an NVFP4 output's block scales.
template <class ST>
nvfp4_status launch_norm(DeviceInfo* info, const nvfp4::NormArgs& a, int64_t rows, cudaStream_t stream) {
  const int64_t vecs = a.cols / 8;
  const nvfp4_status st =
      vecs <= 1024 ? (a.post ? launch_norm_ring<ST, 2, true>(info, a, stream) : launch_norm_ring<ST, 2, false>(info, a, stream))
                   : (a.post ? launch_norm_ring<ST, 4, true>(info, a, stream) : launch_norm_ring<ST, 4, false>(info, a, stream));
  if (st != NVFP4_ERR_UNSUPPORTED_SHAPE) return st;
  if (vecs <= 128) {  // a warp per row, four rows per CTA
    auto kern = vecs <= 32   ? nvfp4::residual_norm_kernel<ST, 1, true>
                : vecs <= 64 ? nvfp4::residual_norm_kernel<ST, 2, true>
                             : nvfp4::residual_norm_kernel<ST, 4, true>;
    return launch_dependent(kern, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, stream, a);
  }
  return launch_dependent(nvfp4::residual_norm_kernel<ST, 2, false>, dim3(static_cast<unsigned>(rows)),
                          static_cast<int>((vecs + 63) / 64 * 32), 0, stream, a);
}

// How the gradient kernel takes a row: CTAs that share its columns (4096 each at most), the columns and
// threads of each, and how many of them share an SM (by registers).
void norm_grad_shape(int64_t cols, int* cluster, int* cta_cols, int* threads, int* per_sm) {
  const int64_t vecs = cols / 8;
  *cluster = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
  const int64_t each = (vecs + *cluster - 1) / *cluster;
  *cta_cols = static_cast<int>(each * 8);
  *threads = static_cast<int>((each + 31) / 32 * 32);
  *per_sm = nvfp4::normcfg::GRAD_THREADS / *threads;
}

// Pieces that the rows are cut into for the gradient: one per CTA or cluster that fits on a B200's 148
// SMs (clusters of 4 do not fill all of its groups of SMs: 32 of 37).
int64_t norm_chunks(int64_t rows, int64_t cols) {
  int cluster, cta_cols, threads, per_sm;
  norm_grad_shape(cols, &cluster, &cta_cols, &threads, &per_sm);
  const int64_t n = cluster == 1 ? 148ll * per_sm : cluster == 2 ? 74ll : 32ll;
  return rows < n ? rows : n;
}

template <class ST, bool POST, bool CLUSTER>
nvfp4_status launch_norm_grad(DeviceInfo* info, nvfp4::NormGradArgs a, cudaStream_t stream) {
  using namespace nvfp4::normcfg;
  auto kern = nvfp4::residual_norm_grad_kernel<ST, POST, CLUSTER>;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    bool& set = info->norm_grad_attr_set[(sizeof(ST) == 4) + 2 * POST + 4 * CLUSTER];
    if (!set) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
        return NVFP4_ERR_CUDA;
      set = true;
    }
  }
  int threads, per_sm;
  norm_grad_shape(a.cols, &a.cluster, &a.cta_cols, &threads, &per_sm);
  const int64_t stage = nvfp4::norm_grad_stage(a.cta_cols, sizeof(ST), a.dxo != nullptr, a.dh != nullptr, a.y != nullptr);
  const int64_t vectors = nvfp4::norm_vector_bytes(a.cta_cols, a.mod_f32, (a.gate != nullptr) + (a.scale != nullptr),
                                                   (a.w_post != nullptr) + (a.w != nullptr));
  int64_t stages = (SMEM / per_sm - SMEM_OTHER - vectors) / stage;  // two at least, whatever width and types
  const int64_t most = (a.rows + a.chunks - 1) / a.chunks;
  if (stages > GRAD_MAX_STAGES) stages = GRAD_MAX_STAGES;
  if (stages > most) stages = most;
  if (stages < 1) stages = 1;
  a.stages = static_cast<int>(stages);
  return launch_dependent(kern, dim3(static_cast<unsigned>(a.chunks * a.cluster)), threads,
                          static_cast<size_t>(stages * stage + vectors), stream, a, a.cluster);
}

template <class ST, bool POST>
nvfp4_status launch_norm_grad(DeviceInfo* info, const nvfp4::NormGradArgs& a, cudaStream_t stream) {
  return a.cols <= 4096 ? launch_norm_grad<ST, POST, false>(info, a, stream)
                        : launch_norm_grad<ST, POST, true>(info, a, stream);
}

}  // namespace

NVFP4_API nvfp4_status residual_norm(const nvfp4_norm_inputs* in, void* x_out, int64_t ldxo, void* h, int64_t ldh,
                                     const nvfp4_tensor* hq, float* stats, cudaStream_t stream) {
  nvfp4_status st;
  if ((st = check_norm(in)) != NVFP4_OK) return st;
  if (x_out == nullptr && h == nullptr && hq == nullptr && stats == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (in->norm == NVFP4_NORM_NONE && (h != nullptr || hq != nullptr)) return NVFP4_ERR_INVALID_ARG;
  if ((x_out != nullptr && ldxo < in->cols) || (h != nullptr && ldh < in->cols)) return NVFP4_ERR_INVALID_ARG;
  if (x_out == in->x && ldxo != in->ldx && in->rows > 1) return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(x_out) || (x_out != nullptr && (ldxo * out_size(in->stream_dtype)) % 16 != 0) || !aligned16(h) ||
      (h != nullptr && ldh % 8 != 0) || !aligned16(stats))
    return NVFP4_ERR_MISALIGNED;
  int64_t rows = in->rows;
  if (hq != nullptr) {
    if (hq->rows != in->rows || hq->cols != in->cols) return NVFP4_ERR_INVALID_ARG;
    if ((st = check_operand(*hq)) != NVFP4_OK) return st;
    if (in->cols % 64 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    rows = (rows + 127) / 128 * 128;
  }
  int dev;
  DeviceInfo* info;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  nvfp4::NormArgs a{};
  a.rows = in->rows;
  a.cols = in->cols;
  a.batches = in->batches;
  a.rows_per_batch = in->offsets == nullptr ? in->rows / in->batches : 1;
  a.offsets = in->offsets;
  a.x = in->x;
  a.ldx = in->ldx;
  a.y = static_cast<const uint16_t*>(in->y);
  a.ldy = in->ldy;
  a.gate = in->gate;
  a.scale = in->scale;
  a.shift = in->shift;
  a.ldgate = in->ldgate;
  a.ldscale = in->ldscale;
  a.ldshift = in->ldshift;
  a.mod_f32 = in->mod_dtype == NVFP4_OUT_F32;
  a.post = in->post_norm;
  a.w_post = in->w_post;
  a.w = in->w;
  a.norm = in->norm;
  a.alpha = in->residual_scale;
  a.eps = in->eps;
  a.x_out = x_out;
  a.ldxo = ldxo;
  a.h = static_cast<uint16_t*>(h);
  a.ldh = ldh;
  if (hq != nullptr) {
    a.q_codes = static_cast<uint8_t*>(hq->codes);
    a.q_sf = static_cast<uint8_t*>(hq->sf);
    a.q_gscale = hq->gscale;
  }
  a.stats = stats;
  return in->stream_dtype == NVFP4_OUT_F32 ? launch_norm<float>(info, a, rows, stream)
                                           : launch_norm<uint16_t>(info, a, rows, stream);
}

NVFP4_API int64_t residual_norm_workspace_bytes(int64_t rows, int64_t cols, int64_t batches) {
  if (rows <= 0 || cols <= 0 || batches <= 0) return -1;
  const int64_t n = norm_chunks(rows, cols);
  return ((n + batches) * 3 + n * 2) * cols * static_cast<int64_t>(sizeof(float)) +
         2 * batches * static_cast<int64_t>(sizeof(int));
}

NVFP4_API nvfp4_status residual_norm_backward(const nvfp4_norm_inputs* in, const float* stats,
                                              const nvfp4_norm_grads* g, void* workspace, cudaStream_t stream) {
  nvfp4_status st;
  if ((st = check_norm(in)) != NVFP4_OK) return st;
  if (g == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (g->dx_out == nullptr && g->dh == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (g->dh != nullptr && in->norm == NVFP4_NORM_NONE) return NVFP4_ERR_INVALID_ARG;
  if (stats == nullptr) return NVFP4_ERR_INVALID_ARG;
  const bool seq = g->dgate != nullptr || g->dscale != nullptr || g->dshift != nullptr;
  const bool weights = g->dw != nullptr || g->dw_post != nullptr;
  if (g->dx == nullptr && g->dy == nullptr && !seq && !weights) return NVFP4_ERR_INVALID_ARG;
  if (in->y == nullptr && (g->dy != nullptr || g->dgate != nullptr || g->dw_post != nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (g->dw_post != nullptr && !in->post_norm) return NVFP4_ERR_INVALID_ARG;
  if (in->norm == NVFP4_NORM_NONE && (g->dscale != nullptr || g->dshift != nullptr || g->dw != nullptr))
    return NVFP4_ERR_INVALID_ARG;
  if ((seq || weights) && workspace == nullptr) return NVFP4_ERR_INVALID_ARG;
  const int64_t es = out_size(in->stream_dtype), cols = in->cols;
  if ((g->dx_out != nullptr && g->lddxo < cols) || (g->dh != nullptr && g->lddh < cols) ||
      (g->dx != nullptr && g->lddx < cols) || (g->dy != nullptr && g->lddy < cols) ||
      (g->dgate != nullptr && g->lddgate < cols) || (g->dscale != nullptr && g->lddscale < cols) ||
      (g->dshift != nullptr && g->lddshift < cols))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(stats) || !aligned16(g->dx_out) || (g->dx_out != nullptr && (g->lddxo * es) % 16 != 0) ||
      !aligned16(g->dh) || (g->dh != nullptr && g->lddh % 8 != 0) || !aligned16(g->dx) ||
      (g->dx != nullptr && (g->lddx * es) % 16 != 0) || !aligned16(g->dy) || (g->dy != nullptr && g->lddy % 8 != 0) ||
      !aligned_to(g->dgate, 4) || !aligned_to(g->dscale, 4) || !aligned_to(g->dshift, 4) || !aligned_to(g->dw, 4) ||
      !aligned_to(g->dw_post, 4) || !aligned16(workspace))
    return NVFP4_ERR_MISALIGNED;
  // in place only where a row's output lies on its own input
  if (in->rows > 1 && ((g->dx != nullptr && g->dx == g->dx_out && g->lddx != g->lddxo) ||
                       (g->dy != nullptr && ((g->dy == g->dh && g->lddy != g->lddh) ||
                                             (g->dy == in->y && g->lddy != in->ldy)))))
    return NVFP4_ERR_INVALID_ARG;
  int dev;
  DeviceInfo* info;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  nvfp4::NormGradArgs a{};
  a.rows = in->rows;
  a.cols = cols;
  a.batches = in->batches;
  a.rows_per_batch = in->offsets == nullptr ? in->rows / in->batches : 1;
  a.offsets = in->offsets;
  a.x = in->x;
  a.ldx = in->ldx;
  a.dxo = g->dx_out;
  a.lddxo = g->lddxo;
  a.dh = static_cast<const uint16_t*>(g->dh);
  a.lddh = g->lddh;
  a.y = static_cast<const uint16_t*>(in->y);
  a.ldy = in->ldy;
  a.gate = in->gate;
  a.scale = in->scale;
  a.ldgate = in->ldgate;
  a.ldscale = in->ldscale;
  a.mod_f32 = in->mod_dtype == NVFP4_OUT_F32;
  a.post = in->post_norm;
  a.w_post = in->w_post;
  a.w = in->w;
  a.norm = in->norm;
  a.alpha = in->residual_scale;
  a.stats = stats;
  a.dx = g->dx;
  a.lddx = g->lddx;
  a.dy = static_cast<uint16_t*>(g->dy);
  a.lddy = g->lddy;
  a.dgate = g->dgate;
  a.dscale = g->dscale;
  a.dshift = g->dshift;
  a.lddgate = g->lddgate;
  a.lddscale = g->lddscale;
  a.lddshift = g->lddshift;
  a.dw = g->dw;
  a.dw_post = g->dw_post;
  a.chunks = static_cast<int>(norm_chunks(in->rows, cols));
  a.chunk_rows = in->rows / a.chunks;
  a.chunk_extra = static_cast<int>(in->rows % a.chunks);
  if (seq || weights) {
    a.seq_part = static_cast<float*>(workspace);
    float* const w_part = a.seq_part + (a.chunks + in->batches) * 3 * cols;
    if (weights) a.w_part = w_part;
    a.seq_pieces = reinterpret_cast<int*>(w_part + static_cast<int64_t>(a.chunks) * 2 * cols);
  }
  st = in->stream_dtype == NVFP4_OUT_F32
           ? (in->post_norm ? launch_norm_grad<float, true>(info, a, stream) : launch_norm_grad<float, false>(info, a, stream))
           : (in->post_norm ? launch_norm_grad<uint16_t, true>(info, a, stream)
                            : launch_norm_grad<uint16_t, false>(info, a, stream));
  if (st != NVFP4_OK || !(seq || weights)) return st;
  const int64_t by = !seq ? 0 : in->batches < 1024 ? in->batches : 1024;
  const dim3 grid(static_cast<unsigned>((cols + 31) / 32), static_cast<unsigned>(by + 1));
  const bool fits = static_cast<int64_t>(grid.x) * grid.y <= 2ll * info->sm_count;
  return launch_dependent(fits ? nvfp4::norm_grad_reduce_kernel<2> : nvfp4::norm_grad_reduce_kernel<4>, grid,
                          32 * nvfp4::normcfg::REDUCE_WARPS, 0, stream, a);
}

namespace {

template <class T>
nvfp4_status launch_rope(const nvfp4::RopeArgs& a, bool interleaved, size_t smem, cudaStream_t stream) {
  // halves: with a number of pairs that 16 bytes do not divide, the second half is not aligned
  auto kern = interleaved                                  ? nvfp4::rope_kernel<T, nvfp4::ROPE_INTERLEAVED>
              : a.npairs % nvfp4::RopeVec<T>::V == 0 ? nvfp4::rope_kernel<T, nvfp4::ROPE_HALVES>
                                                           : nvfp4::rope_kernel<T, nvfp4::ROPE_HALVES_SCALAR>;
  return launch_dependent(kern, dim3(static_cast<unsigned>((a.rows + a.rows_per_cta - 1) / a.rows_per_cta)),
                          nvfp4::ropecfg::THREADS, smem, stream, a);
}

}  // namespace

NVFP4_API nvfp4_status rope_axes(const void* x, int dtype, int64_t rows, int64_t heads, int64_t head_dim,
                                 int64_t x_row_stride, int64_t x_head_stride, const void* positions, int pos_float,
                                 int64_t ldpos, int axes, const int32_t* pairs, const double* freqs, int interleaved,
                                 int inverse, void* y, int64_t y_row_stride, int64_t y_head_stride,
                                 cudaStream_t stream) {
  using namespace nvfp4::ropecfg;
  if (x == nullptr || y == nullptr || positions == nullptr || pairs == nullptr || freqs == nullptr)
    return NVFP4_ERR_INVALID_ARG;
  if (!is_dtype(dtype) || (pos_float & ~1) || (interleaved & ~1) || (inverse & ~1)) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || rows > (1ll << 31) - 1 || heads <= 0 || heads > (1 << 16) || head_dim <= 0 || head_dim % 8 != 0 ||
      head_dim > MAX_HEAD_DIM || axes < 1 || axes > MAX_AXES)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  int64_t n = 0;
  nvfp4::RopeArgs a{};
  for (int i = 0; i < MAX_AXES; ++i) {
    if (i < axes) {
      if (pairs[i] < 1 || pairs[i] > head_dim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
      n += pairs[i];
    }
    a.axis_end[i] = i < axes - 1 ? static_cast<int>(n) : 0x7fffffff;
  }
  if (2 * n > head_dim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ldpos < axes) return NVFP4_ERR_INVALID_ARG;
  // heads of y must not share elements (those of x may: a broadcast input)
  const bool rows_outer = y_row_stride >= y_head_stride;
  const int64_t inner = rows_outer ? y_head_stride : y_row_stride, outer = rows_outer ? y_row_stride : y_head_stride;
  const int64_t inner_n = rows_outer ? heads : rows, outer_n = rows_outer ? rows : heads;
  if ((inner_n > 1 && inner < head_dim) ||
      (outer_n > 1 && (outer < head_dim || (inner_n > 1 && outer / inner < inner_n - 1) ||
                       (inner_n > 1 && outer < (inner_n - 1) * inner + head_dim))))
    return NVFP4_ERR_INVALID_ARG;
  if (x_row_stride < 0 || x_head_stride < 0) return NVFP4_ERR_INVALID_ARG;
  if (x == y && ((rows > 1 && x_row_stride != y_row_stride) || (heads > 1 && x_head_stride != y_head_stride)))
    return NVFP4_ERR_INVALID_ARG;
  const int64_t es = out_size(dtype);
  if (!aligned16(x) || !aligned16(y) || (rows > 1 && ((x_row_stride * es) % 16 != 0 || (y_row_stride * es) % 16 != 0)) ||
      (heads > 1 && ((x_head_stride * es) % 16 != 0 || (y_head_stride * es) % 16 != 0)) || !aligned_to(freqs, 8) ||
      !aligned_to(positions, 4))
    return NVFP4_ERR_MISALIGNED;
  int dev;
  DeviceInfo* info;
  nvfp4_status st;
  if ((st = current_device(&dev, &info)) != NVFP4_OK) return st;
  a.x = x;
  a.y = y;
  a.rows = rows;
  a.heads = static_cast<int>(heads);
  a.head_dim = static_cast<int>(head_dim);
  a.x_row = x_row_stride;
  a.x_head = x_head_stride;
  a.y_row = y_row_stride;
  a.y_head = y_head_stride;
  a.pos = positions;
  a.pos_f32 = pos_float;
  a.ldpos = ldpos;
  a.freqs = freqs;
  a.npairs = static_cast<int>(n);
  a.inverse = inverse;
  a.in_place = x == y;
  // Rows per CTA: as many as fill a thread's batches best, up to two batches (a batch that is half empty
  // was measured at 39.6 us where full ones take 33.4), within the table's limit and with enough CTAs
  // for the GPU.
  a.table_pitch = static_cast<int>((n + 3) / 4 * 4);
  int64_t most = MAX_TABLE_BYTES / (a.table_pitch * 8);
  if (most > rows / (8 * info->sm_count)) most = rows / (8 * info->sm_count);
  const int64_t vec = 16 / es;
  const int64_t units = interleaved        ? head_dim / vec
                        : n % vec == 0 ? n / vec + (head_dim - 2 * n) / vec
                                           : head_dim - n;
  const int64_t slots = units < THREADS ? THREADS / units : 1;
  const int64_t batch = !interleaved && n % vec == 0 ? BATCH_HALVES : BATCH;
  int64_t r = 1;
  double best = 0.0;
  for (int64_t i = 1; i <= most; ++i) {
    const int64_t batches = ((i * heads + slots - 1) / slots + batch - 1) / batch;
    if (batches > 2) break;
    const double full = static_cast<double>(i * heads) / static_cast<double>(slots * batch * batches);
    if (full >= best) {
      best = full;
      r = i;
    }
  }
  a.rows_per_cta = static_cast<int>(r);
  a.units = static_cast<int>(units);
  a.slots = static_cast<int>(slots);
  a.step_rows = static_cast<int>(slots / heads);
  a.step_heads = static_cast<int>(slots % heads);
  a.inv_units = 1.0f / static_cast<float>(units);
  a.inv_heads = 1.0f / static_cast<float>(heads);
  a.inv_pairs = 1.0f / static_cast<float>(n);
  const size_t smem = static_cast<size_t>(r * a.table_pitch) * 2 * sizeof(float);
  const bool inter = interleaved != 0;
  return dtype == NVFP4_OUT_F32   ? launch_rope<float>(a, inter, smem, stream)
         : dtype == NVFP4_OUT_F16 ? launch_rope<__half>(a, inter, smem, stream)
                                  : launch_rope<__nv_bfloat16>(a, inter, smem, stream);
}
