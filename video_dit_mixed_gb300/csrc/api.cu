// extern "C" entry points of libsixbit: argument validation, tensor-map
// construction for the GEMM's TMA loads, and kernel dispatch.  The library
// allocates no device memory.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "ctx_cache.h"
#include "internal.h"

namespace sixbit {

uint64_t current_context_id() {
  struct Fns {
    PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
    PFN_cuCtxGetId_v12000 get_id = nullptr;
  };
  static const Fns fns = [] {
    Fns f;
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      f.get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      f.get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
    return f;
  }();
  if (fns.get_current == nullptr || fns.get_id == nullptr) return 0;
  CUcontext ctx = nullptr;
  if (fns.get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
  unsigned long long id = 0;
  if (fns.get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return static_cast<uint64_t>(id);
}

int sm_count() {
  static ContextCache<int> cache;
  int sms = 0;
  const cudaError_t e = cache.get(&sms, [](int* o) {
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(o, cudaDevAttrMultiProcessorCount, dev);
    return (r == cudaSuccess && *o > 0) ? cudaSuccess : cudaErrorInvalidDevice;
  });
  return (e == cudaSuccess && sms > 0) ? sms : 148;
}

static std::atomic<uint64_t> g_launches{0};
void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

// sixbit_debug_gemm_timeout's setting (0: the normal 2 s limit, no withheld stage).
static std::atomic<uint64_t> g_dbg_wait_ns{0};
static std::atomic<int> g_dbg_withhold{0};
void gemm_debug_params(GemmParams& p) {
  const uint64_t w = g_dbg_wait_ns.load();
  p.wait_ns = w != 0 ? w : kWaitLimitNs;
  p.withhold_first = g_dbg_withhold.load();
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

static bool valid_block(int b) { return b == 16 || b == 64 || b == 256; }

// Checks that the current device is a compute capability 10.3 GPU (once per
// context); the first successful check in a context also resolves the device
// address of the allocation-free entry point's scratch array, so its module
// is loaded at the library's first call on each device.
sixbit_status check_device() {
  static ContextCache<int> ok;
  int v = 0;
  const cudaError_t e = ok.get(&v, [](int* o) {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return cudaErrorInvalidDevice;
    if (major != 10 || minor != 3) return cudaErrorInvalidDevice;
    void* scratch = nullptr;
    (void)noalloc_scratch(&scratch);   // its own call reports a failure
    *o = 1;
    return cudaSuccess;
  });
  return e == cudaSuccess ? SIXBIT_OK : SIXBIT_EUNSUPPORTED;
}

static sixbit_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SIXBIT_OK : SIXBIT_ECUDA; }

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// 2-D row-major tensor [rows, cols] of `dtype`, box = 128 bytes of columns x
// `box_rows` rows, 128-byte swizzle, out-of-bounds rows read as zero.
static bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dtype, int elem_bytes, int rows, int cols,
                     int box_rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem_bytes};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elem_bytes), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, dtype, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// The grouped product's token operand [rows, 2 K bytes] as [K/64][rows][128
// bytes]: a box holds box_chunks chunks of box_rows rows, chunk by chunk, with
// 128-byte swizzle; rows and chunks out of bounds read as zero.
static bool make_token_map(CUtensorMap* m, const uint8_t* base, int rows, int K, int box_rows, int box_chunks) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(K / 64)};
  cuuint64_t strides[2] = {2 * static_cast<cuuint64_t>(K), 128};
  cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_chunks)};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// int8 [rows, cols] for the W4A8 GEMM's activation codes: box 128 bytes of
// columns x 128 rows, 128-byte swizzle (16-byte chunk c of row r lands at
// chunk c ^ (r & 7), so each converter thread's reads of its own row are
// conflict-free), out-of-bounds rows read as zero.
static bool make_map_s8(CUtensorMap* m, const int8_t* base, int rows, int cols) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
  cuuint32_t box[2] = {128, 128};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// bf16 output Y [rows, cols] for the GEMM epilogue's TMA stores: box 32
// columns (64 bytes) x 32 rows, 64-byte swizzle.
static bool make_store_map(CUtensorMap* m, const uint16_t* Y, int rows, int cols) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(Y), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace sixbit

using namespace sixbit;

extern "C" {

size_t sixbit_fp4_scale_bytes(int rows, int K) {
  if (rows < 0 || K < 0) return 0;
  return static_cast<size_t>((rows + 127) / 128) * 128 * static_cast<size_t>(K / 16);
}

size_t sixbit_fp4_scale_offset(int r, int kb, int K) {
  return static_cast<size_t>(r / 128) * (128 * static_cast<size_t>(K / 16)) + static_cast<size_t>(kb / 4) * 512 +
         static_cast<size_t>((r % 32) * 16 + ((r / 32) % 4) * 4 + (kb % 4));
}

size_t sixbit_stats_scratch_bytes(int64_t n) { return stats_scratch_bytes(n); }

size_t sixbit_qgemm_workspace_bytes(int N, int K) {
  if (N <= 0 || K <= 0) return 0;
  return w4a8_workspace_bytes(N, K);
}

uint64_t sixbit_launch_count(void) { return g_launches.load(); }

const char* sixbit_status_str(sixbit_status s) {
  switch (s) {
    case SIXBIT_OK: return "ok";
    case SIXBIT_EINVAL: return "invalid argument";
    case SIXBIT_ESHAPE: return "unsupported shape";
    case SIXBIT_EALIGN: return "pointer not 16-byte aligned";
    case SIXBIT_EUNSUPPORTED: return "no compute capability 10.3 device";
    case SIXBIT_ECUDA: return "CUDA runtime error";
    case SIXBIT_ETIMEOUT: return "device-side wait timed out";
    case SIXBIT_EDEVICE: return "device-side check failed";
    default: return "unknown status";
  }
}

sixbit_status sixbit_debug_gemm_timeout(uint64_t wait_limit_ns, int32_t withhold_first_stage) {
  if (withhold_first_stage != 0 && withhold_first_stage != 1) return SIXBIT_EINVAL;
  g_dbg_wait_ns.store(wait_limit_ns);
  g_dbg_withhold.store(withhold_first_stage);
  return SIXBIT_OK;
}

sixbit_status sixbit_check(int32_t* err_dev, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return SIXBIT_ECUDA;
  if (err_dev == nullptr) return SIXBIT_OK;
  int32_t v = 0;
  if (cudaMemcpy(&v, err_dev, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return SIXBIT_ECUDA;
  if (v != 0) {
    const int32_t z = 0;
    cudaMemcpy(err_dev, &z, sizeof(z), cudaMemcpyHostToDevice);
  }
  return v;
}

sixbit_status sixbit_pack_weights(const float* W, int N, int K, int had_block, const sixbit_weights* out,
                                  int32_t* err_dev, void* stream) {
  (void)err_dev;
  if (W == nullptr || out == nullptr || out->fp4_codes == nullptr || out->fp4_scales == nullptr ||
      out->fp4_amax == nullptr || out->fp4_tensor_scale == nullptr || out->i4_codes == nullptr ||
      out->i4_scales == nullptr || out->bf16_w == nullptr)
    return SIXBIT_EINVAL;
  if (N <= 0 || K <= 0 || K % 128 != 0 || !valid_block(had_block) || K % had_block != 0) return SIXBIT_ESHAPE;
  if (!aligned16(W) || !aligned16(out->fp4_codes) || !aligned16(out->i4_codes) || !aligned16(out->bf16_w))
    return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_pack_weights(W, N, K, had_block, out, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_hadamard_quant(const uint16_t* X, int M, int K, int had_block, int mode,
                                    const int32_t* mode_dev, const float* tamax_in, const sixbit_qact* out,
                                    int32_t* err_dev, void* stream) {
  (void)err_dev;
  if (X == nullptr || out == nullptr) return SIXBIT_EINVAL;
  if (M <= 0 || K <= 0 || K % 128 != 0 || !valid_block(had_block) || K % had_block != 0) return SIXBIT_ESHAPE;
  if (!aligned16(X) || (out->rotated && !aligned16(out->rotated))) return SIXBIT_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool want_fp4 = mode_dev != nullptr || mode == SIXBIT_MODE_NVFP4;
  const bool want_i8 = mode_dev != nullptr || mode == SIXBIT_MODE_INT8;
  if (mode_dev == nullptr && mode != SIXBIT_MODE_NVFP4 && mode != SIXBIT_MODE_INT8) {
    if (mode == SIXBIT_MODE_BF16 || mode == SIXBIT_MODE_SKIP) return SIXBIT_OK;
    return SIXBIT_EINVAL;
  }
  if (want_fp4 && (out->fp4_codes == nullptr || out->fp4_scales == nullptr || out->tensor_scale == nullptr ||
                   (tamax_in == nullptr && out->tensor_amax == nullptr)))
    return SIXBIT_EINVAL;
  if (want_i8 && (out->row_scale == nullptr || out->i8_codes == nullptr)) return SIXBIT_EINVAL;
  if (want_fp4 && !aligned16(out->fp4_codes)) return SIXBIT_EALIGN;
  if (want_i8 && !aligned16(out->i8_codes)) return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  if (want_fp4) {
    const float* amax = tamax_in;
    if (amax == nullptr) {
      cudaError_t e = launch_hq_amax(X, M, K, had_block, mode_dev, out->tensor_amax, st);
      if (e != cudaSuccess) return SIXBIT_ECUDA;
      amax = out->tensor_amax;
    }
    cudaError_t e = launch_hq_nvfp4(X, M, K, had_block, mode_dev, amax, out, st);
    if (e != cudaSuccess) return SIXBIT_ECUDA;
  }
  if (want_i8) {
    cudaError_t e = launch_hq_int8(X, M, K, had_block, mode_dev, out, st);
    if (e != cudaSuccess) return SIXBIT_ECUDA;
  }
  return SIXBIT_OK;
}

static sixbit_status qgemm_impl(const sixbit_qact* A, const uint16_t* X_bf16, const sixbit_weights* W, int M,
                                int N, int K, int mode, const int32_t* mode_dev, int epilogue,
                                const uint16_t* residual, uint16_t* Y, float* Y_f32, int32_t* acc_dbg,
                                void* workspace, int32_t* err_dev, void* stream, int had_block, float* rot_amax,
                                uint16_t* bs_delta = nullptr, void* bs_parts = nullptr) {
  if (W == nullptr || (Y == nullptr && Y_f32 == nullptr)) return SIXBIT_EINVAL;
  if (epilogue != SIXBIT_EPI_NONE && epilogue != SIXBIT_EPI_GELU && epilogue != SIXBIT_EPI_RESIDUAL)
    return SIXBIT_EINVAL;
  if (epilogue == SIXBIT_EPI_RESIDUAL && residual == nullptr) return SIXBIT_EINVAL;
  if (M <= 0 || N <= 0 || K <= 0 || K % 128 != 0 || N % 16 != 0) return SIXBIT_ESHAPE;
  if ((Y && !aligned16(Y)) || (Y_f32 && !aligned16(Y_f32)) || (residual && !aligned16(residual)))
    return SIXBIT_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool only_fp4 = rot_amax != nullptr;  // the rotated-amax epilogue exists for the NVFP4 kind only
  const bool run_fp4 = mode_dev != nullptr || mode == SIXBIT_MODE_NVFP4;
  const bool run_i8 = !only_fp4 && (mode_dev != nullptr || mode == SIXBIT_MODE_INT8);
  const bool run_bf = !only_fp4 && (mode_dev != nullptr || mode == SIXBIT_MODE_BF16);
  if (mode_dev == nullptr && !run_fp4 && !run_i8 && !run_bf) return mode == SIXBIT_MODE_SKIP ? SIXBIT_OK : SIXBIT_EINVAL;
  if ((run_fp4 || run_i8) && A == nullptr) return SIXBIT_EINVAL;
  if (run_fp4 && (A->fp4_codes == nullptr || A->fp4_scales == nullptr || A->tensor_scale == nullptr ||
                  W->fp4_codes == nullptr || W->fp4_scales == nullptr || W->fp4_tensor_scale == nullptr))
    return SIXBIT_EINVAL;
  if (run_i8 && (A->i8_codes == nullptr || A->row_scale == nullptr || W->i4_codes == nullptr ||
                 W->i4_scales == nullptr || workspace == nullptr))
    return SIXBIT_EINVAL;
  if (run_bf && (X_bf16 == nullptr || W->bf16_w == nullptr)) return SIXBIT_EINVAL;
  if ((run_fp4 && (!aligned16(A->fp4_codes) || !aligned16(A->fp4_scales) || !aligned16(W->fp4_codes) ||
                   !aligned16(W->fp4_scales))) ||
      (run_i8 && (!aligned16(A->i8_codes) || !aligned16(W->i4_codes) || !aligned16(workspace))) ||
      (run_bf && (!aligned16(X_bf16) || !aligned16(W->bf16_w))))
    return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  if (rot_amax != nullptr && cudaMemsetAsync(rot_amax, 0, sizeof(float), st) != cudaSuccess) return SIXBIT_ECUDA;

  GemmParams p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.mode_dev = mode_dev;
  p.epilogue = epilogue;
  p.residual = residual;
  p.Y = Y;
  p.Yf = Y_f32;
  p.err = err_dev;
  // Walk the shorter output dimension fastest: the CTAs in flight then share
  // tiles of the larger operand, which streams from HBM once, while the
  // smaller one is re-read from L2 (an A of 17776 x 7680 bf16 does not fit
  // in L2 and would be re-read from HBM once per column-tile pass).
  p.n_fastest = M > N ? 1 : 0;
  p.rot_amax = rot_amax;
  p.had_block = had_block;
  p.bs_delta = bs_delta;
  p.bs_parts = bs_parts;
  gemm_debug_params(p);
  // The bf16-operand kinds (BF16, W4A8) write a bf16 Y through TMA stores
  // (Y 16-byte aligned, N % 16 == 0 checked above); an FP32 Y is stored
  // directly.
  CUtensorMap my{};
  p.y_tma = (Y_f32 == nullptr && (run_bf || run_i8)) ? 1 : 0;
  if (p.y_tma && !make_store_map(&my, Y, M, N)) return SIXBIT_ECUDA;
  if (run_fp4) {
    CUtensorMap ma, mb;
    if (!make_map(&ma, A->fp4_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, M, K / 2, 128) ||
        !make_map(&mb, W->fp4_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K / 2, 256))
      return SIXBIT_ECUDA;
    GemmParams q = p;
    q.want_mode = SIXBIT_MODE_NVFP4;
    q.sfa = A->fp4_scales;
    q.sfb = W->fp4_scales;
    q.s_a = A->tensor_scale;
    q.s_b = W->fp4_tensor_scale;
    if (launch_qgemm_nvf4(ma, mb, q, st) != cudaSuccess) return SIXBIT_ECUDA;
  }
  if (run_i8) {
    // the INT4 weights, expanded to fp16 once per call into the workspace
    uint16_t* wexp = static_cast<uint16_t*>(workspace);
    CUtensorMap ma, mb;
    if (!make_map_s8(&ma, A->i8_codes, M, K) ||
        !make_map(&mb, wexp, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, N, K, 192))
      return SIXBIT_ECUDA;
    if (launch_w4_expand(W->i4_codes, N, K, wexp, mode_dev, st) != cudaSuccess) return SIXBIT_ECUDA;
    GemmParams q = p;
    q.want_mode = SIXBIT_MODE_INT8;
    q.row_scale = A->row_scale;
    q.grp_scale = W->i4_scales;
    q.acc_dbg = acc_dbg;
    if (launch_qgemm_w4a8(ma, mb, my, q, st) != cudaSuccess) return SIXBIT_ECUDA;
  }
  if (run_bf) {
    CUtensorMap ma, mb;
    if (!make_map(&ma, X_bf16, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, K, 128) ||
        !make_map(&mb, W->bf16_w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, N, K, 256))
      return SIXBIT_ECUDA;
    GemmParams q = p;
    q.want_mode = SIXBIT_MODE_BF16;
    if (launch_qgemm_bf16(ma, mb, my, q, st) != cudaSuccess) return SIXBIT_ECUDA;
  }
  return SIXBIT_OK;
}

sixbit_status sixbit_qgemm(const sixbit_qact* A, const uint16_t* X_bf16, const sixbit_weights* W, int M, int N,
                           int K, int mode, const int32_t* mode_dev, int epilogue, const uint16_t* residual,
                           uint16_t* Y, float* Y_f32, int32_t* acc_dbg, void* workspace, int32_t* err_dev,
                           void* stream) {
  return qgemm_impl(A, X_bf16, W, M, N, K, mode, mode_dev, epilogue, residual, Y, Y_f32, acc_dbg, workspace, err_dev,
                    stream, 0, nullptr);
}

sixbit_status sixbit_qgemm_rotamax(const sixbit_qact* A, const sixbit_weights* W, int M, int N, int K,
                                   const int32_t* mode_dev, int epilogue, const uint16_t* residual, uint16_t* Y,
                                   int had_block, float* amax_out, int32_t* err_dev, void* stream) {
  if (Y == nullptr || amax_out == nullptr) return SIXBIT_EINVAL;
  if ((had_block != 16 && had_block != 64) || N % 128 != 0) return SIXBIT_ESHAPE;
  return qgemm_impl(A, nullptr, W, M, N, K, SIXBIT_MODE_NVFP4, mode_dev, epilogue, residual, Y, nullptr, nullptr,
                    nullptr, err_dev, stream, had_block, amax_out);
}

sixbit_status sixbit_qgemm_blockstats(const sixbit_qact* A, const uint16_t* X_bf16, const sixbit_weights* W, int M,
                                      int N, int K, int mode, const int32_t* mode_dev, const uint16_t* residual,
                                      uint16_t* Y, uint16_t* delta_cache, void* parts, void* workspace,
                                      int32_t* err_dev, void* stream) {
  if (residual == nullptr || Y == nullptr || delta_cache == nullptr || parts == nullptr) return SIXBIT_EINVAL;
  if (!aligned16(delta_cache) || !aligned16(parts)) return SIXBIT_EALIGN;
  return qgemm_impl(A, X_bf16, W, M, N, K, mode, mode_dev, SIXBIT_EPI_RESIDUAL, residual, Y, nullptr, nullptr,
                    workspace, err_dev, stream, 0, nullptr, delta_cache, parts);
}

size_t sixbit_blockstats_parts_bytes(void) {
  if (check_device() != SIXBIT_OK) return 0;
  return bs_parts_bytes();
}

sixbit_status sixbit_block_stats_parts(const void* parts, int64_t n, sixbit_stats* stats_dev, int32_t* err_dev,
                                       void* stream) {
  (void)err_dev;
  if (parts == nullptr || stats_dev == nullptr) return SIXBIT_EINVAL;
  if (n <= 0) return SIXBIT_ESHAPE;
  if (!aligned16(parts)) return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_block_stats_parts(parts, n, stats_dev, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_block_stats(const uint16_t* x_in, const uint16_t* x_out, uint16_t* delta_cache, int64_t n,
                                 const int32_t* mode_dev, sixbit_stats* stats_dev, void* scratch, int32_t* err_dev,
                                 void* stream) {
  (void)err_dev;
  if (x_in == nullptr || x_out == nullptr || delta_cache == nullptr || stats_dev == nullptr || scratch == nullptr)
    return SIXBIT_EINVAL;
  if (n <= 0 || n % 8 != 0) return SIXBIT_ESHAPE;
  if (!aligned16(x_in) || !aligned16(x_out) || !aligned16(delta_cache) || !aligned16(scratch)) return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(
      launch_block_stats(x_in, x_out, delta_cache, n, mode_dev, stats_dev, scratch, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_tensor_stats(const uint16_t* x, int64_t n, double* out_dev, void* scratch, int32_t* err_dev,
                                  void* stream) {
  (void)err_dev;
  if (x == nullptr || out_dev == nullptr || scratch == nullptr) return SIXBIT_EINVAL;
  if (n <= 0 || n % 8 != 0) return SIXBIT_ESHAPE;
  if (!aligned16(x) || !aligned16(scratch)) return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_tensor_stats(x, n, out_dev, scratch, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_skip_apply(const uint16_t* x_in, const uint16_t* delta_cache, uint16_t* x_out, int64_t n,
                                const int32_t* mode_dev, sixbit_stats* stats_dev, void* scratch, int32_t* err_dev,
                                void* stream) {
  (void)err_dev;
  if (x_in == nullptr || delta_cache == nullptr || x_out == nullptr || stats_dev == nullptr || scratch == nullptr)
    return SIXBIT_EINVAL;
  if (n <= 0 || n % 8 != 0) return SIXBIT_ESHAPE;
  if (!aligned16(x_in) || !aligned16(x_out) || !aligned16(delta_cache) || !aligned16(scratch)) return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(
      launch_skip_apply(x_in, delta_cache, x_out, n, mode_dev, stats_dev, scratch, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_block_stats_mxfp8(const uint16_t* x_in, const uint16_t* x_out, uint8_t* delta_codes,
                                       uint8_t* delta_scales, int64_t n, const int32_t* mode_dev,
                                       sixbit_stats* stats_dev, void* scratch, int32_t* err_dev, void* stream) {
  (void)err_dev;
  if (x_in == nullptr || x_out == nullptr || delta_codes == nullptr || delta_scales == nullptr ||
      stats_dev == nullptr || scratch == nullptr)
    return SIXBIT_EINVAL;
  if (n <= 0 || n % 32 != 0) return SIXBIT_ESHAPE;
  if (!aligned16(x_in) || !aligned16(x_out) || !aligned16(delta_codes) || !aligned16(scratch)) return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_block_stats_mx(x_in, x_out, delta_codes, delta_scales, n, mode_dev, stats_dev, scratch,
                                           static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_skip_apply_mxfp8(const uint16_t* x_in, const uint8_t* delta_codes, const uint8_t* delta_scales,
                                      uint16_t* x_out, int64_t n, const int32_t* mode_dev, sixbit_stats* stats_dev,
                                      void* scratch, int32_t* err_dev, void* stream) {
  (void)err_dev;
  if (x_in == nullptr || delta_codes == nullptr || delta_scales == nullptr || x_out == nullptr ||
      stats_dev == nullptr || scratch == nullptr)
    return SIXBIT_EINVAL;
  if (n <= 0 || n % 32 != 0) return SIXBIT_ESHAPE;
  if (!aligned16(x_in) || !aligned16(x_out) || !aligned16(delta_codes) || !aligned16(scratch)) return SIXBIT_EALIGN;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_skip_apply_mx(x_in, delta_codes, delta_scales, x_out, n, mode_dev, stats_dev, scratch,
                                          static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_policy_step(const sixbit_policy_cfg* cfg, sixbit_policy_state* state_dev,
                                 const sixbit_stats* last_stats_dev, const double* in_stats_dev, int32_t* mode_dev,
                                 int32_t* err_dev, void* stream) {
  (void)err_dev;
  if (cfg == nullptr || state_dev == nullptr || last_stats_dev == nullptr || in_stats_dev == nullptr ||
      mode_dev == nullptr)
    return SIXBIT_EINVAL;
  sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(
      launch_policy(*cfg, state_dev, last_stats_dev, in_stats_dev, mode_dev, static_cast<cudaStream_t>(stream)));
}

static sixbit_status check_blocks(const sixbit_policy_cfg* cfg, const sixbit_dit_blocks* blocks, int l,
                                  void* scratch) {
  if (cfg == nullptr || blocks == nullptr || scratch == nullptr) return SIXBIT_EINVAL;
  const sixbit_dit_blocks& B = *blocks;
  if (B.states == nullptr || B.stats == nullptr || B.modes == nullptr || B.run_len == nullptr ||
      B.in_stats0 == nullptr || B.x0 == nullptr || B.buf[0] == nullptr || B.buf[1] == nullptr ||
      B.deltas == nullptr)
    return SIXBIT_EINVAL;
  if (B.delta_format != SIXBIT_DELTA_BF16 && B.delta_format != SIXBIT_DELTA_MXFP8) return SIXBIT_EINVAL;
  if (B.delta_format == SIXBIT_DELTA_MXFP8 && B.delta_scales == nullptr) return SIXBIT_EINVAL;
  if (B.L <= 0 || l < 0 || l >= B.L || B.n <= 0 || B.n % 8 != 0) return SIXBIT_ESHAPE;
  if (B.delta_format == SIXBIT_DELTA_MXFP8 && B.n % 32 != 0) return SIXBIT_ESHAPE;
  if (!aligned16(B.x0) || !aligned16(B.buf[0]) || !aligned16(B.buf[1]) || !aligned16(B.deltas) ||
      !aligned16(scratch))
    return SIXBIT_EALIGN;
  return check_device();
}

sixbit_status sixbit_dit_begin(const sixbit_policy_cfg* cfg, const sixbit_dit_blocks* blocks, void* scratch,
                               int32_t* err_dev, void* stream) {
  const sixbit_status s = check_blocks(cfg, blocks, 0, scratch);
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_dit_begin(*cfg, *blocks, scratch, err_dev, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_dit_block_end(const sixbit_policy_cfg* cfg, const sixbit_dit_blocks* blocks, int l,
                                   void* scratch, int32_t* err_dev, void* stream) {
  const sixbit_status s = check_blocks(cfg, blocks, l, scratch);
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_dit_block_end(*cfg, *blocks, l, scratch, err_dev, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_dit_block_end_parts(const sixbit_policy_cfg* cfg, const sixbit_dit_blocks* blocks, int l,
                                         const void* parts, int32_t* err_dev, void* stream) {
  (void)err_dev;
  if (parts == nullptr || (blocks != nullptr && blocks->delta_format != SIXBIT_DELTA_BF16)) return SIXBIT_EINVAL;
  if (!aligned16(parts)) return SIXBIT_EALIGN;
  const sixbit_status s = check_blocks(cfg, blocks, l, const_cast<void*>(parts));
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_dit_block_end_parts(*cfg, *blocks, l, parts, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_dit_skip_run(const sixbit_policy_cfg* cfg, const sixbit_dit_blocks* blocks, int l,
                                  void* scratch, int32_t* err_dev, void* stream) {
  const sixbit_status s = check_blocks(cfg, blocks, l, scratch);
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_dit_skip_run(*cfg, *blocks, l, scratch, err_dev, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_add_rmsnorm_quant(const uint16_t* X, const uint16_t* residual, const float* weight, int M, int K,
                                       float eps, int had_block, const int32_t* mode_dev, uint16_t* sum_out,
                                       const sixbit_qact* out, int32_t* err_dev, void* stream) {
  (void)err_dev;
  if (M < 0 || K <= 0 || K % 128 != 0 || (had_block != 0 && (!valid_block(had_block) || K % had_block != 0)))
    return SIXBIT_ESHAPE;
  if (!(eps > 0.f) || !std::isfinite(eps) || out == nullptr || (sum_out != nullptr && residual == nullptr))
    return SIXBIT_EINVAL;
  if (M == 0) return SIXBIT_OK;
  if (X == nullptr || out->i8_codes == nullptr || out->row_scale == nullptr) return SIXBIT_EINVAL;
  if (!aligned16(X) || !aligned16(residual) || !aligned16(weight) || !aligned16(sum_out) ||
      !aligned16(out->i8_codes) || !aligned_to(out->row_scale, 4))
    return SIXBIT_EALIGN;
  const sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  return cuda_status(launch_add_rmsnorm_quant(X, residual, weight, M, K, eps, had_block, mode_dev, sum_out,
                                              out->i8_codes, out->row_scale, static_cast<cudaStream_t>(stream)));
}

// The checks that sixbit_qgemv and sixbit_qgemm_grouped share, and their
// kernels' parameters.  *empty: there is nothing to do.
static sixbit_status rows_params(const sixbit_qact* A, const sixbit_weights* W, const int32_t* offsets, int E, int M,
                                 int N, int K, const int32_t* mode_dev, int epilogue, const uint16_t* residual,
                                 uint16_t* Y, float* Y_f32, int32_t* err_dev, RowsParams* p, bool* empty) {
  *empty = false;
  if (A == nullptr || W == nullptr) return SIXBIT_EINVAL;
  if (epilogue != SIXBIT_EPI_NONE && epilogue != SIXBIT_EPI_GELU && epilogue != SIXBIT_EPI_RESIDUAL)
    return SIXBIT_EINVAL;
  // (a last tile of up to 128 weight rows ends within 32 bits)
  if (M < 0 || N <= 0 || N > INT32_MAX - 128 || K <= 0 || K % 128 != 0) return SIXBIT_ESHAPE;
  if (M == 0) {
    *empty = true;
    return SIXBIT_OK;
  }
  if (A->i8_codes == nullptr || A->row_scale == nullptr || W->i4_codes == nullptr || W->i4_scales == nullptr ||
      (Y == nullptr && Y_f32 == nullptr) || (epilogue == SIXBIT_EPI_RESIDUAL && residual == nullptr))
    return SIXBIT_EINVAL;
  if (!aligned16(A->i8_codes) || !aligned16(W->i4_codes) || !aligned_to(A->row_scale, 4) ||
      !aligned_to(W->i4_scales, 4) || !aligned_to(offsets, 4) || !aligned_to(residual, 2) || !aligned_to(Y, 2) ||
      !aligned_to(Y_f32, 4))
    return SIXBIT_EALIGN;
  *p = RowsParams{};
  p->codes = A->i8_codes;
  p->row_scale = A->row_scale;
  p->w4 = W->i4_codes;
  p->w4_scale = W->i4_scales;
  p->offsets = offsets;
  p->M = M;
  p->N = N;
  p->K = K;
  p->E = E;
  p->mode_dev = mode_dev;
  p->epilogue = epilogue;
  p->residual = residual;
  p->Y = Y_f32 != nullptr ? nullptr : Y;
  p->Yf = Y_f32;
  p->err = err_dev;
  GemmParams dbg;
  gemm_debug_params(dbg);
  p->wait_ns = dbg.wait_ns;
  p->withhold_first = dbg.withhold_first;
  return check_device();
}

sixbit_status sixbit_qgemv(const sixbit_qact* A, const sixbit_weights* W, int M, int N, int K, const int32_t* mode_dev,
                           int epilogue, const uint16_t* residual, uint16_t* Y, float* Y_f32, int32_t* err_dev,
                           void* stream) {
  if (M > SIXBIT_QGEMV_MAX_ROWS) return SIXBIT_ESHAPE;
  RowsParams p;
  bool empty;
  const sixbit_status s = rows_params(A, W, nullptr, 1, M, N, K, mode_dev, epilogue, residual, Y, Y_f32, err_dev, &p,
                                      &empty);
  if (s != SIXBIT_OK || empty) return s;
  return cuda_status(launch_w4a8_rows(p, static_cast<cudaStream_t>(stream)));
}

size_t sixbit_qgemm_grouped_workspace_bytes(int M, int K) {
  if (M <= 0 || K <= 0) return 0;
  // two digits a code, a sum of each group's codes
  return static_cast<size_t>(M) * static_cast<size_t>(K) * 2 + static_cast<size_t>(M) * (static_cast<size_t>(K) / 128) * 4;
}

sixbit_status sixbit_qgemm_grouped(const sixbit_qact* A, const sixbit_weights* W, const int32_t* offsets, int E, int M,
                                   int N, int K, const int32_t* mode_dev, int epilogue, const uint16_t* residual,
                                   uint16_t* Y, float* Y_f32, void* workspace, int32_t* err_dev, void* stream) {
  // (E N weight rows are a tensor map's coordinate)
  if (E < 1 || E > SIXBIT_MAX_EXPERTS || static_cast<int64_t>(E) * N > INT32_MAX - 128) return SIXBIT_ESHAPE;
  RowsParams p;
  bool empty;
  const sixbit_status s = rows_params(A, W, offsets, E, M, N, K, mode_dev, epilogue, residual, Y, Y_f32, err_dev, &p,
                                      &empty);
  if (s != SIXBIT_OK || empty) return s;
  if (offsets == nullptr || workspace == nullptr) return SIXBIT_EINVAL;
  if (!aligned16(workspace)) return SIXBIT_EALIGN;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Up to 8 rows over up to 16 experts: dot products, an expert's rows one or
  // two at a time, an empty expert's CTAs in vain (7680 x 1920, against the
  // tensor cores: 1 row over 8 experts 5.8 us / 10.2, 8 rows 14.4 / 15.1, over
  // 16 18.9 / 18.6, over 32 23.9 / 18.7; 1920 x 7680, 8 rows over 8 14.1 / 18.4;
  // but 16 skewed rows over 8 20.2 / 16.5, 16 of one expert 17.6 / 10.0).  How the
  // rows fall is known on the device only: eight rows of one expert take 10.4 us.
  // Above: token tiles of 32 up to 48 rows an expert on average, else of 96
  // (8 experts: 256 rows 26.4 us against 31.1, 384 rows 32.5 against 31.9, 1024
  // rows 58.4 against 49.6).
  if (M <= 8 && E <= 16) return cuda_status(launch_w4a8_rows(p, st));
  uint8_t* xd = static_cast<uint8_t*>(workspace);
  const bool narrow = M < 48 * static_cast<int64_t>(E);
  CUtensorMap mw;
  TokenMaps mx;
  if (!make_map(&mw, W->i4_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, E * N, K / 2, 128)) return SIXBIT_ECUDA;
  for (int i = 0; i < token_maps(narrow); ++i)
    if (!make_token_map(&mx.map[i], xd, M, K, (i + 1) * token_box(narrow), token_chunks(narrow))) return SIXBIT_ECUDA;
  float* less = narrow ? reinterpret_cast<float*>(xd + static_cast<size_t>(M) * K * 2) : nullptr;
  p.less = less;
  if (launch_digits(p.codes, M, K, mode_dev, xd, less, st) != cudaSuccess) return SIXBIT_ECUDA;
  return cuda_status(launch_w4a8_grouped(mw, mx, p, narrow, st));
}

sixbit_status sixbit_gated_rmsnorm_quant(const uint16_t* X, const uint16_t* residual, float residual_scale,
                                         const float* weight, const float* post_weight, const float* gate,
                                         const float* scale, const float* shift, const int32_t* segment, int S, int M,
                                         int K, float eps, int had_block, const int32_t* mode_dev, uint16_t* sum_out,
                                         uint16_t* Y, const sixbit_qact* out, int32_t* err_dev, void* stream) {
  if (M < 0 || K <= 0 || K % 128 != 0 || K > 16384 || S < 1 ||
      (had_block != 0 && (!valid_block(had_block) || K % had_block != 0)) || (segment == nullptr && M % S != 0))
    return SIXBIT_ESHAPE;
  if (!(eps > 0.f) || !std::isfinite(eps) || !std::isfinite(residual_scale) || (Y == nullptr && out == nullptr) ||
      (Y != nullptr && had_block != 0))
    return SIXBIT_EINVAL;
  if (M == 0) return SIXBIT_OK;
  if (X == nullptr || (Y == nullptr && (out->i8_codes == nullptr || out->row_scale == nullptr))) return SIXBIT_EINVAL;
  for (const void* q : {static_cast<const void*>(X), static_cast<const void*>(residual),
                        static_cast<const void*>(sum_out), static_cast<const void*>(Y),
                        static_cast<const void*>(weight), static_cast<const void*>(post_weight),
                        static_cast<const void*>(gate), static_cast<const void*>(scale),
                        static_cast<const void*>(shift)})
    if (!aligned16(q)) return SIXBIT_EALIGN;
  if (!aligned_to(segment, 4) || (Y == nullptr && (!aligned16(out->i8_codes) || !aligned_to(out->row_scale, 4))))
    return SIXBIT_EALIGN;
  const sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  GatedNormParams g{};
  g.x = X;
  g.res = residual;
  g.w = weight;
  g.post_w = post_weight;
  g.gate = gate;
  g.scale = scale;
  g.shift = shift;
  g.segment = segment;
  g.res_scale = residual_scale;
  g.eps = eps;
  g.M = M;
  g.K = K;
  g.S = S;
  g.rows_per_seg = M / S > 0 ? M / S : 1;
  g.mode_dev = mode_dev;
  g.sum_out = sum_out;
  g.y = Y;
  if (Y == nullptr) {
    g.codes = out->i8_codes;
    g.row_scale = out->row_scale;
  }
  g.err = err_dev;
  GemmParams dbg;
  gemm_debug_params(dbg);
  g.wait_ns = dbg.wait_ns;
  g.withhold_first = dbg.withhold_first;
  return cuda_status(launch_gated_norm(g, had_block, static_cast<cudaStream_t>(stream)));
}

size_t sixbit_moe_route_workspace_bytes(int T, int E) {
  if (T <= kRouteTurn || E <= 0) return 0;
  return static_cast<size_t>(kRouteRuns) * ((static_cast<size_t>(E) + 3) / 4 * 4) * 4;
}

sixbit_status sixbit_moe_route(const float* logits, const uint16_t* logits_bf16, const float* bias, int T, int E, int k,
                               int score, int groups, int top_groups, int group_best, int renormalize, float factor,
                               int32_t* experts, float* weights, int32_t* rows, int32_t* token, int32_t* offsets,
                               void* workspace, void* stream) {
  if (T < 0 || E < 1 || E > SIXBIT_MAX_EXPERTS || k < 1 || k > SIXBIT_MAX_TOP_K ||
      static_cast<int64_t>(T) * k > INT32_MAX || groups < 1 || groups > SIXBIT_MAX_GROUPS || E % groups != 0 ||
      top_groups < 1 || top_groups > groups || k > top_groups * (E / groups))
    return SIXBIT_ESHAPE;
  if ((score != SIXBIT_SCORE_SOFTMAX && score != SIXBIT_SCORE_SIGMOID) || group_best < 1 || group_best > 2 ||
      !std::isfinite(factor) || offsets == nullptr)
    return SIXBIT_EINVAL;
  if (T > 0 && ((logits == nullptr && logits_bf16 == nullptr) || experts == nullptr || weights == nullptr ||
                rows == nullptr || token == nullptr ||
                (workspace == nullptr && sixbit_moe_route_workspace_bytes(T, E) > 0)))
    return SIXBIT_EINVAL;
  for (const void* q : {static_cast<const void*>(logits), static_cast<const void*>(bias),
                        static_cast<const void*>(experts), static_cast<const void*>(weights),
                        static_cast<const void*>(rows), static_cast<const void*>(token),
                        static_cast<const void*>(offsets)})
    if (!aligned_to(q, 4)) return SIXBIT_EALIGN;
  if (!aligned16(workspace)) return SIXBIT_EALIGN;
  if (!aligned_to(logits_bf16, 2)) return SIXBIT_EALIGN;
  const sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  RouteParams p{};
  p.logits = logits;
  p.logits_bf16 = logits_bf16;
  p.bias = bias;
  p.T = T;
  p.E = E;
  p.k = k;
  p.score = score;
  p.groups = groups;
  p.top_groups = top_groups;
  p.best = group_best;
  p.renorm = renormalize != 0;
  p.factor = factor;
  p.experts = experts;
  p.weights = weights;
  p.rows = rows;
  p.token = token;
  p.offsets = offsets;
  p.counts = static_cast<int32_t*>(workspace);
  return cuda_status(launch_moe_route(p, static_cast<cudaStream_t>(stream)));
}

sixbit_status sixbit_moe_combine(const uint16_t* d, const float* d_f32, const int32_t* rows, const float* weights,
                                 int T, int k, int R, int H, uint16_t* Y, float* Y_f32, int32_t* err_dev,
                                 void* stream) {
  if (T < 0 || k < 1 || k > SIXBIT_MAX_TOP_K || R < 0 || H < 1 || H > 1 << 20) return SIXBIT_ESHAPE;
  if (T == 0) return SIXBIT_OK;
  if ((R > 0 && d == nullptr && d_f32 == nullptr) || rows == nullptr || weights == nullptr ||
      (Y == nullptr && Y_f32 == nullptr))
    return SIXBIT_EINVAL;
  if (!aligned_to(d, 2) || !aligned_to(d_f32, 4) || !aligned_to(rows, 4) || !aligned_to(weights, 4) ||
      !aligned_to(Y, 2) || !aligned_to(Y_f32, 4))
    return SIXBIT_EALIGN;
  const sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  CombineParams p{};
  p.f32 = d_f32 != nullptr;
  p.d = p.f32 ? static_cast<const void*>(d_f32) : d;
  p.rows = rows;
  p.weights = weights;
  p.T = T;
  p.k = k;
  p.H = H;
  p.R = R;
  p.Y = Y_f32 != nullptr ? nullptr : Y;
  p.Yf = Y_f32;
  p.err = err_dev;
  return cuda_status(launch_moe_combine(p, static_cast<cudaStream_t>(stream)));
}

size_t sixbit_lowrank_workspace_bytes(int M, int R) { return M <= 0 || R <= 0 ? 0 : lowrank_workspace(M, R); }

sixbit_status sixbit_lowrank_add(const sixbit_qact* A, const uint16_t* x_bf16, const uint16_t* lr_a,
                                 const uint16_t* lr_b, const float* alpha, const int32_t* ids, int L, int M, int N,
                                 int K, int R, const uint16_t* base, const float* base_f32, const int32_t* mode_dev,
                                 int epilogue, const uint16_t* residual, uint16_t* Y, float* Y_f32, void* workspace,
                                 int32_t* err_dev, void* stream) {
  if (epilogue != SIXBIT_EPI_NONE && epilogue != SIXBIT_EPI_GELU && epilogue != SIXBIT_EPI_RESIDUAL)
    return SIXBIT_EINVAL;
  if (M < 0 || M > INT32_MAX - 512 || N < 1 || N > 1 << 20 || K <= 0 || K > 1 << 20 || K % 128 != 0 || R < 16 ||
      R > SIXBIT_MAX_RANK || R % 16 != 0 || L < 1 || L > SIXBIT_MAX_ADAPTERS)
    return SIXBIT_ESHAPE;
  if (base != nullptr && base_f32 != nullptr) return SIXBIT_EINVAL;
  if (M == 0) return SIXBIT_OK;
  if ((x_bf16 == nullptr && (A == nullptr || A->i8_codes == nullptr || A->row_scale == nullptr)) || lr_a == nullptr ||
      lr_b == nullptr || ids == nullptr || (Y == nullptr && Y_f32 == nullptr) ||
      (workspace == nullptr && lowrank_workspace(M, R) > 0) ||
      (epilogue == SIXBIT_EPI_RESIDUAL && residual == nullptr))
    return SIXBIT_EINVAL;
  if (!aligned16(x_bf16) || !aligned16(lr_a) || !aligned16(lr_b) || !aligned16(workspace) || !aligned_to(alpha, 4) ||
      !aligned_to(ids, 4) || !aligned_to(base, 2) || !aligned_to(base_f32, 4) || !aligned_to(residual, 2) ||
      !aligned_to(Y, 2) || !aligned_to(Y_f32, 4) ||
      (x_bf16 == nullptr && (!aligned16(A->i8_codes) || !aligned_to(A->row_scale, 4))))
    return SIXBIT_EALIGN;
  const sixbit_status s = check_device();
  if (s != SIXBIT_OK) return s;
  LowRankParams p{};
  p.x = x_bf16;
  if (x_bf16 == nullptr) {
    p.codes = A->i8_codes;
    p.row_scale = A->row_scale;
  }
  p.a = lr_a;
  p.b = lr_b;
  p.alpha = alpha;
  p.ids = ids;
  p.M = M;
  p.N = N;
  p.K = K;
  p.R = R;
  p.L = L;
  p.base = base;
  p.base_f32 = base_f32;
  p.epilogue = epilogue;
  p.residual = epilogue == SIXBIT_EPI_RESIDUAL ? residual : nullptr;
  p.Y = Y_f32 != nullptr ? nullptr : Y;
  p.Yf = Y_f32;
  p.mode_dev = mode_dev;
  p.err = err_dev;
  return cuda_status(launch_lowrank(p, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
