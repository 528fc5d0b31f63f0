// qattn_api.cu -- the C ABI (include/qattn.h): argument checks, device checks, launches.
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "launch.h"
#include "qattn.h"
#include "sm100_ptx.cuh"


// The device error word (one per device that loads the library).
static __device__ int g_qattn_error = 0;

namespace {

constexpr int kMaxDevices = 64;
constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
constexpr int kMaxRows = 1 << 30;       // rows, tokens, heads, columns: what the kernels round up stays an int
constexpr int64_t kMaxRowStride = (int64_t{1} << 40) - 16;   // row stride of a TMA map, in bytes

struct DeviceInfo {
  cudaError_t setup = cudaSuccess;   // error of the set-up below, if any
  bool supported = false;
  int num_sms = 0;
  int* err = nullptr;
};
DeviceInfo g_dev[kMaxDevices];
std::once_flag g_dev_once[kMaxDevices];
uint64_t g_timeout_ns = kDefaultTimeoutNs;
qattn::DebugHooks g_dbg;          // test hooks (qattn_debug_*)

thread_local int t_last_cuda_error = 0;   // qattn_last_cuda_error: per calling host thread

qattn_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return QATTN_OK;
  t_last_cuda_error = static_cast<int>(e);
  return QATTN_ERR_CUDA;
}

// Per-device set-up on first use, once per device and thread-safe (std::call_once): capability
// check, SM count, device address of the error word.  Callers on other threads wait for it.
qattn_status device_info(DeviceInfo** out) {
  int dev = 0;
  const cudaError_t ge = cudaGetDevice(&dev);
  if (ge != cudaSuccess) return from_cuda(ge);
  if (dev < 0 || dev >= kMaxDevices) return QATTN_ERR_CUDA;
  DeviceInfo& d = g_dev[dev];
  std::call_once(g_dev_once[dev], [&d, dev] {
    int major = 0, minor = 0, sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    d.supported = e == cudaSuccess && major == 10 && minor == 0;
    d.num_sms = sms;
    if (e == cudaSuccess && d.supported) {
      void* p = nullptr;
      e = cudaGetSymbolAddress(&p, g_qattn_error);
      d.err = static_cast<int*>(p);
    }
    d.setup = e;
  });
  if (d.setup != cudaSuccess) return from_cuda(d.setup);
  if (!d.supported) return QATTN_ERR_UNSUPPORTED;
  *out = &d;
  return QATTN_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }


qattn_status check_attention_common(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                                    const void* out, int H, int D, const qattn_scales* sc,
                                    float sm_scale, qattn_mode mode) {
  if (!q8 || !k8 || !v8 || !out || !sc || !sc->s_q || !sc->s_k || !sc->s_v)
    return QATTN_ERR_INVALID_ARG;
  if (!aligned(q8, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(out, 16))
    return QATTN_ERR_INVALID_ARG;
  if (H < 1 || !(sm_scale > 0.0f) || !(sm_scale < 3.0e38f)) return QATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return QATTN_ERR_UNSUPPORTED;
  const int base = static_cast<int>(mode) & ~static_cast<int>(QATTN_FLAG_P_UNQUANTIZED);
  if (base != QATTN_MODE_FP8 && base != QATTN_MODE_FP4) return QATTN_ERR_INVALID_ARG;
  return QATTN_OK;
}

qattn_status check_quant_rows(const void* x, int64_t ldx, qattn_dtype dtype, int M, int K, const int8_t* out,
                              int64_t ldo, const float* scale) {
  if (!x || !out || !scale || M < 1 || K < 1 || ldx < K || ldo < K || ldo % 16 != 0) return QATTN_ERR_INVALID_ARG;
  if (dtype != QATTN_DTYPE_BF16 && dtype != QATTN_DTYPE_FP16) return QATTN_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(out, 16) || !aligned(scale, 4)) return QATTN_ERR_INVALID_ARG;
  if (ldx > kMaxRowStride || ldo > kMaxRowStride || M > kMaxRows || K > kMaxRows) return QATTN_ERR_UNSUPPORTED;
  return QATTN_OK;
}

// Whether two blocks of rows (`bytes` each, `stride` apart) may share memory.
bool rows_overlap(const void* a, int64_t rows_a, int64_t stride_a, int64_t bytes_a, const void* b, int64_t rows_b,
                  int64_t stride_b, int64_t bytes_b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>((rows_b - 1) * stride_b + bytes_b) &&
         b0 < a0 + static_cast<uintptr_t>((rows_a - 1) * stride_a + bytes_a);
}

qattn_status check_gemm_int8(const int8_t* a8, int64_t lda, const int8_t* b8, int64_t ldb, const void* y,
                             int64_t ldy, qattn_dtype dtype, int M, int N, int K, const float* s_a,
                             const float* s_b, const float* bias) {
  if (!a8 || !b8 || !y || !s_a || !s_b || M < 1 || N < 1 || K < 1) return QATTN_ERR_INVALID_ARG;
  if (lda < K || ldb < K || ldy < N || lda % 16 != 0 || ldb % 16 != 0) return QATTN_ERR_INVALID_ARG;
  if (dtype != QATTN_DTYPE_BF16 && dtype != QATTN_DTYPE_FP16) return QATTN_ERR_INVALID_ARG;
  if (!aligned(a8, 16) || !aligned(b8, 16) || !aligned(y, 2) || !aligned(s_a, 4) || !aligned(s_b, 4) ||
      (bias && !aligned(bias, 4)))
    return QATTN_ERR_INVALID_ARG;
  // |sum| <= K * 2^14 has to fit int32; tile counts have to fit an int
  if (K > QATTN_INT8_MAX_K || lda > kMaxRowStride || ldb > kMaxRowStride || ldy > kMaxRowStride) return QATTN_ERR_UNSUPPORTED;
  if (M > kMaxRows || N > kMaxRows || (static_cast<int64_t>(M) / 256 + 1) * (static_cast<int64_t>(N) / 64 + 1) > (1 << 30))
    return QATTN_ERR_UNSUPPORTED;
  return QATTN_OK;
}

bool p_unquantized(qattn_mode mode) {
  return (static_cast<int>(mode) & static_cast<int>(QATTN_FLAG_P_UNQUANTIZED)) != 0;
}

}  // namespace

extern "C" {

qattn_status qattn_calibrate_amax(const void* x_bf16, size_t n, float* amax_dev,
                                  qattn_stream_t stream) {
  if (!x_bf16 || !amax_dev || n == 0 || !aligned(x_bf16, 16) || !aligned(amax_dev, 4))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_amax(x_bf16, n, amax_dev, d->err, d->num_sms,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_quantize_fp8(const void* x_bf16, size_t n, const float* amax_dev,
                                uint8_t* out_e4m3, float* scale_dev, qattn_stream_t stream) {
  if (!x_bf16 || !amax_dev || !out_e4m3 || !scale_dev || n == 0) return QATTN_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(out_e4m3, 8) || !aligned(amax_dev, 4) ||
      !aligned(scale_dev, 4))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_quant_fp8(x_bf16, n, amax_dev, out_e4m3, scale_dev, d->err,
                                           d->num_sms, reinterpret_cast<cudaStream_t>(stream),
                                           g_dbg.inject_oob));
}

qattn_status qattn_quantize_fp4_block(const void* x_bf16, size_t n, const float* amax_dev,
                                      uint8_t* out_e2m1, uint8_t* blk_scale_e4m3,
                                      float* gscale_dev, uint8_t* out_e4m3_requant,
                                      float* scale8_dev, qattn_stream_t stream) {
  if (!x_bf16 || !amax_dev || !out_e2m1 || !blk_scale_e4m3 || !gscale_dev || n == 0 ||
      n % 16 != 0)
    return QATTN_ERR_INVALID_ARG;
  if ((out_e4m3_requant == nullptr) != (scale8_dev == nullptr)) return QATTN_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(out_e2m1, 8) || !aligned(amax_dev, 4) ||
      !aligned(gscale_dev, 4) || (out_e4m3_requant && !aligned(out_e4m3_requant, 16)) ||
      (scale8_dev && !aligned(scale8_dev, 4)))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_quant_fp4_block(x_bf16, n, amax_dev, out_e2m1, blk_scale_e4m3,
                                                 gscale_dev, out_e4m3_requant, scale8_dev, d->err,
                                                 d->num_sms,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_calibrate_quantize_fp8(const void* x_bf16, size_t n, float* amax_dev,
                                          uint8_t* out_e4m3, float* scale_dev,
                                          void* workspace_dev, size_t workspace_bytes,
                                          qattn_stream_t stream) {
  if (!x_bf16 || !amax_dev || !out_e4m3 || !scale_dev || !workspace_dev || n == 0)
    return QATTN_ERR_INVALID_ARG;
  if (workspace_bytes < QATTN_FUSED_WORKSPACE_BYTES || !aligned(workspace_dev, 16))
    return QATTN_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(out_e4m3, 8) || !aligned(amax_dev, 4) ||
      !aligned(scale_dev, 4))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_calib_quant_fp8(x_bf16, n, amax_dev, out_e4m3, scale_dev,
                                                 workspace_dev, g_timeout_ns, d->err, d->num_sms,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_calibrate_quantize_fp4_block(const void* x_bf16, size_t n, float* amax_dev,
                                                uint8_t* out_e2m1, uint8_t* blk_scale_e4m3,
                                                float* gscale_dev, uint8_t* out_e4m3_requant,
                                                float* scale8_dev, void* workspace_dev,
                                                size_t workspace_bytes, qattn_stream_t stream) {
  if (!x_bf16 || !amax_dev || !out_e2m1 || !blk_scale_e4m3 || !gscale_dev || !workspace_dev ||
      n == 0 || n % 16 != 0)
    return QATTN_ERR_INVALID_ARG;
  if ((out_e4m3_requant == nullptr) != (scale8_dev == nullptr)) return QATTN_ERR_INVALID_ARG;
  if (workspace_bytes < QATTN_FUSED_WORKSPACE_BYTES || !aligned(workspace_dev, 16))
    return QATTN_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(out_e2m1, 8) || !aligned(amax_dev, 4) ||
      !aligned(gscale_dev, 4) || (out_e4m3_requant && !aligned(out_e4m3_requant, 16)) ||
      (scale8_dev && !aligned(scale8_dev, 4)))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_calib_quant_fp4_block(
      x_bf16, n, amax_dev, out_e2m1, blk_scale_e4m3, gscale_dev, out_e4m3_requant, scale8_dev,
      workspace_dev, g_timeout_ns, d->err, d->num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_calibrate_quantize_qkv(const qattn_quant_io* io, size_t n, qattn_mode mode,
                                          void* workspace_dev, size_t workspace_bytes,
                                          qattn_stream_t stream) {
  if (!io || n == 0 || !workspace_dev) return QATTN_ERR_INVALID_ARG;
  if (mode != QATTN_MODE_FP8 && mode != QATTN_MODE_FP4) return QATTN_ERR_INVALID_ARG;
  if (mode == QATTN_MODE_FP4 && n % 16 != 0) return QATTN_ERR_INVALID_ARG;
  if (workspace_bytes < QATTN_FUSED_WORKSPACE_BYTES || !aligned(workspace_dev, 16))
    return QATTN_ERR_INVALID_ARG;
  const void* x[3];
  uint8_t *c8[3], *e2m1[3], *bs[3];
  float *am[3], *sc[3], *gs[3];
  for (int i = 0; i < 3; ++i) {
    const qattn_quant_io& t = io[i];
    if (!t.x_bf16 || !t.out_e4m3 || !t.amax_dev || !t.scale_dev) return QATTN_ERR_INVALID_ARG;
    if (!aligned(t.x_bf16, 16) || !aligned(t.amax_dev, 4) || !aligned(t.scale_dev, 4) ||
        !aligned(t.out_e4m3, mode == QATTN_MODE_FP4 ? 16 : 8))
      return QATTN_ERR_INVALID_ARG;
    if (mode == QATTN_MODE_FP4 && (!t.out_e2m1 || !t.blk_scale_e4m3 || !t.gscale_dev ||
                                   !aligned(t.out_e2m1, 8) || !aligned(t.gscale_dev, 4)))
      return QATTN_ERR_INVALID_ARG;
    x[i] = t.x_bf16;
    c8[i] = t.out_e4m3;
    am[i] = t.amax_dev;
    sc[i] = t.scale_dev;
    e2m1[i] = mode == QATTN_MODE_FP4 ? t.out_e2m1 : nullptr;
    bs[i] = mode == QATTN_MODE_FP4 ? t.blk_scale_e4m3 : nullptr;
    gs[i] = mode == QATTN_MODE_FP4 ? t.gscale_dev : nullptr;
  }
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_calib_quant_qkv(x, c8, am, sc, e2m1, bs, gs, n,
                                                 mode == QATTN_MODE_FP4 ? 1 : 0, workspace_dev,
                                                 g_timeout_ns, d->err, d->num_sms,
                                                 reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_quantize_qkv(const qattn_quant_io* io, size_t n, qattn_mode mode,
                                qattn_stream_t stream) {
  if (!io || n == 0) return QATTN_ERR_INVALID_ARG;
  if (mode != QATTN_MODE_FP8 && mode != QATTN_MODE_FP4) return QATTN_ERR_INVALID_ARG;
  if (mode == QATTN_MODE_FP4 && n % 16 != 0) return QATTN_ERR_INVALID_ARG;
  const void* x[3];
  uint8_t *c8[3], *e2m1[3], *bs[3];
  float *am[3], *sc[3], *gs[3];
  for (int i = 0; i < 3; ++i) {
    const qattn_quant_io& t = io[i];
    if (!t.x_bf16 || !t.out_e4m3 || !t.amax_dev || !t.scale_dev) return QATTN_ERR_INVALID_ARG;
    if (!aligned(t.x_bf16, 16) || !aligned(t.amax_dev, 4) || !aligned(t.scale_dev, 4) ||
        !aligned(t.out_e4m3, mode == QATTN_MODE_FP4 ? 16 : 8))
      return QATTN_ERR_INVALID_ARG;
    if (mode == QATTN_MODE_FP4 && (!t.out_e2m1 || !t.blk_scale_e4m3 || !t.gscale_dev ||
                                   !aligned(t.out_e2m1, 8) || !aligned(t.gscale_dev, 4)))
      return QATTN_ERR_INVALID_ARG;
    x[i] = t.x_bf16;
    c8[i] = t.out_e4m3;
    am[i] = t.amax_dev;
    sc[i] = t.scale_dev;
    e2m1[i] = mode == QATTN_MODE_FP4 ? t.out_e2m1 : nullptr;
    bs[i] = mode == QATTN_MODE_FP4 ? t.blk_scale_e4m3 : nullptr;
    gs[i] = mode == QATTN_MODE_FP4 ? t.gscale_dev : nullptr;
  }
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_quant_qkv(x, c8, am, sc, e2m1, bs, gs, n,
                                           mode == QATTN_MODE_FP4 ? 1 : 0, d->err, d->num_sms,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_gemm_fp8(const uint8_t* a8, const uint8_t* b8, void* y_bf16, int M, int N,
                            int K, const float* s_a_dev, const float* s_b_dev,
                            qattn_stream_t stream) {
  if (!a8 || !b8 || !y_bf16 || !s_a_dev || !s_b_dev) return QATTN_ERR_INVALID_ARG;
  if (M < 1 || N < 32 || K < 128 || N % 32 != 0 || K % 128 != 0) return QATTN_ERR_INVALID_ARG;
  if (!aligned(a8, 16) || !aligned(b8, 16) || !aligned(y_bf16, 16) || !aligned(s_a_dev, 4) ||
      !aligned(s_b_dev, 4))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_gemm_fp8(a8, b8, y_bf16, M, N, K, s_a_dev, s_b_dev, d->err,
                                          g_timeout_ns, d->num_sms,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_gemm_fp8_e4m3(const uint8_t* a8, const uint8_t* b8, void* y_bf16,
                                 uint8_t* codes_out, int M, int N, int K, const float* s_a_dev,
                                 const float* s_b_dev, const float* amax_dev, float* scale_out_dev,
                                 qattn_stream_t stream) {
  if (!a8 || !b8 || !codes_out || !s_a_dev || !s_b_dev || !amax_dev || !scale_out_dev)
    return QATTN_ERR_INVALID_ARG;
  if (M < 1 || N < 32 || K < 128 || N % 32 != 0 || K % 128 != 0) return QATTN_ERR_INVALID_ARG;
  if (!aligned(a8, 16) || !aligned(b8, 16) || (y_bf16 && !aligned(y_bf16, 16)) ||
      !aligned(codes_out, 16) || !aligned(s_a_dev, 4) || !aligned(s_b_dev, 4) ||
      !aligned(amax_dev, 4) || !aligned(scale_out_dev, 4))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_gemm_fp8(a8, b8, y_bf16, M, N, K, s_a_dev, s_b_dev, d->err,
                                          g_timeout_ns, d->num_sms,
                                          reinterpret_cast<cudaStream_t>(stream), codes_out,
                                          amax_dev, scale_out_dev));
}

qattn_status qattn_gemm_fp4(const uint8_t* x_e2m1, const uint8_t* x_bscale, const float* sg_x_dev,
                           const uint8_t* w_e2m1, const uint8_t* w_bscale, const float* sg_w_dev,
                           void* y_bf16, int M, int N, int K, qattn_stream_t stream) {
  if (!x_e2m1 || !x_bscale || !sg_x_dev || !w_e2m1 || !w_bscale || !sg_w_dev || !y_bf16)
    return QATTN_ERR_INVALID_ARG;
  if (M < 1 || N < 32 || K < 256 || N % 32 != 0 || K % 256 != 0) return QATTN_ERR_INVALID_ARG;
  if (!aligned(x_e2m1, 16) || !aligned(w_e2m1, 16) || !aligned(x_bscale, 16) ||
      !aligned(w_bscale, 16) || !aligned(y_bf16, 16) || !aligned(sg_x_dev, 4) || !aligned(sg_w_dev, 4))
    return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_gemm_fp4(x_e2m1, x_bscale, sg_x_dev, w_e2m1, w_bscale, sg_w_dev,
                                          y_bf16, M, N, K, d->err, g_timeout_ns, d->num_sms,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_forward_ws(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                              void* out_bf16, int B, int H, int L, int D,
                              const qattn_scales* scales, float sm_scale, qattn_mode mode,
                              void* workspace_dev, size_t workspace_bytes, qattn_stream_t stream) {
  qattn_status st = check_attention_common(q8, k8, v8, out_bf16, H, D, scales, sm_scale, mode);
  if (st != QATTN_OK) return st;
  if (B < 1 || L < 1) return QATTN_ERR_INVALID_ARG;
  if (B > 65535 || H > 65535) return QATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * H * L * D >= (int64_t(1) << 40)) return QATTN_ERR_UNSUPPORTED;
  if (workspace_dev != nullptr && !aligned(workspace_dev, 16)) return QATTN_ERR_INVALID_ARG;
  DeviceInfo* d = nullptr;
  st = device_info(&d);
  if (st != QATTN_OK) return st;
  if (workspace_dev != nullptr &&
      workspace_bytes < qattn::attention_plan(B, H, L, D, d->num_sms, g_dbg.attn_pair != 0).bytes)
    return QATTN_ERR_INVALID_ARG;
  if (p_unquantized(mode)) {
    if (static_cast<int64_t>(B) * H > 65535) return QATTN_ERR_UNSUPPORTED;
    return from_cuda(qattn::launch_attention_p_unquantized(
        q8, k8, v8, out_bf16, B, H, L, D, nullptr, 0, L, L, scales->s_q, scales->s_k, scales->s_v,
        sm_scale, reinterpret_cast<cudaStream_t>(stream)));
  }
  return from_cuda(qattn::launch_attention(q8, k8, v8, out_bf16, B, H, L, D, nullptr, 0, L, L,
                                           scales->s_q, scales->s_k, scales->s_v, sm_scale,
                                           d->err, g_timeout_ns, g_dbg,
                                           workspace_dev, workspace_bytes, d->num_sms,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_rope_table(const void* pos_dev, qattn_pos_type pos_type, int64_t pos_stride,
                              int tokens, int n_axes, const int* axis_dims, const double* theta,
                              float* table_dev, qattn_stream_t stream) {
  if (!pos_dev || !axis_dims || !theta || !table_dev || tokens < 1) return QATTN_ERR_INVALID_ARG;
  if (pos_type != QATTN_POS_INT32 && pos_type != QATTN_POS_FLOAT32) return QATTN_ERR_INVALID_ARG;
  if (n_axes < 1 || n_axes > QATTN_ROPE_MAX_AXES || pos_stride < n_axes) return QATTN_ERR_INVALID_ARG;
  if (!aligned(pos_dev, 4) || !aligned(table_dev, 16)) return QATTN_ERR_INVALID_ARG;
  if (tokens > kMaxRows) return QATTN_ERR_UNSUPPORTED;
  qattn::RopeFreqs f;
  int pairs = 0;
  for (int a = 0; a < n_axes; ++a) {
    const int d = axis_dims[a];
    if (d < 2 || d % 2 != 0 || d > QATTN_ROPE_MAX_DIM) return QATTN_ERR_INVALID_ARG;
    if (!(theta[a] >= 1.0) || !(theta[a] < 1e300)) return QATTN_ERR_INVALID_ARG;
    if (pairs + d / 2 > QATTN_ROPE_MAX_DIM / 2) return QATTN_ERR_UNSUPPORTED;
    // turns per unit of position, theta^(-2 i / d) / (2 pi) <= 0.16, times 2^64: powers of the first ratio in
    // 64 bits of mantissa (a power for each pair took 13 us of a 14 us call)
    const long double ratio = std::pow(static_cast<long double>(theta[a]), -2.0L / d);
    long double turns = 0.159154943091895335769L;
    for (int i = 0; i < d / 2; ++i, ++pairs, turns *= ratio) {
      f.pair[pairs].turns = static_cast<uint64_t>(turns * 18446744073709551616.0L + 0.5L);
      f.pair[pairs].axis = a;
    }
  }
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_rope_table(pos_dev, pos_type == QATTN_POS_FLOAT32, pos_stride, tokens,
                                            n_axes, pairs, f, table_dev, d->err, d->num_sms,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_norm_rope(const qattn_norm_rope_io* io, int n_io, int B, int D, int rotary_dim,
                             int interleaved, float eps, qattn_dtype dtype, qattn_stream_t stream) {
  if (!io || n_io < 1 || B < 1) return QATTN_ERR_INVALID_ARG;
  if (n_io > QATTN_NORM_ROPE_MAX_IO) return QATTN_ERR_UNSUPPORTED;
  if (dtype != QATTN_DTYPE_BF16 && dtype != QATTN_DTYPE_FP16) return QATTN_ERR_INVALID_ARG;
  if (D < 8 || D % 8 != 0 || rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0)
    return QATTN_ERR_INVALID_ARG;
  if (D > QATTN_ROPE_MAX_DIM) return QATTN_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || !(eps < 3.0e38f)) return QATTN_ERR_INVALID_ARG;
  qattn::NormRopeArgs a;
  for (int i = 0; i < n_io; ++i) {
    const qattn_norm_rope_io& t = io[i];
    qattn::NormRopeSeg& s = a.seg[i];
    if (!t.x || !t.out || t.H < 1 || t.L < 1) return QATTN_ERR_INVALID_ARG;
    if (t.H > kMaxRows || t.L > kMaxRows) return QATTN_ERR_UNSUPPORTED;
    if (!aligned(t.x, 16) || (t.weight && !aligned(t.weight, 16)) || (t.table && !aligned(t.table, 16)) ||
        (t.amax && !aligned(t.amax, 4)))
      return QATTN_ERR_INVALID_ARG;
    if ((t.x_stride_b | t.x_stride_t | t.x_stride_h | t.out_stride_b | t.out_stride_h | t.out_stride_t) % 8 != 0)
      return QATTN_ERR_INVALID_ARG;
    if (t.table && (rotary_dim == 0 || t.table_stride_b % 4 != 0)) return QATTN_ERR_INVALID_ARG;
    // rows of the output must not share elements
    if ((B > 1 && t.out_stride_b == 0) || (t.H > 1 && t.out_stride_h == 0) || (t.L > 1 && t.out_stride_t == 0))
      return QATTN_ERR_INVALID_ARG;
    if (t.out_e4m3) {
      if (!t.amax || !t.scale_out || !aligned(t.scale_out, 4) || !aligned(t.out, 8)) return QATTN_ERR_INVALID_ARG;
    } else if (!aligned(t.out, 16)) {
      return QATTN_ERR_INVALID_ARG;
    }
    s.x = t.x;
    s.out = t.out;
    s.weight = t.weight;
    s.table = t.table;
    s.amax = t.amax;
    s.scale_out = t.out_e4m3 ? t.scale_out : nullptr;
    s.x_b = t.x_stride_b;
    s.x_t = t.x_stride_t;
    s.x_h = t.x_stride_h;
    s.o_b = t.out_stride_b;
    s.o_h = t.out_stride_h;
    s.o_t = t.out_stride_t;
    s.table_b = t.table_stride_b;
    s.H = t.H;
    s.L = t.L;
    s.e4m3 = t.out_e4m3 != 0;
  }
  // No block may read as a given amax what another one writes (a scale, a running amax), nor two write different scales
  // to one place.  Tensors that share a running amax, or a given one and its scale, are fine.
  for (int i = 0; i < n_io; ++i) {
    const qattn::NormRopeSeg& s = a.seg[i];
    for (int j = 0; s.e4m3 && j < n_io; ++j) {
      const qattn::NormRopeSeg& t = a.seg[j];
      if (t.amax == s.scale_out || (!t.e4m3 && t.amax == s.amax)) return QATTN_ERR_INVALID_ARG;
      if (t.e4m3 && t.scale_out == s.scale_out && t.amax != s.amax) return QATTN_ERR_INVALID_ARG;
    }
  }
  a.n = n_io;
  a.D = D;
  a.R = rotary_dim;
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(D);
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  a.err = d->err;
  unsigned grid = 0;
  if (!qattn::plan_norm_rope(a, B, d->num_sms, &grid)) return QATTN_ERR_UNSUPPORTED;
  return from_cuda(qattn::launch_norm_rope(a, grid, interleaved != 0, dtype == QATTN_DTYPE_FP16,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_quantize_int8_rows(const void* x, int64_t ldx, qattn_dtype dtype, int M, int K,
                                      int8_t* out_int8, int64_t ldo, float* scale_dev,
                                      qattn_stream_t stream) {
  const qattn_status ck = check_quant_rows(x, ldx, dtype, M, K, out_int8, ldo, scale_dev);
  if (ck != QATTN_OK) return ck;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  return from_cuda(qattn::launch_quant_int8_rows(x, ldx, dtype == QATTN_DTYPE_FP16, M, K, out_int8, ldo,
                                                 scale_dev, d->err, reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_gemm_int8(const int8_t* a8, int64_t lda, const int8_t* b8, int64_t ldb, void* y,
                             int64_t ldy, qattn_dtype dtype, int M, int N, int K, const float* s_a_dev,
                             const float* s_b_dev, const float* bias_dev, qattn_stream_t stream) {
  const qattn_status ck = check_gemm_int8(a8, lda, b8, ldb, y, ldy, dtype, M, N, K, s_a_dev, s_b_dev, bias_dev);
  if (ck != QATTN_OK) return ck;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  const qattn::GemmInt8Args a{M, N, K, 1, 0, 0, 0, 0, ldy, s_a_dev, s_b_dev, bias_dev, y, d->err, g_timeout_ns};
  return from_cuda(qattn::launch_gemm_int8(a8, lda, b8, ldb, a, dtype == QATTN_DTYPE_FP16, d->num_sms,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_linear_int8(const void* x, int64_t ldx, qattn_dtype dtype, int M, int N, int K,
                               int8_t* x8, int64_t ldx8, float* s_x_dev, const int8_t* w8, int64_t ldw,
                               const float* s_w_dev, const float* bias_dev, void* y, int64_t ldy,
                               qattn_stream_t stream) {
  qattn_status ck = check_quant_rows(x, ldx, dtype, M, K, x8, ldx8, s_x_dev);
  if (ck == QATTN_OK)
    ck = check_gemm_int8(x8, ldx8, w8, ldw, y, ldy, dtype, M, N, K, s_x_dev, s_w_dev, bias_dev);
  if (ck != QATTN_OK) return ck;
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  const qattn::GemmInt8Args a{M, N, K, 1, 0, 0, 0, 0, ldy, s_x_dev, s_w_dev, bias_dev, y, d->err, g_timeout_ns};
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int fp16 = dtype == QATTN_DTYPE_FP16;
  // An output in the place of x, or weights, scales or a bias that are the quantize's own output, need the quantize to
  // be done first: the two launches then follow each other.
  const bool in_order = rows_overlap(y, M, 2 * ldy, 2 * int64_t{N}, x, M, 2 * ldx, 2 * int64_t{K}) ||
                        rows_overlap(w8, N, ldw, K, x8, M, ldx8, K) || rows_overlap(w8, N, ldw, K, s_x_dev, 1, 0, 4 * int64_t{M}) ||
                        rows_overlap(s_w_dev, 1, 0, 4 * int64_t{N}, s_x_dev, 1, 0, 4 * int64_t{M}) ||
                        rows_overlap(s_w_dev, 1, 0, 4 * int64_t{N}, x8, M, ldx8, K) ||
                        (bias_dev && (rows_overlap(bias_dev, 1, 0, 4 * int64_t{N}, s_x_dev, 1, 0, 4 * int64_t{M}) ||
                                      rows_overlap(bias_dev, 1, 0, 4 * int64_t{N}, x8, M, ldx8, K)));
  if (in_order) {
    st = from_cuda(qattn::launch_quant_int8_rows(x, ldx, fp16, M, K, x8, ldx8, s_x_dev, d->err, cs));
    if (st != QATTN_OK) return st;
    return from_cuda(qattn::launch_gemm_int8(x8, ldx8, w8, ldw, a, fp16, d->num_sms, cs));
  }
  return from_cuda(qattn::launch_linear_int8(x, ldx, x8, ldx8, s_x_dev, w8, ldw, a, fp16, d->num_sms, cs));
}

qattn_status qattn_forward(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                           void* out_bf16, int B, int H, int L, int D,
                           const qattn_scales* scales, float sm_scale, qattn_mode mode,
                           qattn_stream_t stream) {
  return qattn_forward_ws(q8, k8, v8, out_bf16, B, H, L, D, scales, sm_scale, mode, nullptr, 0,
                          stream);
}

size_t qattn_forward_workspace_bytes(int B, int H, int L, int D) {
  if (B < 1 || H < 1 || L < 1 || (D != 64 && D != 128)) return 0;
  DeviceInfo* d = nullptr;
  if (device_info(&d) != QATTN_OK) return 0;
  // enough for either D = 128 kernel, so a workspace stays valid if the variant is switched
  const size_t one_sm = qattn::attention_plan(B, H, L, D, d->num_sms, false).bytes;
  const size_t pair = D == 128 ? qattn::attention_plan(B, H, L, D, d->num_sms, true).bytes : 0;
  return one_sm > pair ? one_sm : pair;
}

qattn_status qattn_forward_varlen(const uint8_t* q8, const uint8_t* k8, const uint8_t* v8,
                                  void* out_bf16, const int* cu_seqlens_dev, int nseq,
                                  int max_seqlen, int total_tokens, int H, int D,
                                  const qattn_scales* scales, float sm_scale, qattn_mode mode,
                                  qattn_stream_t stream) {
  qattn_status st = check_attention_common(q8, k8, v8, out_bf16, H, D, scales, sm_scale, mode);
  if (st != QATTN_OK) return st;
  if (!cu_seqlens_dev || !aligned(cu_seqlens_dev, 4) || nseq < 1 || max_seqlen < 1 ||
      total_tokens < 1 || max_seqlen > total_tokens)
    return QATTN_ERR_INVALID_ARG;
  if (nseq > 65535 || H > 65535) return QATTN_ERR_UNSUPPORTED;
  DeviceInfo* d = nullptr;
  st = device_info(&d);
  if (st != QATTN_OK) return st;
  if (p_unquantized(mode))
    return from_cuda(qattn::launch_attention_p_unquantized(
        q8, k8, v8, out_bf16, 1, H, 0, D, cu_seqlens_dev, nseq, max_seqlen, total_tokens,
        scales->s_q, scales->s_k, scales->s_v, sm_scale, reinterpret_cast<cudaStream_t>(stream)));
  return from_cuda(qattn::launch_attention(q8, k8, v8, out_bf16, 1, H, 0, D, cu_seqlens_dev,
                                           nseq, max_seqlen, total_tokens, scales->s_q,
                                           scales->s_k, scales->s_v, sm_scale, d->err,
                                           g_timeout_ns, g_dbg, nullptr, 0,
                                           d->num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

qattn_status qattn_get_error(qattn_stream_t stream) {
  DeviceInfo* d = nullptr;
  qattn_status st = device_info(&d);
  if (st != QATTN_OK) return st;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return QATTN_ERR_CUDA;
  int word = 0;
  if (cudaMemcpyFromSymbol(&word, g_qattn_error, sizeof(int)) != cudaSuccess) return QATTN_ERR_CUDA;
  if (word != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_qattn_error, &zero, sizeof(int)) != cudaSuccess)
      return QATTN_ERR_CUDA;
  }
  switch (word) {
    case 0: return QATTN_OK;
    case qattn::DEV_ERR_NONFINITE: return QATTN_ERR_NONFINITE;
    case qattn::DEV_ERR_TIMEOUT: return QATTN_ERR_TIMEOUT;
    case qattn::DEV_ERR_BOUNDS: return QATTN_ERR_BOUNDS;
    default: return QATTN_ERR_CUDA;
  }
}

int qattn_last_cuda_error(void) { return t_last_cuda_error; }

const char* qattn_status_str(qattn_status status) {
  switch (status) {
    case QATTN_OK: return "QATTN_OK";
    case QATTN_ERR_INVALID_ARG: return "QATTN_ERR_INVALID_ARG";
    case QATTN_ERR_UNSUPPORTED: return "QATTN_ERR_UNSUPPORTED";
    case QATTN_ERR_CUDA: return "QATTN_ERR_CUDA";
    case QATTN_ERR_NONFINITE: return "QATTN_ERR_NONFINITE";
    case QATTN_ERR_TIMEOUT: return "QATTN_ERR_TIMEOUT";
    case QATTN_ERR_BOUNDS: return "QATTN_ERR_BOUNDS";
  }
  return "QATTN_ERR_UNKNOWN";
}

void qattn_debug_set_wait_timeout_ns(uint64_t ns) {
  g_timeout_ns = ns ? ns : kDefaultTimeoutNs;
}

void qattn_debug_inject_missing_q(int enable) { g_dbg.inject_missing_q = enable ? 1 : 0; }

void qattn_debug_use_pair_kernel(int enable) { g_dbg.attn_pair = enable ? 1 : 0; }

int qattn_build_info(void) {
#ifdef QATTN_CHECKED
  return 1;
#else
  return 0;
#endif
}

qattn_status qattn_debug_inject_oob(int enable) {
#ifdef QATTN_CHECKED
  g_dbg.inject_oob = enable ? 1 : 0;
  return QATTN_OK;
#else
  (void)enable;
  return QATTN_ERR_UNSUPPORTED;
#endif
}

qattn_status qattn_debug_capture_p_row(int enable, int slab, int row, uint8_t* codes_dev,
                                       int* maxima_dev) {
  if (!enable) {
    g_dbg.p_codes = nullptr;
    g_dbg.p_maxima = nullptr;
    g_dbg.p_slab = g_dbg.p_row = -1;
    return QATTN_OK;
  }
  if (!codes_dev || !maxima_dev || !aligned(codes_dev, 16) || !aligned(maxima_dev, 4) || slab < 0 ||
      row < 0)
    return QATTN_ERR_INVALID_ARG;
  g_dbg.p_codes = codes_dev;
  g_dbg.p_maxima = maxima_dev;
  g_dbg.p_slab = slab;
  g_dbg.p_row = row;
  return QATTN_OK;
}

qattn_status qattn_debug_attention_plan(int B, int H, int L, int D, int num_sms, int* plan,
                                        size_t* workspace_bytes) {
  if (B < 1 || H < 1 || L < 1 || (D != 64 && D != 128) || num_sms < 1 || !plan ||
      !workspace_bytes)
    return QATTN_ERR_INVALID_ARG;
  const qattn::AttnSplitPlan p = qattn::plan_attention_split(B, H, L, D, num_sms);
  plan[0] = p.pairs_per_head;
  plan[1] = p.nkv;
  plan[2] = p.ctas;
  plan[3] = p.whole;
  plan[4] = p.tail_pairs;
  plan[5] = p.tail_w;
  *workspace_bytes = p.bytes;
  return QATTN_OK;
}

}  // extern "C"
