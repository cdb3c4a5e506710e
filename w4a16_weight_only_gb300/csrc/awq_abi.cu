// C ABI of libawq_gb300.so (declared in include/awq.h): host-side validation, error
// reporting and kernel-family dispatch.  All argument checks run on the host before any
// CUDA call, so an invalid call touches no device.
#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/awq.h"
#include "awq_internal.cuh"
#include "awq_layer.cuh"
#include "awq_step.cuh"

namespace {

thread_local std::string g_err;
thread_local bool g_waits_give_up = false;  // awq_selftest_attention_give_up

awq_status_t fail(awq_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

awq_status_t ok() {
  g_err.clear();
  return AWQ_OK;
}

awq_status_t cuda_fail(cudaError_t e, const char* what) {
  return fail(AWQ_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr int64_t kDimLimit = (int64_t{1} << 31) - 1;
constexpr int64_t kProdLimit = int64_t{1} << 40;

// Shape rules shared by awq_dequant and awq_gemm.  Returns AWQ_OK and the resolved G.
awq_status_t check_weight_shape(int64_t K, int64_t N, int64_t group_size, int* G_out,
                                int per_word = 8) {
  if (K <= 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "K must be positive (got %lld)", (long long)K);
  if (N < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "N must be >= 0 (got %lld)", (long long)N);
  if (group_size == 0 || group_size < -1)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "group_size must be -1 or positive (got %lld)",
                (long long)group_size);
  if (K > kDimLimit || N > kDimLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "K and N must be below 2^31");
  if (K * N >= kProdLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "K*N must be below 2^40");
  if (N % per_word != 0)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "N=%lld is not a multiple of %d (codes per int32 word)",
                (long long)N, per_word);
  const int64_t G = group_size == -1 ? K : group_size;
  if (K % G != 0)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "K=%lld is not a multiple of group_size=%lld",
                (long long)K, (long long)G);
  *G_out = static_cast<int>(G);
  return AWQ_OK;
}

// Current device must be compute capability 10.3 (the only code this library carries).
awq_status_t check_device() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(AWQ_ERR_UNSUPPORTED_DEVICE, "no CUDA device: %s", cudaGetErrorString(e));
  int major = 0, minor = 0;
  e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  if (major != 10 || minor != 3)
    return fail(AWQ_ERR_UNSUPPORTED_DEVICE,
                "device %d is compute capability %d.%d; this library is built for 10.3 (sm_103a)",
                dev, major, minor);
  return AWQ_OK;
}

bool al(const void* p, uintptr_t a) { return awq::aligned(p, a); }

awq_status_t build_problem(const void* x, const int32_t* qweight, const int32_t* qzeros,
                           const void* scales, const void* bias, int64_t M, int64_t K, int64_t N,
                           int64_t group_size, void* y, awq_stream_t stream, awq::GemmProblem* p,
                           bool* empty, bool bf16 = false, int bits = 4) {
  if (M < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "M must be >= 0 (got %lld)", (long long)M);
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G, bits == 8 ? 4 : 8);
  if (st != AWQ_OK) return st;
  if (M > kDimLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "M must be below 2^31");
  if (M * N >= kProdLimit || M * K >= kProdLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "M*N and M*K must be below 2^40");
  *empty = (M == 0 || N == 0);
  if (*empty) return AWQ_OK;
  if (!x || !qweight || !qzeros || !scales || !y)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "null pointer among x, qweight, qzeros, scales, y");
  if (!al(x, 2) || !al(scales, 2) || !al(y, 2) || (bias && !al(bias, 2)))
    return fail(AWQ_ERR_MISALIGNED, "16-bit tensors must be 2-byte aligned");
  if (!al(qweight, 4) || !al(qzeros, 4))
    return fail(AWQ_ERR_MISALIGNED, "qweight and qzeros must be 4-byte aligned");
  p->x = static_cast<const __half*>(x);
  p->qw = reinterpret_cast<const uint32_t*>(qweight);
  p->qz = reinterpret_cast<const uint32_t*>(qzeros);
  p->sc = static_cast<const __half*>(scales);
  p->bias = static_cast<const __half*>(bias);
  p->y = static_cast<__half*>(y);
  p->M = static_cast<int>(M);
  p->K = static_cast<int>(K);
  p->N = static_cast<int>(N);
  p->G = G;
  p->stream = reinterpret_cast<cudaStream_t>(stream);
  p->bf16 = bf16;
  p->bits = bits;
  return AWQ_OK;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    (void)cudaGetLastError();
    return 152;
  }
  return sms;
}

// Above 32 rows both tensor-core families can run; estimates fitted to GB300 timings of
// both kernels on the 7B and 70B linears at M = 8 .. 512 pick the faster.  Decode: the
// first 32-row tile streams the weights (about 3 TB/s plus 8 us of launch chain), each
// further 32-row tile costs 0.25 ns per code (its unpack and MMAs; the weights come from
// L2).  Prefill: the estimate of the plan it would launch (awq_prefill.cu).
bool prefill_faster(const awq::GemmProblem& p) {
  const double kn = static_cast<double>(p.K) * static_cast<double>(p.N);
  const double weight_bytes = kn * p.bits / 8.0 + 3.0 * static_cast<double>(p.K / p.G) * p.N;
  const double row_tiles = static_cast<double>((p.M + 31) / 32);
  const double decode_us = weight_bytes / 3.0e6 + 8.0 + (row_tiles - 1.0) * kn * 2.5e-7;
  return awq::prefill_estimate_us(p, sm_count()) < decode_us;
}

awq::Path choose_path(const awq::GemmProblem& p) {
  const bool dec = awq::decode_supported(p, nullptr);
  if (p.M <= 32 && dec) return awq::kDecode;
  const bool pre = awq::prefill_supported(p, nullptr);
  if (pre && dec) return prefill_faster(p) ? awq::kPrefill : awq::kDecode;
  if (pre) return awq::kPrefill;
  if (dec) return awq::kDecode;
  return awq::kGeneric;
}

awq_status_t run(const awq::GemmProblem& p, awq::Path path) {
  const char* why = "";
  cudaError_t e = cudaSuccess;
  switch (path) {
    case awq::kDecode:
      if (!awq::decode_supported(p, &why)) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "decode path: %s", why);
      e = awq::launch_decode(p);
      break;
    case awq::kPrefill:
      if (!awq::prefill_supported(p, &why)) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "prefill path: %s", why);
      e = awq::launch_prefill(p);
      break;
    case awq::kGeneric:
      e = awq::launch_generic(p);
      break;
    default:
      return fail(AWQ_ERR_INVALID_ARGUMENT, "unknown path %d", static_cast<int>(path));
  }
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

}  // namespace

extern "C" {

int awq_runtime_available(void) {
  if (check_device() != AWQ_OK) return 0;
  cudaFuncAttributes attr;
  const cudaError_t e = awq::probe_kernel_image(&attr);
  if (e != cudaSuccess) {
    cuda_fail(e, "loading sm_103a kernels");
    return 0;
  }
  ok();
  return 1;
}

const char* awq_last_error(void) { return g_err.c_str(); }

const char* awq_status_string(awq_status_t s) {
  switch (s) {
    case AWQ_OK: return "AWQ_OK";
    case AWQ_ERR_INVALID_ARGUMENT: return "AWQ_ERR_INVALID_ARGUMENT";
    case AWQ_ERR_UNSUPPORTED_SHAPE: return "AWQ_ERR_UNSUPPORTED_SHAPE";
    case AWQ_ERR_MISALIGNED: return "AWQ_ERR_MISALIGNED";
    case AWQ_ERR_UNSUPPORTED_DEVICE: return "AWQ_ERR_UNSUPPORTED_DEVICE";
    case AWQ_ERR_CUDA: return "AWQ_ERR_CUDA";
    case AWQ_ERR_TIMEOUT: return "AWQ_ERR_TIMEOUT";
  }
  return "AWQ_ERR_UNKNOWN";
}

awq_status_t awq_dequant(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                         int64_t K, int64_t N, int64_t group_size, void* w_out,
                         awq_dtype_t out_dtype, awq_stream_t stream) {
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G);
  if (st != AWQ_OK) return st;
  if (out_dtype != AWQ_DTYPE_F16 && out_dtype != AWQ_DTYPE_F32)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "out_dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_F32");
  if (N == 0) return ok();
  if (!qweight || !qzeros || !scales_f16 || !w_out)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "null pointer among qweight, qzeros, scales, w_out");
  if (!al(qweight, 4) || !al(qzeros, 4)) return fail(AWQ_ERR_MISALIGNED, "qweight/qzeros must be 4-byte aligned");
  if (!al(scales_f16, 2)) return fail(AWQ_ERR_MISALIGNED, "scales must be 2-byte aligned");
  if (!al(w_out, out_dtype == AWQ_DTYPE_F32 ? 4 : 2)) return fail(AWQ_ERR_MISALIGNED, "w_out misaligned for its dtype");
  st = check_device();
  if (st != AWQ_OK) return st;
  const cudaError_t e = awq::launch_dequant(
      reinterpret_cast<const uint32_t*>(qweight), reinterpret_cast<const uint32_t*>(qzeros),
      static_cast<const __half*>(scales_f16), static_cast<int>(K), static_cast<int>(N), G, w_out,
      out_dtype == AWQ_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "awq_dequant launch");
  return ok();
}

awq_status_t awq_quantize_rtn(const void* w_f16, int64_t N, int64_t K, int64_t group_size,
                              int sym, int32_t* qweight, int32_t* qzeros, void* scales_f16,
                              awq_stream_t stream) {
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G);
  if (st != AWQ_OK) return st;
  if (sym != 0 && sym != 1) return fail(AWQ_ERR_INVALID_ARGUMENT, "sym must be 0 or 1 (got %d)", sym);
  if (G % 8 != 0)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "group size %d is not a multiple of 8 (16-byte group rows)", G);
  if (K / G > 65535) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "K / group_size must be at most 65535");
  if (N == 0) return ok();
  if (!w_f16 || !qweight || !qzeros || !scales_f16)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "null pointer among w, qweight, qzeros, scales");
  if (!al(w_f16, 16)) return fail(AWQ_ERR_MISALIGNED, "w must be 16-byte aligned");
  if (!al(qweight, 4) || !al(qzeros, 4)) return fail(AWQ_ERR_MISALIGNED, "qweight/qzeros must be 4-byte aligned");
  if (!al(scales_f16, 2)) return fail(AWQ_ERR_MISALIGNED, "scales must be 2-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  const cudaError_t e = awq::launch_quantize_rtn(
      static_cast<const __half*>(w_f16), static_cast<int>(N), static_cast<int>(K), G, sym == 1,
      reinterpret_cast<uint32_t*>(qweight), reinterpret_cast<uint32_t*>(qzeros),
      static_cast<__half*>(scales_f16), reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "awq_quantize_rtn launch");
  return ok();
}

static awq_status_t gemm_any(const void* x, const int32_t* qweight, const int32_t* qzeros,
                      const void* scales, const void* bias, int64_t M, int64_t K, int64_t N,
                      int64_t group_size, void* y, awq_path_t path, awq_stream_t stream, bool bf16,
                      int bits = 4, uint32_t flags = 0u) {
  if (path < AWQ_PATH_AUTO || path > AWQ_PATH_GENERIC)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "unknown path %d", static_cast<int>(path));
  if ((flags & ~static_cast<uint32_t>(AWQ_GEMM_STATIC_WEIGHTS)) != 0u)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "unknown flag bits 0x%x", flags);
  awq::GemmProblem p{};
  bool empty = false;
  awq_status_t st = build_problem(x, qweight, qzeros, scales, bias, M, K, N, group_size, y,
                                  stream, &p, &empty, bf16, bits);
  if (st != AWQ_OK) return st;
  if (empty) return ok();
  p.static_weights = (flags & AWQ_GEMM_STATIC_WEIGHTS) != 0u;
  st = check_device();
  if (st != AWQ_OK) return st;
  const awq::Path use = path == AWQ_PATH_AUTO ? choose_path(p) : static_cast<awq::Path>(path);
  return run(p, use);
}

awq_status_t awq_gemm_any(const void* x, const int32_t* qweight, const int32_t* qzeros,
                          const void* scales, const void* bias, int64_t M, int64_t K, int64_t N,
                          int64_t group_size, void* y, awq_dtype_t dtype, int32_t bits,
                          awq_path_t path, uint32_t flags, awq_stream_t stream) {
  if (dtype != AWQ_DTYPE_F16 && dtype != AWQ_DTYPE_BF16)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  if (bits != 4 && bits != 8) return fail(AWQ_ERR_INVALID_ARGUMENT, "bits must be 4 or 8 (got %d)", bits);
  if (bits == 8 && dtype != AWQ_DTYPE_F16)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "8-bit codes take fp16 activations and scales");
  return gemm_any(x, qweight, qzeros, scales, bias, M, K, N, group_size, y, path, stream,
                  dtype == AWQ_DTYPE_BF16, bits, flags);
}

awq_status_t awq_gemm_ex(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                         const void* scales_f16, const void* bias_f16, int64_t M, int64_t K,
                         int64_t N, int64_t group_size, void* y_f16, awq_path_t path,
                         awq_stream_t stream) {
  return gemm_any(x_f16, qweight, qzeros, scales_f16, bias_f16, M, K, N, group_size, y_f16, path,
                  stream, false);
}

awq_status_t awq_gemm_bf16_ex(const void* x_bf16, const int32_t* qweight, const int32_t* qzeros,
                              const void* scales_bf16, const void* bias_bf16, int64_t M, int64_t K,
                              int64_t N, int64_t group_size, void* y_bf16, awq_path_t path,
                              awq_stream_t stream) {
  return gemm_any(x_bf16, qweight, qzeros, scales_bf16, bias_bf16, M, K, N, group_size, y_bf16,
                  path, stream, true);
}

awq_status_t awq_gemm_grouped(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                              const void* scales_f16, const void* bias_f16,
                              const int32_t* expert_offsets, int64_t R, int64_t E, int64_t K,
                              int64_t N, int64_t group_size, void* y_f16, awq_stream_t stream) {
  if (E <= 0 || E > 4096) return fail(AWQ_ERR_INVALID_ARGUMENT, "E must be in 1..4096 (got %lld)", (long long)E);
  awq::GemmProblem p{};
  bool empty = false;
  awq_status_t st = build_problem(x_f16, qweight, qzeros, scales_f16, bias_f16, R, K, N, group_size,
                                  y_f16, stream, &p, &empty, false);
  if (st != AWQ_OK) return st;
  if (K * N * E >= kProdLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "E*K*N must be below 2^40");
  if ((R + 7) / 8 + E > 65535) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "R/8 + E must be at most 65535");
  if (empty) return ok();
  if (!expert_offsets) return fail(AWQ_ERR_INVALID_ARGUMENT, "null expert_offsets");
  if (!al(expert_offsets, 4)) return fail(AWQ_ERR_MISALIGNED, "expert_offsets must be 4-byte aligned");
  p.offsets = expert_offsets;
  p.E = static_cast<int>(E);
  const char* why = "";
  if (!awq::decode_grouped_supported(p, &why)) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "grouped: %s", why);
  st = check_device();
  if (st != AWQ_OK) return st;
  const cudaError_t e = awq::launch_decode_grouped(p);
  if (e != cudaSuccess) return cuda_fail(e, "awq_gemm_grouped launch");
  return ok();
}

awq_status_t awq_gemm_w8_ex(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                            const void* scales_f16, const void* bias_f16, int64_t M, int64_t K,
                            int64_t N, int64_t group_size, void* y_f16, awq_path_t path,
                            awq_stream_t stream) {
  return gemm_any(x_f16, qweight, qzeros, scales_f16, bias_f16, M, K, N, group_size, y_f16, path,
                  stream, false, 8);
}

awq_status_t awq_gemm_w8(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                         const void* scales_f16, const void* bias_f16, int64_t M, int64_t K,
                         int64_t N, int64_t group_size, void* y_f16, awq_stream_t stream) {
  return gemm_any(x_f16, qweight, qzeros, scales_f16, bias_f16, M, K, N, group_size, y_f16,
                  AWQ_PATH_AUTO, stream, false, 8);
}

awq_status_t awq_dequant_w8(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                            int64_t K, int64_t N, int64_t group_size, void* w_out,
                            awq_dtype_t out_dtype, awq_stream_t stream) {
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G, 4);
  if (st != AWQ_OK) return st;
  if (out_dtype != AWQ_DTYPE_F16 && out_dtype != AWQ_DTYPE_F32)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "out_dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_F32");
  if (N == 0) return ok();
  if (!qweight || !qzeros || !scales_f16 || !w_out)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "null pointer among qweight, qzeros, scales, w_out");
  if (!al(qweight, 4) || !al(qzeros, 4)) return fail(AWQ_ERR_MISALIGNED, "qweight/qzeros must be 4-byte aligned");
  if (!al(scales_f16, 2)) return fail(AWQ_ERR_MISALIGNED, "scales must be 2-byte aligned");
  if (!al(w_out, out_dtype == AWQ_DTYPE_F32 ? 4 : 2)) return fail(AWQ_ERR_MISALIGNED, "w_out misaligned for its dtype");
  st = check_device();
  if (st != AWQ_OK) return st;
  const cudaError_t e = awq::launch_dequant8(
      reinterpret_cast<const uint32_t*>(qweight), reinterpret_cast<const uint32_t*>(qzeros),
      static_cast<const __half*>(scales_f16), static_cast<int>(K), static_cast<int>(N), G, w_out,
      out_dtype == AWQ_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "awq_dequant_w8 launch");
  return ok();
}

awq_status_t awq_gemm_bf16(const void* x_bf16, const int32_t* qweight, const int32_t* qzeros,
                           const void* scales_bf16, const void* bias_bf16, int64_t M, int64_t K,
                           int64_t N, int64_t group_size, void* y_bf16, awq_stream_t stream) {
  return gemm_any(x_bf16, qweight, qzeros, scales_bf16, bias_bf16, M, K, N, group_size, y_bf16,
                  AWQ_PATH_AUTO, stream, true);
}

awq_status_t awq_dequant_bf16(const int32_t* qweight, const int32_t* qzeros, const void* scales_bf16,
                              int64_t K, int64_t N, int64_t group_size, void* w_out,
                              awq_dtype_t out_dtype, awq_stream_t stream) {
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G);
  if (st != AWQ_OK) return st;
  if (out_dtype != AWQ_DTYPE_BF16 && out_dtype != AWQ_DTYPE_F32)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "out_dtype must be AWQ_DTYPE_BF16 or AWQ_DTYPE_F32");
  if (N == 0) return ok();
  if (!qweight || !qzeros || !scales_bf16 || !w_out)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "null pointer among qweight, qzeros, scales, w_out");
  if (!al(qweight, 4) || !al(qzeros, 4)) return fail(AWQ_ERR_MISALIGNED, "qweight/qzeros must be 4-byte aligned");
  if (!al(scales_bf16, 2)) return fail(AWQ_ERR_MISALIGNED, "scales must be 2-byte aligned");
  if (!al(w_out, out_dtype == AWQ_DTYPE_F32 ? 4 : 2)) return fail(AWQ_ERR_MISALIGNED, "w_out misaligned for its dtype");
  st = check_device();
  if (st != AWQ_OK) return st;
  const cudaError_t e = awq::launch_dequant(
      reinterpret_cast<const uint32_t*>(qweight), reinterpret_cast<const uint32_t*>(qzeros),
      static_cast<const __half*>(scales_bf16), static_cast<int>(K), static_cast<int>(N), G, w_out,
      out_dtype == AWQ_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream), true);
  if (e != cudaSuccess) return cuda_fail(e, "awq_dequant_bf16 launch");
  return ok();
}

awq_status_t awq_gemm(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                      const void* scales_f16, const void* bias_f16, int64_t M, int64_t K,
                      int64_t N, int64_t group_size, void* y_f16, awq_stream_t stream) {
  return awq_gemm_ex(x_f16, qweight, qzeros, scales_f16, bias_f16, M, K, N, group_size, y_f16,
                     AWQ_PATH_AUTO, stream);
}

awq_path_t awq_gemm_select_path(int64_t M, int64_t K, int64_t N, int64_t group_size,
                                const void* x_f16, const int32_t* qweight,
                                const int32_t* qzeros, const void* scales_f16,
                                const void* bias_f16, const void* y_f16) {
  awq::GemmProblem p{};
  bool empty = false;
  if (build_problem(x_f16, qweight, qzeros, scales_f16, bias_f16, M, K, N, group_size,
                    const_cast<void*>(y_f16), nullptr, &p, &empty) != AWQ_OK || empty)
    return AWQ_PATH_AUTO;
  ok();
  return static_cast<awq_path_t>(choose_path(p));
}

awq_path_t awq_gemm_select_path_ex(int64_t M, int64_t K, int64_t N, int64_t group_size,
                                   const void* x, const int32_t* qweight, const int32_t* qzeros,
                                   const void* scales, const void* bias, const void* y,
                                   awq_dtype_t dtype, int32_t bits) {
  if ((dtype != AWQ_DTYPE_F16 && dtype != AWQ_DTYPE_BF16) || (bits != 4 && bits != 8) ||
      (bits == 8 && dtype != AWQ_DTYPE_F16))
    return AWQ_PATH_AUTO;
  awq::GemmProblem p{};
  bool empty = false;
  if (build_problem(x, qweight, qzeros, scales, bias, M, K, N, group_size, const_cast<void*>(y),
                    nullptr, &p, &empty, dtype == AWQ_DTYPE_BF16, bits) != AWQ_OK || empty)
    return AWQ_PATH_AUTO;
  ok();
  return static_cast<awq_path_t>(choose_path(p));
}

// Tile-packed layout of 4- or 8-bit codes: size and the one-off conversion.
static awq_status_t repack_size_bits(int64_t K, int64_t N, int64_t group_size, size_t* bytes, int bits) {
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G, bits == 8 ? 4 : 8);
  if (st != AWQ_OK) return st;
  if (!bytes) return fail(AWQ_ERR_INVALID_ARGUMENT, "null bytes pointer");
  const char* why = "";
  if (!(bits == 8 ? awq::packed8_supported(K, N, G, &why) : awq::packed_supported(K, N, G, &why)))
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "%s", why);
  *bytes = bits == 8 ? awq::packed8_bytes(K, N) : awq::packed_bytes(K, N);
  return ok();
}

static awq_status_t repack_bits(const int32_t* qweight, const int32_t* qzeros, const void* scales,
                                int64_t K, int64_t N, int64_t group_size, void* packed_out,
                                awq_stream_t stream, int bits) {
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G, bits == 8 ? 4 : 8);
  if (st != AWQ_OK) return st;
  const char* why = "";
  if (!(bits == 8 ? awq::packed8_supported(K, N, G, &why) : awq::packed_supported(K, N, G, &why)))
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "%s", why);
  if (N == 0) return ok();
  if (!qweight || !qzeros || !scales || !packed_out)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "null pointer among qweight, qzeros, scales, packed_out");
  if (!al(qweight, 4) || !al(qzeros, 4)) return fail(AWQ_ERR_MISALIGNED, "qweight/qzeros must be 4-byte aligned");
  if (!al(scales, 2)) return fail(AWQ_ERR_MISALIGNED, "scales must be 2-byte aligned");
  if (!al(packed_out, 16)) return fail(AWQ_ERR_MISALIGNED, "packed_out must be 16-byte aligned");
  if (K / 64 > 65535) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "K / 64 must be at most 65535");
  st = check_device();
  if (st != AWQ_OK) return st;
  const auto* qw = reinterpret_cast<const uint32_t*>(qweight);
  const auto* qz = reinterpret_cast<const uint32_t*>(qzeros);
  const auto* sc = static_cast<const __half*>(scales);
  const auto strm = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      bits == 8 ? awq::launch_repack8(qw, qz, sc, static_cast<int>(K), static_cast<int>(N), G, packed_out, strm)
                : awq::launch_repack(qw, qz, sc, static_cast<int>(K), static_cast<int>(N), G, packed_out, strm);
  if (e != cudaSuccess) return cuda_fail(e, "awq_repack launch");
  return ok();
}

awq_status_t awq_repack_size(int64_t K, int64_t N, int64_t group_size, size_t* bytes) {
  return repack_size_bits(K, N, group_size, bytes, 4);
}
awq_status_t awq_repack(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                        int64_t K, int64_t N, int64_t group_size, void* packed_out,
                        awq_stream_t stream) {
  return repack_bits(qweight, qzeros, scales_f16, K, N, group_size, packed_out, stream, 4);
}
awq_status_t awq_repack_w8_size(int64_t K, int64_t N, int64_t group_size, size_t* bytes) {
  return repack_size_bits(K, N, group_size, bytes, 8);
}
awq_status_t awq_repack_w8(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                           int64_t K, int64_t N, int64_t group_size, void* packed_out,
                           awq_stream_t stream) {
  return repack_bits(qweight, qzeros, scales_f16, K, N, group_size, packed_out, stream, 8);
}

// Checks of the packed linear's arguments; fills *p, and *launch = false when there is nothing
// to compute (M == 0 or N == 0).
static awq_status_t packed_problem(const void* x_f16, const void* packed, const void* bias_f16, int64_t M,
                                   int64_t K, int64_t N, int64_t group_size, void* y_f16,
                                   awq_stream_t stream, awq::GemmProblem* p, bool* launch, bool bf16 = false,
                                   int bits = 4) {
  *launch = false;
  if (M < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "M must be >= 0 (got %lld)", (long long)M);
  int G = 0;
  awq_status_t st = check_weight_shape(K, N, group_size, &G, bits == 8 ? 4 : 8);
  if (st != AWQ_OK) return st;
  const char* why = "";
  if (!(bits == 8 ? awq::packed8_supported(K, N, G, &why) : awq::packed_supported(K, N, G, &why)))
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "%s", why);
  if (M > kDimLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "M must be below 2^31");
  if (M * N >= kProdLimit || M * K >= kProdLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "M*N and M*K must be below 2^40");
  if (M == 0 || N == 0) return ok();
  if (!x_f16 || !packed || !y_f16) return fail(AWQ_ERR_INVALID_ARGUMENT, "null pointer among x, packed, y");
  if (!al(x_f16, 16)) return fail(AWQ_ERR_MISALIGNED, "x must be 16-byte aligned");
  if (!al(packed, 16)) return fail(AWQ_ERR_MISALIGNED, "packed must be 16-byte aligned");
  if (!al(y_f16, 2) || (bias_f16 && !al(bias_f16, 2)))
    return fail(AWQ_ERR_MISALIGNED, "y and bias must be 2-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  p->x = static_cast<const __half*>(x_f16);
  p->bias = static_cast<const __half*>(bias_f16);
  p->y = static_cast<__half*>(y_f16);
  p->M = static_cast<int>(M);
  p->K = static_cast<int>(K);
  p->N = static_cast<int>(N);
  p->G = G;
  p->stream = reinterpret_cast<cudaStream_t>(stream);
  p->bf16 = bf16;
  p->bits = bits;
  *launch = true;
  return ok();
}

static awq_status_t gemm_packed(const void* x_f16, const void* packed, const void* bias_f16, int64_t M,
                                int64_t K, int64_t N, int64_t group_size, void* y_f16, void* workspace,
                                size_t workspace_bytes, awq_stream_t stream) {
  awq::GemmProblem p{};
  bool launch = false;
  const awq_status_t st = packed_problem(x_f16, packed, bias_f16, M, K, N, group_size, y_f16, stream, &p, &launch);
  if (st != AWQ_OK || !launch) return st;
  const cudaError_t e = awq::launch_packed(p, packed, workspace, workspace_bytes);
  if (e != cudaSuccess) return cuda_fail(e, "awq_gemm_packed launch");
  return ok();
}

awq_status_t awq_gemm_packed(const void* x_f16, const void* packed, const void* bias_f16, int64_t M,
                             int64_t K, int64_t N, int64_t group_size, void* y_f16,
                             awq_stream_t stream) {
  return gemm_packed(x_f16, packed, bias_f16, M, K, N, group_size, y_f16, nullptr, 0, stream);
}

awq_status_t awq_gemm_packed_workspace_size(size_t* bytes) {
  if (!bytes) return fail(AWQ_ERR_INVALID_ARGUMENT, "null bytes pointer");
  awq_status_t st = check_device();
  if (st != AWQ_OK) return st;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "reading the SM count");
  *bytes = awq::packed_workspace_bytes(sms);
  return ok();
}

awq_status_t awq_gemm_packed_noalloc(const void* x_f16, const void* packed, const void* bias_f16, int64_t M,
                                     int64_t K, int64_t N, int64_t group_size, void* y_f16,
                                     awq_stream_t stream) {
  awq::GemmProblem p{};
  bool launch = false;
  awq_status_t st = packed_problem(x_f16, packed, bias_f16, M, K, N, group_size, y_f16, stream, &p, &launch);
  if (st != AWQ_OK || !launch) return st;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "reading the SM count");
  const size_t need = awq::packed_workspace_bytes(sms);
  if (need > awq::packed_static_scratch_bytes())
    return fail(AWQ_ERR_UNSUPPORTED_DEVICE,
                "this device's %d SMs need %zu bytes of scratch, more than the %zu-byte static array", sms,
                need, awq::packed_static_scratch_bytes());
  void* scratch = nullptr;
  e = awq::packed_static_scratch(&scratch);
  if (e != cudaSuccess) return cuda_fail(e, "locating the static scratch");
  // the ready flags start every call lowered (a call that gave up a wait may leave some raised)
  e = cudaMemsetAsync(scratch, 0, awq::packed_workspace_flag_bytes(sms), p.stream);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the scratch flags");
  e = awq::launch_packed(p, packed, scratch, need);
  if (e != cudaSuccess) return cuda_fail(e, "awq_gemm_packed_noalloc launch");
  return ok();
}

awq_status_t awq_gemm_packed_ex(const void* x, const void* packed, const void* bias, int64_t M, int64_t K,
                                int64_t N, int64_t group_size, void* y, awq_dtype_t dtype, void* workspace,
                                size_t workspace_bytes, awq_stream_t stream) {
  if (dtype != AWQ_DTYPE_F16 && dtype != AWQ_DTYPE_BF16)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  if (workspace && !al(workspace, 256)) return fail(AWQ_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  awq::GemmProblem p{};
  bool launch = false;
  const awq_status_t st = packed_problem(x, packed, bias, M, K, N, group_size, y, stream, &p, &launch,
                                         dtype == AWQ_DTYPE_BF16);
  if (st != AWQ_OK || !launch) return st;
  const cudaError_t e = awq::launch_packed(p, packed, workspace, workspace_bytes);
  if (e != cudaSuccess) return cuda_fail(e, "awq_gemm_packed_ex launch");
  return ok();
}

awq_status_t awq_gemm_packed_w8(const void* x_f16, const void* packed, const void* bias_f16, int64_t M,
                                int64_t K, int64_t N, int64_t group_size, void* y_f16, void* workspace,
                                size_t workspace_bytes, awq_stream_t stream) {
  if (workspace && !al(workspace, 256)) return fail(AWQ_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  awq::GemmProblem p{};
  bool launch = false;
  const awq_status_t st = packed_problem(x_f16, packed, bias_f16, M, K, N, group_size, y_f16, stream, &p,
                                         &launch, false, 8);
  if (st != AWQ_OK || !launch) return st;
  const cudaError_t e = awq::launch_packed(p, packed, workspace, workspace_bytes);
  if (e != cudaSuccess) return cuda_fail(e, "awq_gemm_packed_w8 launch");
  return ok();
}

awq_status_t awq_gemm_packed_grouped(const void* x, const void* packed, const void* bias,
                                     const int32_t* expert_offsets, int64_t R, int64_t E, int64_t K,
                                     int64_t N, int64_t group_size, void* y, awq_dtype_t dtype,
                                     awq_stream_t stream) {
  if (dtype != AWQ_DTYPE_F16 && dtype != AWQ_DTYPE_BF16)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  if (E <= 0 || E > awq::kPackedGroupedMaxE)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "E must be in 1..%d (got %lld)", awq::kPackedGroupedMaxE, (long long)E);
  awq::GemmProblem p{};
  bool launch = false;
  awq_status_t st = packed_problem(x, packed, bias, R, K, N, group_size, y, stream, &p, &launch,
                                   dtype == AWQ_DTYPE_BF16);
  if (st != AWQ_OK || !launch) return st;
  if (K * N * E >= kProdLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "E*K*N must be below 2^40");
  if (!expert_offsets) return fail(AWQ_ERR_INVALID_ARGUMENT, "null expert_offsets");
  if (!al(expert_offsets, 4)) return fail(AWQ_ERR_MISALIGNED, "expert_offsets must be 4-byte aligned");
  p.offsets = expert_offsets;
  p.E = static_cast<int>(E);
  const cudaError_t e = awq::launch_packed_grouped(p, packed);
  if (e != cudaSuccess) return cuda_fail(e, "awq_gemm_packed_grouped launch");
  return ok();
}

awq_status_t awq_gemm_packed_ws(const void* x_f16, const void* packed, const void* bias_f16, int64_t M,
                                int64_t K, int64_t N, int64_t group_size, void* y_f16, void* workspace,
                                size_t workspace_bytes, awq_stream_t stream) {
  if (workspace && !al(workspace, 256)) return fail(AWQ_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  return gemm_packed(x_f16, packed, bias_f16, M, K, N, group_size, y_f16, workspace, workspace_bytes, stream);
}

awq_status_t awq_device_status(awq_stream_t stream) {
  awq_status_t st = check_device();
  if (st != AWQ_OK) return st;
  unsigned int v = 0u;
  const cudaError_t e = awq::read_and_clear_status(reinterpret_cast<cudaStream_t>(stream), &v);
  if (e != cudaSuccess) return cuda_fail(e, "reading device status");
  if (v != 0u) return fail(AWQ_ERR_TIMEOUT, "a kernel gave up a bounded wait (code 0x%x)", v);
  return ok();
}

awq_status_t awq_selftest_wait_timeout(uint64_t limit_ns, awq_stream_t stream) {
  if (limit_ns < 1000ull || limit_ns > 1000000000ull)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "limit_ns must be within [1e3, 1e9]");
  awq_status_t st = check_device();
  if (st != AWQ_OK) return st;
  const cudaError_t e = awq::launch_selftest_wait(static_cast<unsigned long long>(limit_ns),
                                                  reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "launching the wait self test");
  return ok();
}

awq_status_t awq_selftest_attention_give_up(int on) {
  g_waits_give_up = on != 0;
  return ok();
}

// ------------------------------------------------ operators between a layer's linears ----

namespace {

awq_status_t check_half(awq_dtype_t dtype) {
  if (dtype != AWQ_DTYPE_F16 && dtype != AWQ_DTYPE_BF16)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "dtype must be AWQ_DTYPE_F16 or AWQ_DTYPE_BF16");
  return AWQ_OK;
}

awq_status_t check_cache(const awq_paged_kv_t* c, awq::PagedKV* out) {
  if (!c) return fail(AWQ_ERR_INVALID_ARGUMENT, "null cache");
  if (c->num_pages < 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "cache: num_pages >= 0, page_size, heads, head_dim > 0 needed");
  // a dimension of one entry is never stepped along: its stride may be anything
  const int64_t page_stride = c->num_pages > 1 ? c->page_stride : c->head_dim;
  const int64_t token_stride = c->page_size > 1 ? c->token_stride : c->head_dim;
  const int64_t head_stride = c->heads > 1 ? c->head_stride : c->head_dim;
  if (page_stride < 0 || token_stride < 0 || head_stride < 0)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "cache strides must not be negative");
  if (c->num_pages > kDimLimit || c->page_size > kDimLimit || c->heads > 65536 || c->head_dim > 65536 ||
      c->num_pages * c->page_size > kDimLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "cache: num_pages * page_size must be below 2^31, heads and head_dim <= 65536");
  if (c->num_pages > 0 && (!c->k || !c->v)) return fail(AWQ_ERR_INVALID_ARGUMENT, "cache: null k or v");
  if (!al(c->k, 2) || !al(c->v, 2)) return fail(AWQ_ERR_MISALIGNED, "cache tensors must be 2-byte aligned");
  *out = {static_cast<uint16_t*>(c->k), static_cast<uint16_t*>(c->v), static_cast<int>(c->num_pages),
          static_cast<int>(c->page_size), static_cast<int>(c->heads), static_cast<int>(c->head_dim),
          page_stride, token_stride, head_stride};
  return AWQ_OK;
}

awq_status_t rope(awq::RopeProblem* p, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rotary_dim,
                  int64_t max_position, awq_dtype_t dtype, const char* what) {
  awq_status_t st = check_half(dtype);
  if (st != AWQ_OK) return st;
  if (T < 0 || Hq < 0 || Hkv < 0 || max_position < 0)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "T, Hq, Hkv, max_position must be >= 0");
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > D)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "rotary_dim must be even, in 2..D (got %lld of D %lld)",
                (long long)rotary_dim, (long long)D);
  if (D > 65536 || Hq > 65536 || Hkv > 65536 || Hq + 2 * Hkv > 65536 || T > kDimLimit || max_position > kDimLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "D and Hq + 2 Hkv must be <= 65536, T and max_position below 2^31");
  if ((Hq + 2 * Hkv) * D > kDimLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "a token's heads must be below 2^31 elements");
  if (p->append && (p->kv.heads != Hkv || p->kv.head_dim != D))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "the cache must have Hkv heads of D elements");
  if (T == 0 || Hq + Hkv == 0) return ok();
  if ((Hq && (!p->q || !p->q_out)) || (Hkv && (!p->k || (p->append ? !p->v : !p->k_out))) || !p->positions || !p->table ||
      (p->append && !p->slots))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "%s: null pointer", what);
  if (!al(p->q, 2) || !al(p->k, 2) || !al(p->v, 2) || !al(p->q_out, 2) || !al(p->k_out, 2))
    return fail(AWQ_ERR_MISALIGNED, "16-bit tensors must be 2-byte aligned");
  if (!al(p->positions, 4) || !al(p->table, 4) || !al(p->slots, 4))
    return fail(AWQ_ERR_MISALIGNED, "positions, slots and table must be 4-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  p->T = T;
  p->Hq = static_cast<int>(Hq);
  p->Hkv = static_cast<int>(Hkv);
  p->D = static_cast<int>(D);
  p->rot = static_cast<int>(rotary_dim);
  p->max_position = static_cast<int>(max_position);
  p->bf16 = dtype == AWQ_DTYPE_BF16;
  // dense outputs; in place: the input's strides
  p->qo_st = p->q_out == p->q ? p->q_st : Hq * D;
  p->qo_sh = p->q_out == p->q ? p->q_sh : D;
  p->ko_st = p->k_out == p->k ? p->k_st : Hkv * D;
  p->ko_sh = p->k_out == p->k ? p->k_sh : D;
  const cudaError_t e = awq::launch_rope(*p);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return ok();
}

constexpr int64_t kAttentionLimit = (int64_t{1} << 31) - 256;  // keys: the end of a step stays below 2^31

// Shape rules of awq_attention_shared and its workspace; fills the host-side sizes of p.
awq_status_t attention_shape(int64_t B, int64_t n, int64_t Hq, int64_t heads, int64_t D, int64_t prefix_len,
                             int64_t max_len, awq::AttentionProblem* p) {
  if (B < 0 || n < 0 || Hq < 0 || prefix_len < 0 || max_len < 0)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "B, n, Hq, prefix_len, max_len must be >= 0");
  if (heads <= 0 || Hq % heads)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "Hq must be a multiple of the cache's heads (got %lld of %lld)",
                (long long)Hq, (long long)heads);
  if (!awq::attention_head_dim_supported(D))
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "head_dim must be 64, 96, 128 or 256 (got %lld)", (long long)D);
  if (Hq > 65536 || B > kDimLimit || n > kDimLimit || prefix_len > kAttentionLimit || max_len > kAttentionLimit || B * n > kDimLimit ||
      B * n * Hq > kDimLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "B * n * Hq must be below 2^31, prefix_len and max_len <= 2^31 - 256, Hq <= 65536");
  p->B = static_cast<int>(B);
  p->n = static_cast<int>(n);
  p->Hq = static_cast<int>(Hq);
  p->kv.heads = static_cast<int>(heads);
  p->kv.head_dim = static_cast<int>(D);
  p->prefix_len = prefix_len;
  p->max_len = max_len;
  return AWQ_OK;
}

awq_status_t dispatch_shape(int64_t T, int64_t k, int64_t E) {
  if (T < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %lld)", (long long)T);
  if (E < 1 || E > awq::kDispatchMaxE)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "E must be in 1..%d (got %lld)", awq::kDispatchMaxE, (long long)E);
  if (k < 1 || k > 1024) return fail(AWQ_ERR_INVALID_ARGUMENT, "k must be in 1..1024 (got %lld)", (long long)k);
  if (T > kDimLimit || T * k > kDimLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "T * k must be below 2^31");
  return AWQ_OK;
}

}  // namespace

awq_status_t awq_rope_table(float* table, int64_t max_position, int64_t rotary_dim, double base,
                            awq_rope_scaling_t scaling, double factor, int64_t original_max_position, double p0,
                            double p1, double attention_factor, awq_stream_t stream) {
  if (max_position < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "max_position must be >= 0");
  if (rotary_dim < 2 || rotary_dim % 2) return fail(AWQ_ERR_INVALID_ARGUMENT, "rotary_dim must be even and >= 2");
  if (max_position > kDimLimit || rotary_dim > 65536)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "max_position must be below 2^31, rotary_dim <= 65536");
  if (!(base > 1.0) || !(base < 1e300)) return fail(AWQ_ERR_INVALID_ARGUMENT, "base must be finite and > 1");
  if (scaling < AWQ_ROPE_NONE || scaling > AWQ_ROPE_BANDED)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "unknown scaling %d", static_cast<int>(scaling));
  if (scaling != AWQ_ROPE_NONE && (!(factor > 0.0) || !(factor < 1e300)))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "factor must be finite and > 0");
  if (scaling == AWQ_ROPE_NTK && rotary_dim < 4) return fail(AWQ_ERR_INVALID_ARGUMENT, "NTK scaling needs rotary_dim >= 4");
  if (scaling >= AWQ_ROPE_YARN && original_max_position <= 0)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "original_max_position must be positive");
  if (scaling == AWQ_ROPE_YARN && !(p0 > p1 && p1 > 0.0 && p0 < 1e300))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "YARN needs p0 > p1 > 0");
  if (scaling == AWQ_ROPE_BANDED && !(p1 > p0 && p0 > 0.0 && p1 < 1e300))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "BANDED needs p1 > p0 > 0");
  if (!(attention_factor > 0.0) || !(attention_factor < 1e30))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "attention_factor must be finite and > 0");
  if (max_position == 0) return ok();
  if (!table) return fail(AWQ_ERR_INVALID_ARGUMENT, "null table");
  if (!al(table, 4)) return fail(AWQ_ERR_MISALIGNED, "table must be 4-byte aligned");
  const awq_status_t st = check_device();
  if (st != AWQ_OK) return st;
  const awq::RopeTableProblem p{table, max_position, static_cast<int>(rotary_dim), base, static_cast<int>(scaling), factor,
                                static_cast<double>(original_max_position), p0, p1, attention_factor,
                                reinterpret_cast<cudaStream_t>(stream)};
  const cudaError_t e = awq::launch_rope_table(p);
  if (e != cudaSuccess) return cuda_fail(e, "awq_rope_table launch");
  return ok();
}

awq_status_t awq_rope(const void* q, const void* k, const int32_t* positions, const float* table, int64_t T, int64_t Hq,
                      int64_t Hkv, int64_t D, int64_t rotary_dim, int64_t max_position, int64_t q_token_stride,
                      int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride, void* q_out, void* k_out,
                      int interleaved, awq_dtype_t dtype, awq_stream_t stream) {
  awq::RopeProblem p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.positions = positions;
  p.table = table;
  p.q_st = q_token_stride;
  p.q_sh = q_head_stride;
  p.k_st = k_token_stride;
  p.k_sh = k_head_stride;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.interleaved = interleaved != 0;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return rope(&p, T, Hq, Hkv, D, rotary_dim, max_position, dtype, "awq_rope");
}

awq_status_t awq_rope_append(const void* q, const void* k, const void* v, const int32_t* positions, const float* table,
                             int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rotary_dim, int64_t max_position,
                             int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, void* q_out, const awq_paged_kv_t* cache,
                             const int32_t* slots, int interleaved, awq_dtype_t dtype, awq_stream_t stream) {
  awq::RopeProblem p{};
  const awq_status_t st = check_cache(cache, &p.kv);
  if (st != AWQ_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.positions = positions;
  p.table = table;
  p.q_st = q_token_stride;
  p.q_sh = q_head_stride;
  p.k_st = k_token_stride;
  p.k_sh = k_head_stride;
  p.v_st = v_token_stride;
  p.v_sh = v_head_stride;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.slots = slots;
  p.append = true;
  p.interleaved = interleaved != 0;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  return rope(&p, T, Hq, Hkv, D, rotary_dim, max_position, dtype, "awq_rope_append");
}

awq_status_t awq_attention_shared_workspace_size(int64_t B, int64_t n, int64_t Hq, int64_t heads, int64_t D,
                                                 int64_t prefix_len, int64_t max_len, size_t* bytes) {
  if (!bytes) return fail(AWQ_ERR_INVALID_ARGUMENT, "null bytes pointer");
  awq::AttentionProblem p{};
  const awq_status_t st = attention_shape(B, n, Hq, heads, D, prefix_len, max_len, &p);
  if (st != AWQ_OK) return st;
  *bytes = B * n * Hq == 0 ? 0 : awq::attention_workspace_bytes(p, sm_count());
  return ok();
}

awq_status_t awq_attention_shared(const void* q, int64_t B, int64_t n, int64_t Hq, int64_t q_batch_stride,
                                  int64_t q_token_stride, int64_t q_head_stride, const awq_paged_kv_t* cache,
                                  const int32_t* prefix_pages, int64_t prefix_len, const int32_t* pages, int64_t W,
                                  int64_t pages_stride, const int32_t* lens, int64_t max_len, float scale, void* out,
                                  awq_dtype_t dtype, void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  awq::AttentionProblem p{};
  awq_status_t st = check_half(dtype);
  if (st == AWQ_OK) st = check_cache(cache, &p.kv);
  if (st == AWQ_OK) st = attention_shape(B, n, Hq, p.kv.heads, p.kv.head_dim, prefix_len, max_len, &p);
  if (st != AWQ_OK) return st;
  if (W < 0 || W > kDimLimit) return fail(AWQ_ERR_INVALID_ARGUMENT, "W must be in 0..2^31 - 1");
  if (max_len > W * p.kv.page_size)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "max_len %lld is more than W = %lld pages of %d tokens", (long long)max_len,
                (long long)W, p.kv.page_size);
  if (B * n * Hq == 0) return ok();
  if (!q || !out || (prefix_len && !prefix_pages) || (max_len && (!pages || !lens)))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_attention_shared: null pointer");
  if (!al(q, 16) || !al(out, 16) || !al(p.kv.k, 16) || !al(p.kv.v, 16))
    return fail(AWQ_ERR_MISALIGNED, "q, out and the cache's tensors must be 16-byte aligned");
  if (B == 1) q_batch_stride = 0;
  if (n == 1) q_token_stride = 0;
  if (Hq == 1) q_head_stride = 0;
  if (q_batch_stride % 8 || q_token_stride % 8 || q_head_stride % 8 || p.kv.page_stride % 8 || p.kv.token_stride % 8 ||
      p.kv.head_stride % 8)
    return fail(AWQ_ERR_MISALIGNED, "strides of q and the cache must be multiples of 8 elements");
  if (!al(prefix_pages, 4) || !al(pages, 4) || !al(lens, 4))
    return fail(AWQ_ERR_MISALIGNED, "prefix_pages, pages and lens must be 4-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  const int sms = sm_count();
  const size_t need = awq::attention_workspace_bytes(p, sms);
  if (need && !workspace) return fail(AWQ_ERR_INVALID_ARGUMENT, "null workspace");
  if (!al(workspace, 256)) return fail(AWQ_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  if (workspace_bytes < need)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "the workspace has %zu bytes, this call needs %zu", workspace_bytes, need);
  p.q = static_cast<const uint16_t*>(q);
  p.q_sb = q_batch_stride;
  p.q_sn = q_token_stride;
  p.q_sh = q_head_stride;
  p.prefix_pages = prefix_pages;
  p.pages = pages;
  p.pages_ld = pages_stride;
  p.W = static_cast<int>(W);
  p.lens = lens;
  p.scale = scale;
  p.out = static_cast<uint16_t*>(out);
  p.bf16 = dtype == AWQ_DTYPE_BF16;
  p.give_up = g_waits_give_up;
  p.workspace = workspace;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = awq::launch_attention(p, sms);
  if (e != cudaSuccess) return cuda_fail(e, "awq_attention_shared launch");
  return ok();
}

awq_status_t awq_moe_route(const void* logits, int64_t T, int64_t E, int64_t row_stride, awq_dtype_t dtype, int64_t k,
                           int sigmoid, const float* bias, int64_t groups, int64_t topk_groups, int64_t group_best,
                           int renormalize, float scale, float* weights, int32_t* experts, awq_stream_t stream) {
  if (dtype != AWQ_DTYPE_F16 && dtype != AWQ_DTYPE_BF16 && dtype != AWQ_DTYPE_F32)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "unknown dtype %d", static_cast<int>(dtype));
  if (T < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %lld)", (long long)T);
  if (E < 1 || E > awq::kRouteMaxE)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "E must be in 1..%d (got %lld)", awq::kRouteMaxE, (long long)E);
  if (groups < 1 || groups > 32 || E % groups || topk_groups < 1 || topk_groups > groups)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "groups must divide E, 1 <= topk_groups <= groups <= 32");
  if (group_best != 1 && group_best != 2) return fail(AWQ_ERR_INVALID_ARGUMENT, "group_best must be 1 or 2");
  if (k < 1 || k > awq::kRouteMaxK || k > E / groups * topk_groups)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "k must be in 1..min(%d, E / groups * topk_groups) (got %lld)", awq::kRouteMaxK,
                (long long)k);
  if (T > kDimLimit || T * E >= kProdLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "T must be below 2^31, T * E below 2^40");
  if (T == 0) return ok();
  if (!logits || !weights || !experts) return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_moe_route: null pointer");
  if (!al(logits, dtype == AWQ_DTYPE_F32 ? 4 : 2) || !al(bias, 4) || !al(weights, 4) || !al(experts, 4))
    return fail(AWQ_ERR_MISALIGNED, "awq_moe_route: a tensor is not aligned to its elements");
  const awq_status_t st = check_device();
  if (st != AWQ_OK) return st;
  const awq::RouteProblem p{logits, T, row_stride, static_cast<int>(E), static_cast<int>(k), static_cast<int>(dtype),
                            sigmoid != 0, bias, static_cast<int>(groups), static_cast<int>(topk_groups),
                            static_cast<int>(group_best), renormalize != 0, scale, weights, experts,
                            reinterpret_cast<cudaStream_t>(stream)};
  const cudaError_t e = awq::launch_route(p);
  if (e != cudaSuccess) return cuda_fail(e, "awq_moe_route launch");
  return ok();
}

awq_status_t awq_moe_dispatch_workspace_size(int64_t T, int64_t k, int64_t E, size_t* bytes) {
  if (!bytes) return fail(AWQ_ERR_INVALID_ARGUMENT, "null bytes pointer");
  const awq_status_t st = dispatch_shape(T, k, E);
  if (st != AWQ_OK) return st;
  *bytes = awq::dispatch_workspace_bytes(T * k, static_cast<int>(E));
  return ok();
}

awq_status_t awq_moe_dispatch(const void* x, int64_t T, int64_t W, int64_t row_stride, const int32_t* experts, int64_t k,
                              int64_t E, void* routed, int32_t* offsets, int32_t* rows, void* workspace,
                              size_t workspace_bytes, awq_stream_t stream) {
  awq_status_t st = dispatch_shape(T, k, E);
  if (st != AWQ_OK) return st;
  if (W < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "W must be >= 0 (got %lld)", (long long)W);
  if (W > kDimLimit || T * k * W >= kProdLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "W must be below 2^31, T * k * W below 2^40");
  if (!offsets || (T && (!experts || !rows || (W && (!x || !routed)))))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_moe_dispatch: null pointer");
  if (!al(x, 2) || !al(routed, 2)) return fail(AWQ_ERR_MISALIGNED, "16-bit tensors must be 2-byte aligned");
  if (!al(experts, 4) || !al(offsets, 4) || !al(rows, 4))
    return fail(AWQ_ERR_MISALIGNED, "experts, offsets and rows must be 4-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  if (T == 0) {
    const cudaError_t e = cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 4, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ok() : cuda_fail(e, "awq_moe_dispatch offsets");
  }
  const size_t need = awq::dispatch_workspace_bytes(T * k, static_cast<int>(E));
  if (need && !workspace) return fail(AWQ_ERR_INVALID_ARGUMENT, "null workspace");
  if (!al(workspace, 256)) return fail(AWQ_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  if (workspace_bytes < need)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "the workspace has %zu bytes, this call needs %zu", workspace_bytes, need);
  const awq::DispatchProblem p{static_cast<const uint16_t*>(x), T, row_stride, static_cast<int>(W), experts,
                               static_cast<int>(k), static_cast<int>(E), static_cast<uint16_t*>(routed), offsets, rows,
                               workspace, reinterpret_cast<cudaStream_t>(stream)};
  const cudaError_t e = awq::launch_dispatch(p);
  if (e != cudaSuccess) return cuda_fail(e, "awq_moe_dispatch launch");
  return ok();
}

awq_status_t awq_moe_combine(const void* y, int64_t R, int64_t W, const float* weights, const int32_t* rows, int64_t T,
                             int64_t k, const void* base, void* out, awq_dtype_t dtype, awq_stream_t stream) {
  awq_status_t st = check_half(dtype);
  if (st != AWQ_OK) return st;
  if (R < 0 || W < 0 || T < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "R, W, T must be >= 0");
  if (k < 0 || k > 1024) return fail(AWQ_ERR_INVALID_ARGUMENT, "k must be in 0..1024 (got %lld)", (long long)k);
  if (R > kDimLimit || W > kDimLimit || T > kDimLimit || T * k > kDimLimit || R * W >= kProdLimit || T * W >= kProdLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "R, W, T * k must be below 2^31, R * W and T * W below 2^40");
  if (T == 0 || W == 0) return ok();
  if (!out || (R && !y) || (k && (!weights || !rows)))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_moe_combine: null pointer");
  if (!al(y, 2) || !al(base, 2) || !al(out, 2)) return fail(AWQ_ERR_MISALIGNED, "16-bit tensors must be 2-byte aligned");
  if (!al(weights, 4) || !al(rows, 4)) return fail(AWQ_ERR_MISALIGNED, "weights and rows must be 4-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  const awq::CombineProblem p{static_cast<const uint16_t*>(y), R, static_cast<int>(W), weights, rows, T,
                              static_cast<int>(k), static_cast<const uint16_t*>(base), static_cast<uint16_t*>(out),
                              dtype == AWQ_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)};
  const cudaError_t e = awq::launch_combine(p);
  if (e != cudaSuccess) return cuda_fail(e, "awq_moe_combine launch");
  return ok();
}

// ------------------------------- a 4-bit cache, norms, a layer of a few tokens' experts ----

namespace {

awq_status_t check_kv4_shape(int64_t page_size, int64_t head_dim, int64_t group_size) {
  if (page_size <= 0 || head_dim <= 0 || group_size <= 0)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "cache: page_size, head_dim, group_size > 0 needed");
  if (!awq::kv4_shape_supported(head_dim, group_size))
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE,
                "cache: head_dim must be 64, 96, 128 or 256 and group_size 32, 64 or 128 dividing it (got %lld, %lld)",
                (long long)head_dim, (long long)group_size);
  if (page_size % 16) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "cache: page_size must be a multiple of 16 (got %lld)", (long long)page_size);
  if (page_size > kDimLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "cache: page_size must be below 2^31");
  return AWQ_OK;
}

awq_status_t check_kv4(const awq_kv4_cache_t* c, awq::Kv4Cache* out) {
  if (!c) return fail(AWQ_ERR_INVALID_ARGUMENT, "null cache");
  const awq_status_t st = check_kv4_shape(c->page_size, c->head_dim, c->group_size);
  if (st != AWQ_OK) return st;
  if (c->num_pages < 0 || c->heads <= 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "cache: num_pages >= 0 and heads > 0 needed");
  if (c->num_pages > kDimLimit || c->heads > 65536 || c->num_pages * c->page_size > kDimLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "cache: num_pages * page_size must be below 2^31, heads <= 65536");
  // a dimension of one entry is never stepped along: its stride may be anything
  const int64_t page_stride = c->num_pages > 1 ? c->page_stride : 0, head_stride = c->heads > 1 ? c->head_stride : 0;
  if (page_stride < 0 || head_stride < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "cache strides must not be negative");
  if (c->num_pages > 0 && !c->data) return fail(AWQ_ERR_INVALID_ARGUMENT, "cache: null data");
  if (!al(c->data, 16) || page_stride % 16 || head_stride % 16)
    return fail(AWQ_ERR_MISALIGNED, "cache: data must be 16-byte aligned, its strides multiples of 16 bytes");
  *out = {static_cast<uint8_t*>(c->data), static_cast<int>(c->num_pages), static_cast<int>(c->page_size), static_cast<int>(c->heads),
          static_cast<int>(c->head_dim), static_cast<int>(c->group_size), page_stride, head_stride};
  return AWQ_OK;
}

awq_status_t attention_kv4_shape(int64_t B, int64_t n, int64_t Hq, int64_t heads, int64_t D, awq::AttentionKv4Problem* p) {
  if (B < 0 || n < 0 || Hq < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "B, n, Hq must be >= 0");
  if (heads <= 0 || Hq % heads)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "Hq must be a multiple of the cache's heads (got %lld of %lld)", (long long)Hq,
                (long long)heads);
  if (!awq::kv4_shape_supported(D, 32))
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "head_dim must be 64, 96, 128 or 256 (got %lld)", (long long)D);
  if (Hq > 65536 || B > kDimLimit || n > kDimLimit || B * n > kDimLimit || B * n * Hq > kDimLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "B * n * Hq must be below 2^31, Hq <= 65536");
  p->B = static_cast<int>(B);
  p->n = static_cast<int>(n);
  p->Hq = static_cast<int>(Hq);
  p->cache.heads = static_cast<int>(heads);
  p->cache.head_dim = static_cast<int>(D);
  return AWQ_OK;
}

awq_status_t check_workspace(const void* workspace, size_t have, size_t need) {
  if (need && !workspace) return fail(AWQ_ERR_INVALID_ARGUMENT, "null workspace");
  if (!al(workspace, 256)) return fail(AWQ_ERR_MISALIGNED, "workspace must be 256-byte aligned");
  if (have < need) return fail(AWQ_ERR_INVALID_ARGUMENT, "the workspace has %zu bytes, this call needs %zu", have, need);
  return AWQ_OK;
}

awq_status_t moe_layer_shape(int64_t T, int64_t k, int64_t H, int64_t I) {
  if (T < 0 || T > awq::kMoeLayerMaxT)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "T must be in 0..%d (got %lld): route more tokens through awq_moe_dispatch",
                awq::kMoeLayerMaxT, (long long)T);
  if (k < 0 || k > awq::kRouteMaxK) return fail(AWQ_ERR_INVALID_ARGUMENT, "k must be in 0..%d (got %lld)", awq::kRouteMaxK, (long long)k);
  if (H < 0 || I < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "H and I must be >= 0 (got %lld, %lld)", (long long)H, (long long)I);
  if (H >= (int64_t{1} << 30) || I >= (int64_t{1} << 30)) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "H and I must be below 2^30");
  return AWQ_OK;
}

}  // namespace

awq_status_t awq_kv4_page_bytes(int64_t page_size, int64_t head_dim, int64_t group_size, size_t* bytes) {
  if (!bytes) return fail(AWQ_ERR_INVALID_ARGUMENT, "null bytes pointer");
  const awq_status_t st = check_kv4_shape(page_size, head_dim, group_size);
  if (st != AWQ_OK) return st;
  *bytes = static_cast<size_t>(page_size) * (head_dim + 8 * (head_dim / group_size));
  return ok();
}

awq_status_t awq_rope_append_kv4(const void* q, const void* k, const void* v, const int32_t* positions, const float* table,
                                 int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rotary_dim, int64_t max_position,
                                 int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                                 int64_t v_token_stride, int64_t v_head_stride, void* q_out, const awq_kv4_cache_t* cache,
                                 const int32_t* slots, int interleaved, awq_dtype_t dtype, awq_stream_t stream) {
  awq::AppendKv4Problem p{};
  awq_status_t st = check_half(dtype);
  if (st == AWQ_OK) st = check_kv4(cache, &p.cache);
  if (st != AWQ_OK) return st;
  if (!table) rotary_dim = max_position = 0;
  if (T < 0 || Hq < 0 || Hkv < 0 || max_position < 0)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "T, Hq, Hkv, max_position must be >= 0");
  if (table && (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > D))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "rotary_dim must be even, in 2..D (got %lld of D %lld)", (long long)rotary_dim, (long long)D);
  if (p.cache.heads != Hkv || p.cache.head_dim != D)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "the cache must have Hkv heads of D elements");
  if (Hq + 2 * Hkv > 65536 || T > kDimLimit || T * (Hq + 2 * Hkv) > kDimLimit || max_position > kDimLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "Hq + 2 Hkv must be <= 65536, T * (Hq + 2 Hkv) and max_position below 2^31");
  if (T == 0) return ok();
  if ((Hq && (!q || !q_out)) || !k || !v || (table && !positions) || !slots)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_rope_append_kv4: null pointer");
  if (!al(q, 2) || !al(k, 2) || !al(v, 2) || !al(q_out, 2)) return fail(AWQ_ERR_MISALIGNED, "16-bit tensors must be 2-byte aligned");
  if (!al(positions, 4) || !al(table, 4) || !al(slots, 4))
    return fail(AWQ_ERR_MISALIGNED, "positions, slots and table must be 4-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.positions = positions;
  p.table = table;
  p.T = T;
  p.Hq = static_cast<int>(Hq);
  p.Hkv = static_cast<int>(Hkv);
  p.D = static_cast<int>(D);
  p.rot = static_cast<int>(rotary_dim);
  p.max_position = static_cast<int>(max_position);
  p.q_st = q_token_stride;
  p.q_sh = q_head_stride;
  p.k_st = k_token_stride;
  p.k_sh = k_head_stride;
  p.v_st = v_token_stride;
  p.v_sh = v_head_stride;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.qo_st = q_out == q ? q_token_stride : Hq * D;  // in place: the input's strides
  p.qo_sh = q_out == q ? q_head_stride : D;
  p.slots = slots;
  p.interleaved = interleaved != 0;
  p.bf16 = dtype == AWQ_DTYPE_BF16;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = awq::launch_append_kv4(p, sm_count());
  if (e != cudaSuccess) return cuda_fail(e, "awq_rope_append_kv4 launch");
  return ok();
}

awq_status_t awq_kv4_read(const awq_kv4_cache_t* cache, const int32_t* slots, int64_t T, void* k, void* v, awq_dtype_t dtype,
                          awq_stream_t stream) {
  awq::ReadKv4Problem p{};
  awq_status_t st = check_half(dtype);
  if (st == AWQ_OK) st = check_kv4(cache, &p.cache);
  if (st != AWQ_OK) return st;
  if (T < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "T must be >= 0 (got %lld)", (long long)T);
  if (T > kDimLimit || T * p.cache.heads > kDimLimit) return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "T * heads must be below 2^31");
  if (T == 0) return ok();
  if (!slots || !k || !v) return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_kv4_read: null pointer");
  if (!al(k, 2) || !al(v, 2) || !al(slots, 4)) return fail(AWQ_ERR_MISALIGNED, "k, v and slots must be aligned to their elements");
  st = check_device();
  if (st != AWQ_OK) return st;
  p.slots = slots;
  p.T = T;
  p.k = static_cast<uint16_t*>(k);
  p.v = static_cast<uint16_t*>(v);
  p.bf16 = dtype == AWQ_DTYPE_BF16;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = awq::launch_read_kv4(p);
  if (e != cudaSuccess) return cuda_fail(e, "awq_kv4_read launch");
  return ok();
}

awq_status_t awq_attention_kv4_workspace_size(int64_t B, int64_t n, int64_t Hq, int64_t heads, int64_t D, size_t* bytes) {
  if (!bytes) return fail(AWQ_ERR_INVALID_ARGUMENT, "null bytes pointer");
  awq::AttentionKv4Problem p{};
  const awq_status_t st = attention_kv4_shape(B, n, Hq, heads, D, &p);
  if (st != AWQ_OK) return st;
  *bytes = B * n * Hq == 0 ? 0 : awq::attention_kv4_workspace_bytes(p, sm_count());
  return ok();
}

awq_status_t awq_attention_kv4(const void* q, int64_t B, int64_t n, int64_t Hq, int64_t q_batch_stride, int64_t q_token_stride,
                               int64_t q_head_stride, const awq_kv4_cache_t* cache, const int32_t* pages, int64_t W,
                               int64_t pages_stride, const int32_t* lens, int64_t window, int64_t sinks, float scale, void* out,
                               awq_dtype_t dtype, void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  awq::AttentionKv4Problem p{};
  awq_status_t st = check_half(dtype);
  if (st == AWQ_OK) st = check_kv4(cache, &p.cache);
  if (st == AWQ_OK) st = attention_kv4_shape(B, n, Hq, p.cache.heads, p.cache.head_dim, &p);
  if (st != AWQ_OK) return st;
  if (W < 0 || W > kDimLimit || W * p.cache.page_size > kDimLimit)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "W * page_size must be in 0..2^31 - 1");
  if (window < 0 || window > kDimLimit || sinks < 0 || sinks > kDimLimit)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "window and sinks must be in 0..2^31 - 1");
  if (B * n * Hq == 0) return ok();
  if (!q || !out || !lens || (W && !pages)) return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_attention_kv4: null pointer");
  if (!al(q, 16) || !al(out, 16)) return fail(AWQ_ERR_MISALIGNED, "q and out must be 16-byte aligned");
  if (B == 1) q_batch_stride = 0;
  if (n == 1) q_token_stride = 0;
  if (Hq == 1) q_head_stride = 0;
  if (q_batch_stride % 8 || q_token_stride % 8 || q_head_stride % 8)
    return fail(AWQ_ERR_MISALIGNED, "strides of q must be multiples of 8 elements");
  if (!al(pages, 4) || !al(lens, 4)) return fail(AWQ_ERR_MISALIGNED, "pages and lens must be 4-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  const int sms = sm_count();
  st = check_workspace(workspace, workspace_bytes, awq::attention_kv4_workspace_bytes(p, sms));
  if (st != AWQ_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.q_sb = q_batch_stride;
  p.q_sn = q_token_stride;
  p.q_sh = q_head_stride;
  p.pages = pages;
  p.pages_ld = pages_stride;
  p.W = static_cast<int>(W);
  p.lens = lens;
  p.window = static_cast<int>(window);
  p.sinks = static_cast<int>(sinks);
  p.scale = scale;
  p.out = static_cast<uint16_t*>(out);
  p.bf16 = dtype == AWQ_DTYPE_BF16;
  p.give_up = g_waits_give_up;
  p.workspace = workspace;
  p.stream = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = awq::launch_attention_kv4(p, sms);
  if (e != cudaSuccess) return cuda_fail(e, "awq_attention_kv4 launch");
  return ok();
}

awq_status_t awq_residual_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, const void* gate,
                               int64_t gate_stride, const void* post_weight, const void* post_bias, float scale,
                               const void* weight, const void* bias, int64_t T, int64_t W, awq_norm_t kind, float eps, void* h,
                               void* y, awq_dtype_t dtype, awq_stream_t stream) {
  awq_status_t st = check_half(dtype);
  if (st != AWQ_OK) return st;
  if (T < 0 || W < 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "T and W must be >= 0");
  if (kind != AWQ_NORM_RMS && kind != AWQ_NORM_LAYER) return fail(AWQ_ERR_INVALID_ARGUMENT, "unknown norm %d", static_cast<int>(kind));
  if (!(eps >= 0.f) || !(eps < 1e30f)) return fail(AWQ_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
  if (T > kDimLimit || W > kDimLimit || T * W >= kProdLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "T and W must be below 2^31, T * W below 2^40");
  if ((post_bias && !post_weight) || (bias && !weight)) return fail(AWQ_ERR_INVALID_ARGUMENT, "a bias needs its weight");
  if (T == 0 || W == 0) return ok();
  if (!x || !h || (weight && !y)) return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_residual_norm: null pointer");
  if (!al(x, 2) || !al(residual, 2) || !al(gate, 2) || !al(post_weight, 2) || !al(post_bias, 2) || !al(weight, 2) || !al(bias, 2) ||
      !al(h, 2) || !al(y, 2))
    return fail(AWQ_ERR_MISALIGNED, "16-bit tensors must be 2-byte aligned");
  if (T == 1) x_stride = residual_stride = W;  // a dimension of one entry: its stride may be anything
  if ((h == residual && residual_stride != W) || (weight && y == x && x_stride != W))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "in place needs dense rows");
  st = check_device();
  if (st != AWQ_OK) return st;
  const auto u16 = [](const void* t) { return static_cast<const uint16_t*>(t); };
  const awq::ResidualNormProblem p{u16(x), u16(residual), u16(gate), x_stride, residual_stride, gate_stride, u16(post_weight),
                                   u16(post_bias), u16(weight), u16(bias), scale, eps, T, static_cast<int>(W),
                                   kind == AWQ_NORM_LAYER, static_cast<uint16_t*>(h), static_cast<uint16_t*>(y),
                                   dtype == AWQ_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)};
  const cudaError_t e = awq::launch_residual_norm(p, sm_count());
  if (e != cudaSuccess) return cuda_fail(e, "awq_residual_norm launch");
  return ok();
}

awq_status_t awq_moe_layer_workspace_size(int64_t T, int64_t k, int64_t H, int64_t I, size_t* bytes) {
  if (!bytes) return fail(AWQ_ERR_INVALID_ARGUMENT, "null bytes pointer");
  const awq_status_t st = moe_layer_shape(T, k, H, I);
  if (st != AWQ_OK) return st;
  *bytes = awq::moe_layer_workspace_bytes(static_cast<int>(T), static_cast<int>(k), static_cast<int>(H), static_cast<int>(I));
  return ok();
}

awq_status_t awq_moe_layer(const void* x, int64_t T, int64_t H, int64_t row_stride, const int32_t* experts, const float* weights,
                           int64_t k, int64_t E, int64_t I, int64_t group_size, const int32_t* up_qweight,
                           const int32_t* up_qzeros, const void* up_scales, const int32_t* down_qweight,
                           const int32_t* down_qzeros, const void* down_scales, const void* base, void* out, awq_dtype_t dtype,
                           void* workspace, size_t workspace_bytes, awq_stream_t stream) {
  awq_status_t st = check_half(dtype);
  if (st == AWQ_OK) st = moe_layer_shape(T, k, H, I);
  if (st != AWQ_OK) return st;
  if (E < 1 || E > awq::kDispatchMaxE)
    return fail(AWQ_ERR_INVALID_ARGUMENT, "E must be in 1..%d (got %lld)", awq::kDispatchMaxE, (long long)E);
  if (group_size <= 0) return fail(AWQ_ERR_INVALID_ARGUMENT, "group_size must be positive (got %lld)", (long long)group_size);
  if (H * I >= kProdLimit / 2 || E * (2 * H * I) >= kProdLimit)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "E * H * 2 I must be below 2^40");
  if (H % 8 || I % 8 || H % group_size || I % group_size)
    return fail(AWQ_ERR_UNSUPPORTED_SHAPE, "H and I must be multiples of 8 and of group_size");
  if (T == 0 || H == 0) return ok();
  if (!x || !out || (k && (!experts || !weights))) return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_moe_layer: null pointer");
  if (k && I && (!up_qweight || !up_qzeros || !up_scales || !down_qweight || !down_qzeros || !down_scales))
    return fail(AWQ_ERR_INVALID_ARGUMENT, "awq_moe_layer: null weights");
  if (out == x) return fail(AWQ_ERR_INVALID_ARGUMENT, "out must not be x");
  if (!al(x, 2) || !al(base, 2) || !al(out, 2) || !al(up_scales, 2) || !al(down_scales, 2))
    return fail(AWQ_ERR_MISALIGNED, "16-bit tensors must be 2-byte aligned");
  if (!al(experts, 4) || !al(weights, 4) || !al(up_qweight, 4) || !al(up_qzeros, 4) || !al(down_qweight, 4) || !al(down_qzeros, 4))
    return fail(AWQ_ERR_MISALIGNED, "experts, weights, qweight and qzeros must be 4-byte aligned");
  st = check_device();
  if (st != AWQ_OK) return st;
  st = check_workspace(workspace, workspace_bytes,
                       awq::moe_layer_workspace_bytes(static_cast<int>(T), static_cast<int>(k), static_cast<int>(H), static_cast<int>(I)));
  if (st != AWQ_OK) return st;
  const auto stacked = [](const int32_t* qw, const int32_t* qz, const void* sc) {
    return awq::Stacked{reinterpret_cast<const uint32_t*>(qw), reinterpret_cast<const uint32_t*>(qz), static_cast<const uint16_t*>(sc)};
  };
  const awq::MoeLayerProblem p{static_cast<const uint16_t*>(x), row_stride, static_cast<int>(T), static_cast<int>(H),
                               static_cast<int>(I), static_cast<int>(E), I ? static_cast<int>(k) : 0,  // I == 0: nothing to add
                               static_cast<int>(group_size), experts, weights, stacked(up_qweight, up_qzeros, up_scales),
                               stacked(down_qweight, down_qzeros, down_scales), static_cast<const uint16_t*>(base),
                               static_cast<uint16_t*>(out), dtype == AWQ_DTYPE_BF16, g_waits_give_up, workspace,
                               reinterpret_cast<cudaStream_t>(stream)};
  const cudaError_t e = awq::launch_moe_layer(p, sm_count());
  if (e != cudaSuccess) return cuda_fail(e, "awq_moe_layer launch");
  return ok();
}

}  // extern "C"
