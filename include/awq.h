/*
 * awq.h -- C ABI of libawq_gb300.so: AWQ W4A16 weight-only linear on GB300 (sm_103a).
 *
 * The weight layout is the AWQ "GEMM" checkpoint pack (tensref.org/formats/awq,
 * "Reader" pseudo-code; GPTQModel wiki "AWQ", "Saved formats and packing"):
 *
 *   qweight int32 [K, N/8]    row-major; nibble i (bits 4i..4i+3) of word c in row k
 *                             holds the 4-bit code of output column 8c + ORDER[i],
 *                             ORDER = {0,2,4,6,1,3,5,7}
 *   qzeros  int32 [K/G, N/8]  zero points, packed exactly like qweight
 *   scales  fp16  [K/G, N]    row-major
 *   bias    fp16  [N]         optional
 *
 * with K = in_features, N = out_features, G = group_size (G = K when group_size is -1:
 * one group across the row, GPTQModel wiki "AWQ", "Group quantization and zero points").
 * Every weight is  w[k][n] = (code[k][n] - zero[k/G][n]) * scale[k/G][n]  with the zero
 * used as stored (no +1; format page, reject rule AWQ-005).
 *
 * Conventions shared by every entry point:
 *  - Tensor pointers are DEVICE pointers owned by the caller, dense and row-major.  The
 *    library never frees or retains them and allocates no device memory per call.
 *  - Calls are asynchronous on `stream` (NULL = the legacy default stream) and never
 *    synchronize.  Argument errors are found on the host BEFORE any launch and returned
 *    synchronously; nothing is launched then.
 *  - On failure the call returns a non-zero awq_status_t and awq_last_error() holds a
 *    message for the calling thread.  On success awq_last_error() returns "".
 *  - Launch failures (cudaGetLastError after the launch) return AWQ_ERR_CUDA with the CUDA
 *    error string.
 *  - The library is built for compute capability 10.3 only; on another device every
 *    compute entry point returns AWQ_ERR_UNSUPPORTED_DEVICE.
 *  - Sizes are int64; each of M, K, N must be below 2^31, and M*N, K*N below 2^40.
 */
#ifndef AWQ_GB300_H
#define AWQ_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st* awq_stream_t;

typedef enum awq_status {
  AWQ_OK = 0,
  AWQ_ERR_INVALID_ARGUMENT = 1,  /* null pointer, negative size, bad group_size, bad enum */
  AWQ_ERR_UNSUPPORTED_SHAPE = 2, /* N not a multiple of 8, K not a multiple of G, size limits */
  AWQ_ERR_MISALIGNED = 3,        /* a pointer below its element alignment */
  AWQ_ERR_UNSUPPORTED_DEVICE = 4,/* current device is not compute capability 10.3 */
  AWQ_ERR_CUDA = 5,              /* a CUDA runtime call or launch failed */
  AWQ_ERR_TIMEOUT = 6            /* a bounded device-side wait gave up (see awq_device_status) */
} awq_status_t;

typedef enum awq_dtype { AWQ_DTYPE_F16 = 0, AWQ_DTYPE_F32 = 1, AWQ_DTYPE_BF16 = 2 } awq_dtype_t;

/* Kernel family used by awq_gemm_ex.  AUTO picks by M, K, N, G and alignment: decode for
 * M <= 32; above that, when both tensor-core families take the shape, whichever a cost
 * model fitted to GB300 timings predicts faster (decode's 32-row tiles win up to M = 64 ..
 * 192 depending on N and K); else the family whose contract holds, else generic. */
typedef enum awq_path {
  AWQ_PATH_AUTO = 0,
  AWQ_PATH_DECODE = 1,   /* split-K streaming kernel for small M (tensor-core m16n8k16) */
  AWQ_PATH_PREFILL = 2,  /* tcgen05/TMEM tensor-core kernel with TMA-fed tiles, large M */
  AWQ_PATH_GENERIC = 3   /* any valid shape and alignment; slow, used for ragged shapes */
} awq_path_t;

/* 1 when the current CUDA device is compute capability 10.3 and this library's kernels
 * load on it, else 0 (the reason is then in awq_last_error()).  Mirrors the wiki's
 * awq_runtime_available() / awq_runtime_error() pair (GPTQModel wiki "AWQ",
 * "Native AWQ runtime helpers"). */
int awq_runtime_available(void);

/* Thread-local message of the last failing call on this thread; "" after a success. */
const char* awq_last_error(void);

/* Static name of a status code ("AWQ_OK", ...). */
const char* awq_status_string(awq_status_t status);

/*
 * awq_dequant -- unpack and dequantize the whole weight (format page, "Reader"; the
 * wiki's awq_dequantize_weights in "Native AWQ runtime helpers").
 *
 *   w_out[k][n] = (code[k][n] - zero[k/G][n]) * scale[k/G][n]     row-major [K, N]
 *
 * out_dtype AWQ_DTYPE_F32: the exact fp32 value (it is always representable).
 * out_dtype AWQ_DTYPE_F16: that value rounded once, to nearest even.
 * Note the orientation: [K, N] (what x @ W needs); the format page's pseudo-code returns
 * the transpose [N, K].
 * Requirements: K > 0, N >= 0, N % 8 == 0, group_size == -1 or (> 0 and K % group_size
 * == 0); qweight/qzeros 4-byte aligned, scales 2-byte aligned, w_out aligned to its
 * element size.  N == 0 returns AWQ_OK without a launch.  One kernel launch otherwise.
 */
awq_status_t awq_dequant(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                         int64_t K, int64_t N, int64_t group_size,
                         void* w_out, awq_dtype_t out_dtype, awq_stream_t stream);

/*
 * bf16 activations and scales on the same weight layout (the native GEMM kernel's declared
 * contract lists FP16/BF16: GPTQModel wiki "AWQ", "Selection and compatibility", its
 * kernel table; vLLM accepts half and bfloat16: the vLLM article, section 4).  Same contract as awq_gemm_ex / awq_gemm / awq_dequant with
 * bf16 in place of fp16 for x, scales, bias and y (and for w_out when out_dtype is
 * AWQ_DTYPE_BF16):
 *
 *   y[m][n] = bf16_rne( sum_k x[m][k] * w[k][n]  (+ bias[n]) ),  w = (code - zero) * scale
 *
 * fp32 accumulation always.  The decode kernel carries each code into the MMA as the exact
 * bf16 value 128 + c and folds (128 + zero) * sum x out per group; the prefill kernel rounds
 * (c - zero) * scale once to bf16 for its tensor-core operand.  Paths: DECODE needs the
 * TMA decode kernel's contract (K % 64, G % 64, N % 32, 16-byte aligned x, qweight,
 * qzeros, scales); PREFILL as for fp16; GENERIC any valid shape.  AUTO chooses among them.
 * awq_dequant_bf16 writes the exact fp32 value (AWQ_DTYPE_F32) or that value rounded once
 * to bf16 (AWQ_DTYPE_BF16).
 */
awq_status_t awq_gemm_bf16_ex(const void* x_bf16, const int32_t* qweight, const int32_t* qzeros,
                              const void* scales_bf16, const void* bias_bf16, int64_t M, int64_t K,
                              int64_t N, int64_t group_size, void* y_bf16, awq_path_t path,
                              awq_stream_t stream);
awq_status_t awq_gemm_bf16(const void* x_bf16, const int32_t* qweight, const int32_t* qzeros,
                           const void* scales_bf16, const void* bias_bf16, int64_t M, int64_t K,
                           int64_t N, int64_t group_size, void* y_bf16, awq_stream_t stream);
awq_status_t awq_dequant_bf16(const int32_t* qweight, const int32_t* qzeros, const void* scales_bf16,
                              int64_t K, int64_t N, int64_t group_size, void* w_out,
                              awq_dtype_t out_dtype, awq_stream_t stream);

/*
 * 8-bit weights in the GEMM layout (GPTQModel wiki "AWQ", "Saved formats and packing":
 * widths other than 4 pack as a continuous little-endian bit stream, without the INT4
 * order; Marlin-class kernels take 8 bits, "Selection and compatibility").  Column 4c + i of
 * a row is byte i of word c:
 *
 *   qweight int32 [K, N/4], qzeros int32 [K/G, N/4], scales fp16 [K/G, N]
 *   w[k][n] = (code[k][n] - zero[k/G][n]) * scale[k/G][n],  codes 0..255
 *
 * awq_gemm_w8 / awq_gemm_w8_ex: the awq_gemm contract with 8-bit weights (N % 4 == 0).
 * The tensor-core families take 8-bit codes when K % 64 == 0, group_size % 64 == 0,
 * N % 16 == 0 and x, qweight, qzeros, scales are 16-byte aligned (AWQ_PATH_DECODE and
 * AWQ_PATH_PREFILL for any M, chosen as for 4-bit codes); everything else runs
 * AWQ_PATH_GENERIC.  Forcing a family whose contract the shape breaks returns
 * AWQ_ERR_UNSUPPORTED_SHAPE.  (awq_gemm_select_path_ex describes 8-bit calls.)
 * awq_dequant_w8: the awq_dequant contract (exact fp32, or one rounding to fp16).
 */
awq_status_t awq_gemm_w8_ex(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                            const void* scales_f16, const void* bias_f16, int64_t M, int64_t K,
                            int64_t N, int64_t group_size, void* y_f16, awq_path_t path,
                            awq_stream_t stream);
awq_status_t awq_gemm_w8(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                         const void* scales_f16, const void* bias_f16, int64_t M, int64_t K,
                         int64_t N, int64_t group_size, void* y_f16, awq_stream_t stream);
awq_status_t awq_dequant_w8(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                            int64_t K, int64_t N, int64_t group_size, void* w_out,
                            awq_dtype_t out_dtype, awq_stream_t stream);

/*
 * awq_gemm_grouped -- grouped (mixture-of-experts) W4A16 linear in one launch (routed expert
 * layers with 4-bit AWQ weights: the vLLM article, section 5.4).  E experts' weights are
 * stacked; the routed rows of x are sorted by expert:
 *
 *   y[r][n] = fp16_rne( sum_k x[r][k] * w_e[k][n] (+ bias[e][n]) )  for offsets[e] <= r < offsets[e+1]
 *
 *   x_f16           fp16 [R, K]            routed rows, sorted by expert
 *   qweight         int32 [E, K, N/8], qzeros int32 [E, K/G, N/8], scales_f16 fp16 [E, K/G, N]
 *   bias_f16        fp16 [E, N] or NULL
 *   expert_offsets  DEVICE int32 [E + 1]: 0 = offsets[0] <= ... <= offsets[E] = R (may come
 *                   from a routing kernel on the same stream; it is read on the device only,
 *                   after the preceding kernel completes)
 *   y_f16           fp16 [R, N]
 *
 * Requirements: those of the decode path's TMA kernel (K % 64 == 0, group size % 64 == 0,
 * N % 32 == 0, x / qweight / qzeros / scales 16-byte aligned), 1 <= E <= 4096,
 * R / 8 + E <= 65535, E*K*N < 2^40.  Offsets outside [0, R] or not rising give unspecified
 * values in y but never an access outside x, y or the stacked weights.  R == 0 returns
 * AWQ_OK without a launch.  One kernel launch; asynchronous on `stream`.
 */
awq_status_t awq_gemm_grouped(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                              const void* scales_f16, const void* bias_f16,
                              const int32_t* expert_offsets, int64_t R, int64_t E, int64_t K,
                              int64_t N, int64_t group_size, void* y_f16, awq_stream_t stream);

/*
 * awq_quantize_rtn -- round-to-nearest 4-bit group quantization of a linear layer's fp16
 * weight into this layout (GPTQModel wiki "AWQ", "Group quantization and zero points":
 * the asymmetric and symmetric modes of its table; packing with ORDER as the format
 * page's "Reader" unpacks it).  Per output channel n and group g of G input features:
 *
 *   sym == 0:  scale = max(max - min, 1e-5) / 15
 *              zero  = clamp(-round(min / scale), 0, 15)
 *              code  = clamp(round(w / scale) + zero, 0, 15)
 *   sym == 1:  scale = max(max |w|, 1e-5) / 7,  zero = 8
 *              code  = clamp(round(w / scale), -8, 7) + 8
 *
 * Arithmetic is fp32 on the fp16 weights with every operation correctly rounded; the
 * scale is rounded to fp16 (as stored) and the codes are taken against the stored scale;
 * round is half to even.  Weights must be finite.
 *
 *   w_f16        fp16 [N, K] row-major: out_features x in_features (an nn.Linear weight)
 *   qweight      int32 [K, N/8] out, qzeros int32 [K/G, N/8] out, scales_f16 fp16 [K/G, N] out
 *
 * Requirements: K > 0, N >= 0, N % 8 == 0, group_size == -1 or (> 0 and K % group_size
 * == 0), the group size a multiple of 8 and K / group_size <= 65535; w 16-byte aligned,
 * qweight/qzeros 4-byte aligned, scales 2-byte aligned; outputs must not overlap w.
 * N == 0 returns AWQ_OK without a launch.  Argument errors are returned before any device
 * access.  One kernel launch otherwise; asynchronous on `stream`.
 */
awq_status_t awq_quantize_rtn(const void* w_f16, int64_t N, int64_t K, int64_t group_size,
                              int sym, int32_t* qweight, int32_t* qzeros, void* scales_f16,
                              awq_stream_t stream);

/*
 * awq_gemm -- fused W4A16 linear (the wiki's awq_gemm_forward in "Native GEMM" /
 * "Native AWQ runtime helpers"; fp32 accumulation always, as with its default
 * GPTQMODEL_FP32_ACCUM):
 *
 *   y[m][n] = fp16_rne( sum_k x[m][k] * w[k][n]  (+ bias[n]) )
 *
 *   x_f16     fp16 [M, K] activations
 *   qweight   int32 [K, N/8], qzeros int32 [K/G, N/8], scales_f16 fp16 [K/G, N]
 *   bias_f16  fp16 [N] or NULL
 *   y_f16     fp16 [M, N] output; must not overlap any input
 *
 * Argument order is x, qweight, qzeros, scales, bias: qzeros BEFORE scales.  (The wiki's
 * Python wrappers pass scales before qzeros; bindings must not copy that order here.)
 * The dense weight is never written to memory.  The dequantized values never leave
 * registers or shared memory.  Accumulation is fp32 with a fixed summation order for a
 * given (M, K, N, G): repeated calls give bitwise-identical y.
 * Requirements: as awq_dequant, plus x/y/bias 2-byte aligned.  M == 0 or N == 0 returns
 * AWQ_OK without a launch (the wiki's "Empty input returns an appropriately shaped output
 * without launching").  Exactly one kernel launch otherwise.
 * Accuracy: |y - y_exact| <= 1e-2 * max(1, |y_exact|) elementwise, y_exact being the
 * same sum in exact arithmetic.
 * Stream ordering: plain stream order.  The small-M kernel is a programmatic dependent
 * launch (its set-up overlaps the tail of the preceding kernel on `stream`), but it reads
 * no input and writes no output before that kernel's results are visible, so a kernel
 * that writes x or the weights (awq_quantize_rtn, a copy kernel, ...) may come directly
 * before it.  awq_gemm_any with AWQ_GEMM_STATIC_WEIGHTS relaxes this for the weights.
 */
awq_status_t awq_gemm(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                      const void* scales_f16, const void* bias_f16,
                      int64_t M, int64_t K, int64_t N, int64_t group_size,
                      void* y_f16, awq_stream_t stream);

/* awq_gemm with an explicit kernel family (tests and benchmarks).  A family that cannot
 * take the shape or alignment returns AWQ_ERR_UNSUPPORTED_SHAPE / AWQ_ERR_MISALIGNED. */
awq_status_t awq_gemm_ex(const void* x_f16, const int32_t* qweight, const int32_t* qzeros,
                         const void* scales_f16, const void* bias_f16,
                         int64_t M, int64_t K, int64_t N, int64_t group_size,
                         void* y_f16, awq_path_t path, awq_stream_t stream);

/* Flags of awq_gemm_any. */
typedef enum awq_gemm_flags {
  AWQ_GEMM_DEFAULT = 0,
  /* The caller promises that qweight, qzeros, scales and bias are complete before the kernel
   * launched immediately before this call on `stream` is launched (weights loaded once, as
   * at model load): the small-M kernel then starts streaming them before that kernel has
   * finished, under its tail.  x is still read, and y written, only after that kernel's
   * results are visible.  Breaking the promise (e.g. the preceding kernel writes the
   * weights) gives unspecified y. */
  AWQ_GEMM_STATIC_WEIGHTS = 1
} awq_gemm_flags_t;

/*
 * awq_gemm_any -- one entry point for every activation type and code width, with flags:
 * dtype AWQ_DTYPE_F16 (the awq_gemm_ex contract) or AWQ_DTYPE_BF16 (awq_gemm_bf16_ex),
 * bits 4 (qweight [K, N/8]) or 8 (awq_gemm_w8_ex: qweight [K, N/4], fp16 only); flags a
 * combination of awq_gemm_flags_t (unknown bits: AWQ_ERR_INVALID_ARGUMENT).  With
 * AWQ_GEMM_DEFAULT it behaves exactly as the matching entry point above.
 */
awq_status_t awq_gemm_any(const void* x, const int32_t* qweight, const int32_t* qzeros,
                          const void* scales, const void* bias, int64_t M, int64_t K, int64_t N,
                          int64_t group_size, void* y, awq_dtype_t dtype, int32_t bits,
                          awq_path_t path, uint32_t flags, awq_stream_t stream);

/* The family awq_gemm would pick for this shape and these pointers (no launch; above
 * 32 rows it reads the current device's SM count, 152 if there is none).  Returns
 * AWQ_PATH_AUTO (0) on an invalid shape. */
awq_path_t awq_gemm_select_path(int64_t M, int64_t K, int64_t N, int64_t group_size,
                                const void* x_f16, const int32_t* qweight,
                                const int32_t* qzeros, const void* scales_f16,
                                const void* bias_f16, const void* y_f16);

/* The same for any entry point: dtype AWQ_DTYPE_F16 or AWQ_DTYPE_BF16 (activations, scales,
 * bias, output), bits 4 (qweight [K, N/8]) or 8 (qweight [K, N/4], fp16 only).  Returns
 * AWQ_PATH_AUTO (0) on an invalid shape or combination. */
awq_path_t awq_gemm_select_path_ex(int64_t M, int64_t K, int64_t N, int64_t group_size,
                                   const void* x, const int32_t* qweight, const int32_t* qzeros,
                                   const void* scales, const void* bias, const void* y,
                                   awq_dtype_t dtype, int32_t bits);

/*
 * Tile-packed layout: an optional one-off conversion of the checkpoint layout into this
 * library's kernel-native order, and the linear that reads it.  (No page prints such a
 * layout; converting the AWQ order away for a kernel is the prior art of the vLLM article,
 * section 5.1, and of the GPTQModel wiki, "Marlin and Machete".)  Lossless on codes, zeros
 * and scales.  For output-column tile t (128 columns) and K stage s (64 rows) one block of
 * 1152 uint32 words at word (t * K/64 + s) * 1152:
 *   word 512 h + 4 c + j (h < 2, c < 128, j < 4): 4-bit codes of column 128 t + c for rows
 *     64 s + 32 h + 8 j + 0..7, row offset ORDER[p] in nibble p (ORDER = {0,2,4,6,1,3,5,7});
 *   word 1024 + c: scale bits (fp16 or bf16) | zero << 16 of column 128 t + c, group of row 64 s;
 *   columns past N: zero.
 * Requirements: those of awq_dequant plus K % 64 == 0 and group size % 64 == 0 (or -1).
 *
 * awq_repack_size: bytes of the packed weights, ceil(N / 128) * (K / 64) * 4608 (host only,
 *   no device access).
 * awq_repack: writes them to packed_out (DEVICE, caller-owned, 16-byte aligned,
 *   awq_repack_size bytes); reads qweight/qzeros/scales as awq_dequant does; K / 64 <=
 *   65535.  The scale words are copied bit for bit, so bf16 scales give the packed weights
 *   of awq_gemm_packed_ex with AWQ_DTYPE_BF16.  One kernel launch, asynchronous on `stream`.
 *   N == 0: AWQ_OK, no launch.
 * awq_gemm_packed: y = fp16_rne(x W (+ bias)) as awq_gemm, W read from the packed layout
 *   (x fp16 [M, K] 16-byte aligned, packed 16-byte aligned, bias fp16 [N] or NULL, y fp16
 *   [M, N]; fp32 accumulation, a fixed summation order: repeated calls are bitwise
 *   identical; |y - y_exact| <= 1e-2 * max(1, |y_exact|)).  A tcgen05 kernel whose
 *   dequantized weights stay in tensor memory; built for prefill-sized M (any M >= 1 runs;
 *   below 128 rows awq_gemm on the checkpoint layout is mostly faster, except near 32 rows
 *   on wide linears).  M == 0 or N == 0:
 *   AWQ_OK, no launch.  One kernel launch otherwise, asynchronous on `stream`, plain stream
 *   order.
 */
awq_status_t awq_repack_size(int64_t K, int64_t N, int64_t group_size, size_t* bytes);
awq_status_t awq_repack(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                        int64_t K, int64_t N, int64_t group_size, void* packed_out,
                        awq_stream_t stream);
awq_status_t awq_gemm_packed(const void* x_f16, const void* packed, const void* bias_f16,
                             int64_t M, int64_t K, int64_t N, int64_t group_size, void* y_f16,
                             awq_stream_t stream);

/*
 * The packed linear with a workspace, for prefill shapes whose 256-row x 128-column tiles
 * leave SMs idle in the last round (e.g. 512 x 4096 x 11008: 172 tiles on 152 SMs).  Such
 * calls run a stream-K kernel: the tiles' 64-row K stages form one sequence split evenly over
 * one CTA per SM; a tile cut between CTAs is finished by the CTA holding its first stages,
 * which adds the other CTAs' fp32 partial sums (written to the workspace) in CTA order.  Other
 * shapes run exactly as awq_gemm_packed.  (No page prints a work split; stream-K is the
 * published decomposition of Osama et al., "Stream-K", PPoPP 2023.)
 *
 * awq_gemm_packed_workspace_size: bytes the current device needs (256-byte flag area sized by
 *   the SM count, then 128 KB per SM).
 * awq_gemm_packed_ws: arguments as awq_gemm_packed, plus workspace (DEVICE, caller-owned,
 *   256-byte aligned, workspace_bytes >= awq_gemm_packed_workspace_size, its first
 *   256-byte-rounded 4 * SM-count bytes ZERO before the first call; each call leaves them
 *   zero).  A workspace smaller than required (or NULL) gives awq_gemm_packed's plan.
 *   Results: awq_gemm_packed's criterion, and bitwise repeatable for a given shape and
 *   device; they may differ from awq_gemm_packed's in the last bits (another summation
 *   order).  Calls that share a workspace must not overlap in time (order them on one
 *   stream).  After awq_device_status reports a timeout, zero the flag area again.
 */
awq_status_t awq_gemm_packed_workspace_size(size_t* bytes);
awq_status_t awq_gemm_packed_ws(const void* x_f16, const void* packed, const void* bias_f16,
                                int64_t M, int64_t K, int64_t N, int64_t group_size, void* y_f16,
                                void* workspace, size_t workspace_bytes, awq_stream_t stream);

/*
 * awq_gemm_packed_noalloc: awq_gemm_packed_ws without a caller workspace.  No page has a
 * counterpart: it is a convenience of this library.  It works in scratch memory the library
 * reserves on each device when it is loaded, one fixed 20 MiB array (the workspace of a device
 * with up to 159 SMs; GB300 has 152).  On a device that would need more it returns
 * AWQ_ERR_UNSUPPORTED_DEVICE and launches nothing.
 *
 * It is meant for callers that cannot give the library device memory at the call site: a
 * host application whose device memory is all handed to its own pool before the first call,
 * or code behind an interface that passes only the layer's tensors, so that neither an
 * allocation inside the library nor an extra buffer argument is possible.
 *
 * It allocates nothing.  The first call on a device looks up the array's address (once per
 * device, with that device current, kept for the life of the process: do not use this entry
 * point after resetting the device); make that first call before any stream capture that is
 * to contain it.  Every call then clears the array's flag area with one asynchronous memset
 * on `stream` and launches what awq_gemm_packed_ws would launch with a workspace of its own,
 * with the same results.  All calls on one device share the array: calls that overlap in time
 * (on different streams, or from host threads without ordering between them) race on it and
 * may produce wrong results; order them on one stream.  Arguments, requirements and errors
 * otherwise as awq_gemm_packed.
 */
awq_status_t awq_gemm_packed_noalloc(const void* x_f16, const void* packed, const void* bias_f16,
                                     int64_t M, int64_t K, int64_t N, int64_t group_size,
                                     void* y_f16, awq_stream_t stream);

/*
 * awq_gemm_packed_ex: the packed linear for either activation type.  dtype AWQ_DTYPE_F16 (x,
 * bias, y fp16; the packed weights written from fp16 scales) or AWQ_DTYPE_BF16 (x, bias, y
 * bf16; the packed weights written by awq_repack from bf16 scales: it copies the 16-bit scale
 * words as they are).  bf16 dequantizes exactly as awq_dequant_bf16 does (c - z exact, one
 * rounding of (c - z) * s to bf16; GPTQModel wiki "AWQ", "Selection and compatibility": FP16
 * and BF16 activations) and accumulates in fp32; y is rounded once to bf16.  workspace /
 * workspace_bytes as awq_gemm_packed_ws (NULL / 0: awq_gemm_packed's plan).  Other arguments,
 * requirements, results and errors as awq_gemm_packed_ws; AWQ_ERR_INVALID_ARGUMENT for
 * another dtype.
 */
awq_status_t awq_gemm_packed_ex(const void* x, const void* packed, const void* bias, int64_t M,
                                int64_t K, int64_t N, int64_t group_size, void* y,
                                awq_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                awq_stream_t stream);

/*
 * Tile-packed layout of 8-bit codes (GPTQModel wiki "AWQ", "Saved formats and packing": the
 * 8-bit GEMM layout, byte i of word c = column 4c + i; qweight [K, N/4], qzeros [K/G, N/4],
 * fp16 scales).  Same tiles and meta words as the 4-bit layout; for tile t, stage s one block
 * of 2176 uint32 words at word (t * K/64 + s) * 2176:
 *   word 1024 h + 512 k + 4 c + j (h, k < 2, c < 128, j < 4): the 8-bit codes of column
 *     128 t + c for rows 64 s + 32 h + 16 k + 4 j + 0..3, row offset b in byte b;
 *   word 2048 + c: fp16 scale bits | zero << 16 (8-bit zero) of column 128 t + c;
 *   columns past N: zero.
 * Requirements: those of awq_dequant_w8 plus K % 64 == 0 and group size % 64 == 0 (or -1).
 * awq_repack_w8_size: ceil(N / 128) * (K / 64) * 8704 bytes (host only).
 * awq_repack_w8: as awq_repack, from 8-bit checkpoint tensors.
 * awq_gemm_packed_w8: y = fp16_rne(x W (+ bias)) from the 8-bit packed layout (fp16 x, bias,
 *   y; (c - z) * s formed exactly and rounded once to fp16, fp32 accumulation), with an
 *   optional workspace as awq_gemm_packed_ws (NULL / 0: no stream-K).  Arguments, results and
 *   errors otherwise as awq_gemm_packed_ws.
 */
/*
 * awq_gemm_packed_grouped: the grouped (mixture-of-experts) linear of awq_gemm_grouped on
 * tile-packed weights, for routed batches of prefill size (vLLM article, section 5.4: routed
 * expert layers).  packed holds E tile-packed layouts of 4-bit experts back to back, expert
 * e's at byte e * awq_repack_size(K, N, group_size) (awq_repack of qweight[e], qzeros[e],
 * scales[e] into that slice); x [R, K] routed rows sorted by expert, expert_offsets DEVICE
 * int32 [E + 1] as for awq_gemm_grouped (read on the device only), bias [E, N] or NULL,
 * y [R, N]; x, bias, y (and the scales the layouts were written from) fp16 (dtype
 * AWQ_DTYPE_F16) or bf16 (AWQ_DTYPE_BF16, as awq_gemm_packed_ex).  One persistent launch over (expert, 256-row tile,
 * column tile); a tile's rows of the next expert are computed and discarded.  Requirements:
 * those of awq_gemm_packed, 1 <= E <= 256, E*K*N < 2^40.  Offsets outside [0, R] or not
 * rising give unspecified values in y but never an access outside x, y, bias or packed.
 * R == 0 or N == 0: AWQ_OK, no launch.
 */
awq_status_t awq_gemm_packed_grouped(const void* x, const void* packed, const void* bias,
                                     const int32_t* expert_offsets, int64_t R, int64_t E,
                                     int64_t K, int64_t N, int64_t group_size, void* y,
                                     awq_dtype_t dtype, awq_stream_t stream);

awq_status_t awq_repack_w8_size(int64_t K, int64_t N, int64_t group_size, size_t* bytes);
awq_status_t awq_repack_w8(const int32_t* qweight, const int32_t* qzeros, const void* scales_f16,
                           int64_t K, int64_t N, int64_t group_size, void* packed_out,
                           awq_stream_t stream);
awq_status_t awq_gemm_packed_w8(const void* x_f16, const void* packed, const void* bias_f16,
                                int64_t M, int64_t K, int64_t N, int64_t group_size, void* y_f16,
                                void* workspace, size_t workspace_bytes, awq_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Operators between a decoder layer's linears: rotary positions, attention over a paged cache
 * whose sequences share a prefix, routing of tokens to experts, and the dispatch / combine pair
 * around the grouped linears above.  Elements are fp16 or bf16 (dtype AWQ_DTYPE_F16 or
 * AWQ_DTYPE_BF16) unless stated; strides are in elements; arithmetic is fp32 (or wider), rounded
 * once to the element type (awq_attention_shared rounds its probabilities as well).  The conventions at the top of this file hold: device pointers, no
 * allocation, asynchronous on `stream`, argument errors on the host before any launch.  Values
 * that only the device sees (positions, slots, pages, lengths, expert ids, rows) are checked
 * there: one outside its range never leads to an access outside the tensors.
 * ------------------------------------------------------------------------------------------ */

/* Scaling of the rotary frequencies f_i = base^(-2 i / rotary_dim) for contexts `factor` times
 * the trained one. */
typedef enum awq_rope_scaling {
  AWQ_ROPE_NONE = 0,
  AWQ_ROPE_LINEAR = 1, /* f / factor */
  AWQ_ROPE_NTK = 2,    /* base * factor^(rotary_dim / (rotary_dim - 2)) in place of base */
  AWQ_ROPE_YARN = 3,   /* pairs that turn over p0 times in original_max_position positions keep f,
                        * pairs below p1 turns take f / factor, a ramp over the pair index between */
  AWQ_ROPE_BANDED = 4  /* turns t = original_max_position * f / (2 pi): above p1 keeps f, below p0
                        * takes f / factor, between f (b + (1 - b) / factor), b = (t - p0) / (p1 - p0) */
} awq_rope_scaling_t;

/*
 * awq_rope_table -- the fp32 table [max_position, rotary_dim] that awq_rope reads: line p holds
 * cos(p f_i) * attention_factor for the rotary_dim / 2 pairs, then the sines.  Angles, sines and
 * cosines are computed in 64 bits and rounded once.  Written once per model.
 * Requirements: rotary_dim even and in 2..65536 (NTK: >= 4), 0 <= max_position < 2^31, base > 1 and
 * finite, factor > 0 (NONE: ignored); YARN: original_max_position > 0, p0 > p1 > 0; BANDED:
 * original_max_position > 0, p1 > p0 > 0; attention_factor > 0; table 4-byte aligned.
 */
awq_status_t awq_rope_table(float* table, int64_t max_position, int64_t rotary_dim, double base,
                            awq_rope_scaling_t scaling, double factor, int64_t original_max_position,
                            double p0, double p1, double attention_factor, awq_stream_t stream);

/*
 * awq_rope -- rotates the first rotary_dim elements of every query and key head by the angles of
 * its token's position and copies the rest:
 *
 *   (a, b) -> (a c - b s, b c + a s)   c, s: the table's line positions[t]
 *
 * with pairs (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when interleaved.
 *   q [T, Hq, D], k [T, Hkv, D]: strides given, a head's D elements contiguous (slices of a fused
 *   projection's output do)
 *   positions int32 [T]; table fp32 [max_position, rotary_dim] (awq_rope_table)
 *   q_out [T, Hq, D], k_out [T, Hkv, D] dense; or q_out == q (k_out == k): in place, in q's (k's)
 *   strides.  Outputs must not overlap inputs otherwise.
 * A position outside [0, max_position) gives NaN in the rotated part.  T == 0: AWQ_OK, no launch.
 * Requirements: rotary_dim even, 2 <= rotary_dim <= D <= 65536; Hq + 2 Hkv <= 65536; 16-bit tensors
 * 2-byte, the others 4-byte aligned.  One launch.
 */
awq_status_t awq_rope(const void* q, const void* k, const int32_t* positions, const float* table,
                      int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rotary_dim,
                      int64_t max_position, int64_t q_token_stride, int64_t q_head_stride,
                      int64_t k_token_stride, int64_t k_head_stride, void* q_out, void* k_out,
                      int interleaved, awq_dtype_t dtype, awq_stream_t stream);

/* A paged key/value cache: cell (page, token, head) of keys starts at element page * page_stride +
 * token * token_stride + head * head_stride of k, of values at the same element of v; head_dim
 * elements contiguous; the stride of a dimension of one entry is not looked at.  Slot s is token
 * s % page_size of page s / page_size. */
typedef struct awq_paged_kv {
  void* k;
  void* v;
  int64_t num_pages, page_size, heads, head_dim;
  int64_t page_stride, token_stride, head_stride;
} awq_paged_kv_t;

/*
 * awq_rope_append -- awq_rope whose rotated keys, with the values, go straight to a paged cache:
 * token t's key and value heads to cell slots[t] (int32 [T]).  A slot outside the cache keeps
 * nothing (padding tokens: -1).  Two tokens must not share a slot.  v [T, Hkv, D] as k; the cache
 * has Hkv heads of D elements and must not overlap the inputs.  Otherwise as awq_rope.
 */
awq_status_t awq_rope_append(const void* q, const void* k, const void* v, const int32_t* positions,
                             const float* table, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                             int64_t rotary_dim, int64_t max_position, int64_t q_token_stride,
                             int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, void* q_out,
                             const awq_paged_kv_t* cache, const int32_t* slots, int interleaved,
                             awq_dtype_t dtype, awq_stream_t stream);

/*
 * awq_attention_shared -- attention of the n newest tokens of B sequences that share a prefix, the
 * prefix's keys and values taken for the query rows of all sequences together:
 *
 *   out[b][i][h] = sum_j softmax_j(scale * q[b][i][h] . k_j) v_j
 *
 * over the prefix's prefix_len keys and those keys of sequence b that query token i sees: the
 * first lens[b] - n + i + 1 of its own (the n tokens are its last).  Query head h reads
 * key/value head h / (Hq / heads).
 *   q [B, n, Hq, D]: strides given, a head contiguous; out [B, n, Hq, D] dense
 *   cache: D = 64, 96, 128 or 256, Hq a multiple of its heads
 *   prefix_pages int32 [ceil(prefix_len / page_size)]: the prefix's pages, in order
 *   pages int32 [B, W] (row stride pages_stride), lens int32 [B]: each sequence's own pages and its
 *   number of own tokens; max_len >= every lens[b] (a longer one is cut to max_len), max_len <=
 *   W * page_size.  prefix_len, max_len are host values: the plan depends on them.
 * The B * n * Hq / heads rows that share a key/value head read the prefix once if they are more than
 * 32 and D <= 128, else once per 8 to 32 rows (D = 256: per 16).  A sequence's own keys are read
 * once per 8 to 32 of its rows: the call is made for few new tokens per sequence, and a prompt is right
 * but slow (4096 tokens, 64 / 8 heads of 128: 4.5 ms).
 * max_len sets the least share of the own keys that a warp takes: up to four times the average length
 * it costs nothing, far beyond that time grows with it (128 sequences of 1024 own keys on average over
 * 32768: 0.16 ms at max_len 2048 and 8192, 0.37 ms at 32768, 1.35 ms at 131072).
 * Precision: logits, statistics and sums are fp32.  Each probability is rounded to the element type as
 * the factor of its value (the second matrix product's operand type; the sum that divides uses the
 * unrounded ones), the result once more.
 * A row uses only the keys that it sees: what the cache holds past a length, or a newer token's value,
 * may be infinite or NaN.  A page outside [0, num_pages) gives unspecified values for its sequence.
 * A row that sees no key is zero; one whose logits are all -inf is NaN.  B, n or Hq 0: AWQ_OK, no launch.
 *   workspace: awq_attention_shared_workspace_size bytes (partial sums; same host values), 256-byte
 *   aligned; any content.  Calls that overlap in time need workspaces of their own.
 * Repeated calls give the same bits.  Requirements: q, the cache's tensors and out 16-byte aligned,
 * q's and the cache's strides multiples of 8 (of dimensions of more than one entry); prefix_len and max_len <= 2^31 - 256, other sizes below
 * 2^31.
 */
awq_status_t awq_attention_shared_workspace_size(int64_t B, int64_t n, int64_t Hq, int64_t heads,
                                                 int64_t D, int64_t prefix_len, int64_t max_len,
                                                 size_t* bytes);
awq_status_t awq_attention_shared(const void* q, int64_t B, int64_t n, int64_t Hq,
                                  int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride,
                                  const awq_paged_kv_t* cache, const int32_t* prefix_pages,
                                  int64_t prefix_len, const int32_t* pages, int64_t W,
                                  int64_t pages_stride, const int32_t* lens, int64_t max_len,
                                  float scale, void* out, awq_dtype_t dtype, void* workspace,
                                  size_t workspace_bytes, awq_stream_t stream);

/*
 * awq_moe_route -- k experts and their weights for each token from the router's logits [T, E]
 * (row stride given; dtype fp16, bf16 or AWQ_DTYPE_F32):
 *
 *   score = softmax over the row, or sigmoid;  key = score (+ bias, fp32 [E] or NULL)
 *   groups > 1: experts form `groups` equal runs; a group's score is the sum of its group_best (1 or
 *     2) best keys; experts outside the topk_groups best groups are out
 *   the k best keys, best first; equal keys (and groups): the lower index first
 *   weight = score (not the key), over the sum of the k scores if renormalize (0 if that is 0),
 *     times scale
 *
 * A logit of -inf takes its expert out; a place left without an expert gets id -1, weight 0.  A row
 * whose scores hold a NaN gets NaN weights and the ids 0 .. k - 1.
 *   weights fp32 [T, k], experts int32 [T, k], dense
 * Requirements: 1 <= E <= 1024, 1 <= k <= min(32, E / groups * topk_groups), 1 <= topk_groups <=
 * groups <= 32, E % groups == 0.  T == 0: AWQ_OK, no launch.  One launch.
 */
awq_status_t awq_moe_route(const void* logits, int64_t T, int64_t E, int64_t row_stride,
                           awq_dtype_t dtype, int64_t k, int sigmoid, const float* bias, int64_t groups,
                           int64_t topk_groups, int64_t group_best, int renormalize, float scale,
                           float* weights, int32_t* experts, awq_stream_t stream);

/*
 * awq_moe_dispatch -- sorts the T k places (token t, place j) by expert, equal experts in the order
 * of the places, and gathers the tokens' rows accordingly: what awq_gemm_grouped and
 * awq_gemm_packed_grouped take.
 *   x 16-bit [T, W] (row stride given), experts int32 [T, k]
 *   routed [T k, W] dense, offsets int32 [E + 1], rows int32 [T, k]: the place's row of routed
 * A place whose id lies outside [0, E) (-1: no expert) gets rows = -1; offsets[E] counts the places
 * with an expert, and routed's rows from there on are zero.
 *   workspace: awq_moe_dispatch_workspace_size bytes, 256-byte aligned; any content.  Calls that
 *   overlap in time need workspaces of their own.
 * Requirements: 1 <= E <= 4096, 1 <= k <= 1024, T k < 2^31, outputs do not overlap inputs.  T == 0:
 * offsets are set to 0.  W == 0: no rows are copied.
 */
awq_status_t awq_moe_dispatch_workspace_size(int64_t T, int64_t k, int64_t E, size_t* bytes);
awq_status_t awq_moe_dispatch(const void* x, int64_t T, int64_t W, int64_t row_stride,
                              const int32_t* experts, int64_t k, int64_t E, void* routed,
                              int32_t* offsets, int32_t* rows, void* workspace, size_t workspace_bytes,
                              awq_stream_t stream);

/*
 * awq_moe_combine -- out[t] = base[t] + sum_j weights[t][j] * y[rows[t][j]], in fp32 in the order of
 * the places, rounded once.  Places whose row lies outside [0, R) (-1) are left out, whatever their
 * weight.
 *   y [R, W], base [T, W] (a residual or a shared expert's output) or NULL, out [T, W] (may be base),
 *   dense; weights fp32 [T, k], rows int32 [T, k]
 * Requirements: 0 <= k <= 1024, R and T k < 2^31.  T == 0 or W == 0: AWQ_OK, no launch.  One launch.
 */
awq_status_t awq_moe_combine(const void* y, int64_t R, int64_t W, const float* weights,
                             const int32_t* rows, int64_t T, int64_t k, const void* base, void* out,
                             awq_dtype_t dtype, awq_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * A key/value cache held in 4 bits, and what stands around it in a decode step: the append that
 * quantizes, attention with a sliding window and first tokens that stay visible, the norms around a
 * residual sum, and a mixture-of-experts layer for a few tokens.  As above: fp16 or bf16 elements,
 * strides in elements unless stated, fp32 arithmetic, values that only the device sees checked there.
 * ------------------------------------------------------------------------------------------ */

/*
 * A paged cache of 4-bit keys and values.  `group_size` (32, 64 or 128, dividing head_dim) neighbouring
 * elements x of a token's head are kept as 4-bit codes c, a minimum m and a scale s of the 16-bit
 * element type; c stands for c * s + m:
 *
 *   m = min x,  s = rn16((max x - m) / 15),  c = clamp(rint((x - m) / s), 0, 15)   (s = 0: c = 0)
 *
 * a group that holds an infinity or a NaN reads NaN.  Page p's tokens of head h are the page_size / 16 tiles
 * of 16 tokens from byte p * page_stride + h * head_stride of data on.  A tile has 16 (D + 8 G) bytes, D =
 * head_dim, G = D / group_size:
 *
 *   8 D bytes of key codes, 8 D of value codes, 64 G of the keys' (s, m) pairs, [token][group], 64 G of the
 *   values'.  The low nibble of a byte is an even element's, the high one the next element's.
 *   Keys: element 8 w + j (j < 8) of token r, w = 16 a + 4 b + t (t < 4; b < W, W = min(D, 128) / 32), is in byte
 *     1024 a + 16 W r + 4 (W t + b) + j / 2.
 *   Values: element 32 u + 4 g + j (j < 4) of token r = 8 h + 2 t + o (o < 2) is in byte
 *     512 (u / 2) + 16 (4 g + t) + 8 (u % 2) + 4 h + 2 o + j / 2, or, for the last u of an odd number,
 *     512 (u / 2) +  8 (4 g + t)               + 4 h + 2 o + j / 2.
 *
 * (the order in which tensor-core fragments take them).  Slot s is token s % page_size of page s / page_size.
 * Requirements: D = 64, 96, 128 or 256; page_size a multiple of 16; data 16-byte aligned, page_stride and
 * head_stride (bytes; of a dimension of more than one entry) multiples of 16, not negative; num_pages *
 * page_size below 2^31.
 */
typedef struct awq_kv4_cache {
  void* data;
  int64_t num_pages, page_size, heads, head_dim, group_size;
  int64_t page_stride, head_stride;
} awq_kv4_cache_t;

/* Bytes of one head's tokens of a page: page_size * (head_dim + 8 * head_dim / group_size).  Host only. */
awq_status_t awq_kv4_page_bytes(int64_t page_size, int64_t head_dim, int64_t group_size, size_t* bytes);

/*
 * awq_rope_append_kv4 -- awq_rope_append to a 4-bit cache: rotated keys, rounded to the element type, and
 * values are quantized to cell slots[t].  A rotated element is a c - b s with both products and the
 * difference rounded to fp32 by themselves, in q_out as in the cache.  table NULL: nothing is rotated
 * (positions, rotary_dim, max_position are not looked at), q is copied; Hq may be 0.  Otherwise as
 * awq_rope_append: a slot outside the cache keeps nothing, two tokens must not share a slot, q_out may
 * be q.  A position outside the table gives NaN: groups of the key that hold rotated elements read NaN.
 * T * (Hq + 2 Hkv) must be below 2^31.  One launch.
 */
awq_status_t awq_rope_append_kv4(const void* q, const void* k, const void* v, const int32_t* positions,
                                 const float* table, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                 int64_t rotary_dim, int64_t max_position, int64_t q_token_stride,
                                 int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                                 int64_t v_token_stride, int64_t v_head_stride, void* q_out,
                                 const awq_kv4_cache_t* cache, const int32_t* slots, int interleaved,
                                 awq_dtype_t dtype, awq_stream_t stream);

/*
 * awq_kv4_read -- the keys and values that the cache holds at slots int32 [T], c * s + m rounded once to
 * the element type: k, v [T, heads, head_dim] dense.  A slot outside the cache reads zero.  T * heads must
 * be below 2^31.  One launch.
 */
awq_status_t awq_kv4_read(const awq_kv4_cache_t* cache, const int32_t* slots, int64_t T, void* k, void* v,
                          awq_dtype_t dtype, awq_stream_t stream);

/*
 * awq_attention_kv4 -- attention of the n newest tokens of B sequences over a 4-bit cache:
 *
 *   out[b][i][h] = sum_j softmax_j(scale * q[b][i][h] . k_j) v_j
 *
 * over the keys j that query token i of sequence b, at P = lens[b] - n + i, sees: j <= P, and with a window
 * > 0 of these j > P - window or j < sinks (the first tokens of a sequence stay visible).  Query head h
 * reads key/value head h / (Hq / heads).
 *   q [B, n, Hq, D]: strides given, a head contiguous; out [B, n, Hq, D] dense
 *   pages int32 [B, W] (row stride pages_stride): the sequences' pages, in order; lens int32 [B], the n new
 *   tokens counted (one above W * page_size is cut to it).  Pages that a window leaves out may be any
 *   number: they are not read.
 * k_j and v_j are what the codes stand for, unrounded; logits, statistics and sums are fp32.  The factor of a
 * value's code, counted from 8, is probability times scale, rounded to fp16's 11 bits (fp16 elements: 22), in
 * steps of at least 2^-31 of the largest factor of the same query row and group of elements, and an element of a bf16 query in steps
 * of at least 2^-28 of the row's largest.  A sequence's keys are cut into parts by all sequences' lengths, so
 * other lengths may change its result's last bits.  Keys and values above 2^100 in size (bf16) may overflow.
 * A row uses only the keys that it sees: what the cache holds elsewhere
 * may be anything.  A page outside [0, num_pages) gives unspecified values for its sequence.  A row that
 * sees no key is zero; one whose logits are all -inf is NaN.  B, n or Hq 0: AWQ_OK, no launch.
 *   workspace: awq_attention_kv4_workspace_size bytes, 256-byte aligned; any content.  Calls that overlap in
 *   time need workspaces of their own.
 * Repeated calls give the same bits.  The call is made for few new tokens per sequence: a prompt is right
 * but slow.  Requirements: q and out 16-byte aligned, q's strides multiples of 8 (of dimensions of more than
 * one entry), Hq a multiple of heads; W * page_size below 2^31, window and sinks in 0..2^31 - 1.
 */
awq_status_t awq_attention_kv4_workspace_size(int64_t B, int64_t n, int64_t Hq, int64_t heads, int64_t D,
                                              size_t* bytes);
awq_status_t awq_attention_kv4(const void* q, int64_t B, int64_t n, int64_t Hq, int64_t q_batch_stride,
                               int64_t q_token_stride, int64_t q_head_stride, const awq_kv4_cache_t* cache,
                               const int32_t* pages, int64_t W, int64_t pages_stride, const int32_t* lens,
                               int64_t window, int64_t sinks, float scale, void* out, awq_dtype_t dtype,
                               void* workspace, size_t workspace_bytes, awq_stream_t stream);

typedef enum awq_norm { AWQ_NORM_RMS = 0, AWQ_NORM_LAYER = 1 } awq_norm_t;

/*
 * awq_residual_norm -- the norms before and after a block, around its residual sum:
 *
 *   t = norm(x) * post_weight (+ post_bias), or x where post_weight is NULL
 *   h = residual + scale * gate * t          (a NULL residual counts 0, a NULL gate 1)
 *   y = norm(h) * weight (+ bias)            (not formed where weight is NULL)
 *   norm(z) = z / sqrt(mean(z^2) + eps) over the row; LAYER: of z - mean(z)
 *
 *   x, residual [T, W]: row strides given; gate [T, W] with a row stride, 0 for one row of all tokens;
 *   weights and biases [W]; h, y [T, W] dense.  h may be residual and y may be x where those are dense.
 * fp32 arithmetic, y from the unrounded h, each output rounded once.  T == 0 or W == 0: AWQ_OK, no launch.
 * Requirements: post_bias only with post_weight, bias only with weight, y with weight; eps >= 0; outputs
 * overlap nothing else.  One launch.
 */
awq_status_t awq_residual_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                               const void* gate, int64_t gate_stride, const void* post_weight,
                               const void* post_bias, float scale, const void* weight, const void* bias,
                               int64_t T, int64_t W, awq_norm_t kind, float eps, void* h, void* y,
                               awq_dtype_t dtype, awq_stream_t stream);

/*
 * awq_moe_layer -- a mixture-of-experts layer of a few tokens on 4-bit experts, in two launches:
 *
 *   act[t][j] = silu(x[t] Wg) * (x[t] Wu),   out[t] = base[t] + sum_j weights[t][j] * (act[t][j] Wd)
 *
 * with the matrices of expert experts[t][j] (awq_moe_route's ids and weights), w = (code - zero) * scale.
 *   x [T, H] (row stride given), weights fp32 [T, k], experts int32 [T, k]; base [T, H] or NULL, out [T, H]
 *   dense (may be base, not x)
 *   up_qweight int32 [E, H, 2 I / 8], up_qzeros [E, H / G, 2 I / 8], up_scales 16-bit [E, H / G, 2 I]: gate
 *   columns, then up columns; down_qweight [E, I, H / 8], down_qzeros [E, I / G, H / 8], down_scales [E, I /
 *   G, H]: stacked linears as awq_gemm_grouped takes them, G = group_size
 * A place whose id lies outside [0, E) (-1) is left out, whatever its weight.  Sums are fp32, of a token's
 * places in their order; act is the sum of two elements (22 bits of fp16, 16 of bf16; infinite beyond the type's
 * range) as the factor of the second product, and the result is rounded once.  A token with an element that is not finite gives NaN.  Repeated calls give the same
 * bits.
 *   workspace: awq_moe_layer_workspace_size bytes, 256-byte aligned; any content.  Calls that overlap in
 *   time need workspaces of their own.
 * Requirements: 0 <= T <= 16 (more: awq_moe_dispatch and the grouped linears), 0 <= k <= 32, 1 <= E <= 4096;
 * H and I multiples of 8 and of G > 0; E * H * 2 I below 2^40.  T == 0 or H == 0: AWQ_OK, no launch.
 */
awq_status_t awq_moe_layer_workspace_size(int64_t T, int64_t k, int64_t H, int64_t I, size_t* bytes);
awq_status_t awq_moe_layer(const void* x, int64_t T, int64_t H, int64_t row_stride, const int32_t* experts,
                           const float* weights, int64_t k, int64_t E, int64_t I, int64_t group_size,
                           const int32_t* up_qweight, const int32_t* up_qzeros, const void* up_scales,
                           const int32_t* down_qweight, const int32_t* down_qzeros, const void* down_scales,
                           const void* base, void* out, awq_dtype_t dtype, void* workspace,
                           size_t workspace_bytes, awq_stream_t stream);

/* Synchronizes `stream`, then reads and clears the library's device status word on the
 * current device.  Returns AWQ_ERR_TIMEOUT if a kernel gave up a bounded wait since the
 * last check (its output is then unspecified), AWQ_OK otherwise. */
awq_status_t awq_device_status(awq_stream_t stream);

/* Failure-detection self test.  Launches one thread that waits on an mbarrier nothing
 * ever completes, bounded by limit_ns of wall time (1e3 .. 1e9, else
 * AWQ_ERR_INVALID_ARGUMENT): the wait gives up the same way a stalled stage of the GEMM
 * kernels would -- it sets the device status word and the kernel returns, with no fault,
 * trap or hang -- so a following awq_device_status returns AWQ_ERR_TIMEOUT (and clears
 * the word).  Asynchronous on `stream`; one launch.  No counterpart on the pages. */
awq_status_t awq_selftest_wait_timeout(uint64_t limit_ns, awq_stream_t stream);

/* Failure-detection self test of awq_attention_shared, awq_attention_kv4 and awq_moe_layer: after on != 0, the
 * calling host thread's calls give up their kernels' waits for copies as if they had run out (on == 0: back to
 * normal).  Such a call's output is unspecified, it touches nothing outside its tensors, and a following
 * awq_device_status returns AWQ_ERR_TIMEOUT; calls whose copies have no wait that can run out
 * (awq_attention_shared: page_size % 16 != 0, fewer than 3 steps of a block; awq_moe_layer: H or I no multiple of
 * 64, group_size neither 32 nor one) are unaffected.  Host only. */
awq_status_t awq_selftest_attention_give_up(int on);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_GB300_H */
