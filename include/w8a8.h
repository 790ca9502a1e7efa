/*
 * w8a8.h -- C ABI of libw8a8, the GB300 (sm_103a) W8A8 / W4A8 quantized
 * linear layer.
 *
 * The method: "Apple Silicon의 AI 한계치는 당신의 생각보다 높습니다"
 * (molayo1419.me), section "INT8 TensorOps 커널 설계", describes a four-step
 * pipeline -- (1) a min/max reduction that gives each activation row its
 * scale, (2) a streaming fp16 -> INT8 mapping, (3) an INT8 x INT8 GEMM that
 * accumulates in INT32, (4) a rescale of the INT32 result by the product of
 * the activation and weight scales into fp16 -- and section
 * "입도(Granularity)" adds per-group scales (64 or 128 elements) that need
 * grouped dequantization during accumulation.  "cider 소개"
 * (discuss.pytorch.kr), section "cider의 양자화 모드와 적용 가능한 영역",
 * fixes the modes: symmetric INT8 weights, per-token INT8 activations,
 * per-channel or per-group (gs 128 / 64) scales, and W4A8 with INT4 weights
 * packed in uint8 and unpacked before the INT8 matmul; its section
 * "cider 설치와 사용법" names quantize_weight_int8 / pack_weight_int4 and
 * the seq_len rule of CiderLinear (seq_len > 1: GEMM, seq_len == 1: INT8
 * matrix-vector kernel).
 *
 * Conventions for every entry point below
 * ---------------------------------------
 *  - Shapes: x [M, K] fp16 row-major (K contiguous); W [N, K] row-major
 *    (out_features x in_features); y = x . W^T, [M, N] fp16 row-major.
 *    G = K / group_size groups along K (G = 1 when group_size == 0).
 *  - fp16 buffers are IEEE binary16 bit patterns (w8a8_half).
 *  - Every pointer is a DEVICE pointer on the current CUDA device, owned by
 *    the caller.  The library allocates no device memory and keeps no
 *    pointer after a call returns.
 *  - The library caches per-device state (function attributes, the SM
 *    count, the device addresses of its own device variables) on the first
 *    call on each device; the caches are thread-safe.  Do not use the
 *    library on a device after cudaDeviceReset() in the same process: the
 *    cached addresses would be stale.
 *  - Matrix pointers (x, W, Wq, Wp, xq, y, acc, workspace) must be 16-byte
 *    aligned, scale pointers 4-byte aligned, and K a multiple of 16 (32 for
 *    packed INT4 weights), else W8A8_ERR_MISALIGNED.  K is at most 32768
 *    (else W8A8_ERR_INVALID_ARG); this also keeps every INT32 sum in range
 *    (127 * 127 * 32768 < 2^31).
 *  - group_size is 0 (one scale per row: per-token activations,
 *    per-output-channel weights), 64 or 128; K % group_size must be 0.
 *  - M == 0 or N == 0 is an empty problem: the call returns W8A8_OK and
 *    launches nothing.  Negative sizes and K <= 0 are W8A8_ERR_INVALID_ARG.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream).  Argument errors are detected on the host before any
 *    launch, and then no output is touched.
 *  - Inputs must be finite; the result of a NaN or Inf input is unspecified.
 *  - Rounding: scale = absmax / qmax with one IEEE fp32 division; q =
 *    clamp(rint(x / scale), -qmax, qmax) with an IEEE fp32 division and
 *    ties to even; a group whose absmax is 0 gets scale 0 and q 0; -128 is
 *    never produced.  Dequant: per channel y = fp16_rn((float)acc *
 *    (s_a * s_w)); per group y = fp16_rn(sum over g of (float)acc_g *
 *    (s_a,g * s_w,g)), INT32 partials per group.
 */
#ifndef W8A8_H
#define W8A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t w8a8_half;   /* IEEE binary16 bit pattern */
typedef void *w8a8_stream_t;  /* a cudaStream_t */

/* Status codes returned by every call. */
#define W8A8_OK 0
#define W8A8_ERR_INVALID_ARG 1        /* null pointer, bad size, bad group_size */
#define W8A8_ERR_MISALIGNED 2         /* pointer not 16-byte aligned, K % 16 */
#define W8A8_ERR_UNSUPPORTED_DEVICE 3 /* current device is not compute 10.3 */
#define W8A8_ERR_CUDA 4               /* a CUDA runtime call or launch failed */
#define W8A8_ERR_TIMEOUT 5            /* a bounded device-side wait gave up */
#define W8A8_ERR_WORKSPACE 6          /* workspace too small */
#define W8A8_ERR_INDEX 7              /* a cache index on the device was out of range */

/* 1 if the current CUDA device is a compute-capability 10.3 GPU (GB300)
 * that this library's kernels were built for, else 0.  The analogue of the
 * SDK's is_available() ("cider 설치와 사용법"). */
int w8a8_is_available(void);

/* Static, human-readable name of a status code. */
const char *w8a8_status_string(int status);

/* Reads and clears the device-side error words that the kernels set when a
 * bounded wait on the tensor-core pipeline gives up, or when a GEMM kernel
 * finds its shared memory not 1 KB aligned and returns without doing
 * anything (both leave the outputs of that call undefined), or when a
 * key/value cache kernel meets a slot, page, length or query offset outside
 * its range (which it leaves out).  Synchronizes `stream`.  Returns W8A8_OK,
 * W8A8_ERR_TIMEOUT (for either of the first two causes, whatever else was
 * reported), W8A8_ERR_INDEX or W8A8_ERR_CUDA. */
int w8a8_check_status(w8a8_stream_t stream);

/* Offline INT8 weight quantization ("cider 설치와 사용법":
 * quantize_weight_int8(W) -> (w_int8, scale); mode table: symmetric INT8).
 *   W        fp16 [N, K]
 *   Wq       int8 [N, K]        (out)
 *   scale_w  fp32 [N, G]        (out) absmax / 127 per row (per group)
 * group_size 0 = per output channel. */
int quantize_weight_int8(const w8a8_half *W, int N, int K, int group_size,
                         int8_t *Wq, float *scale_w, w8a8_stream_t stream);

/* Offline INT4 weight quantization and packing ("cider 설치와 사용법":
 * pack_weight_int4(W) -> (packed, scale); mode table: W4A8, INT4 packed in
 * uint8).  Per output channel: s4 = absmax / 7, q4 = clamp(rint(W / s4),
 * -7, 7); byte j of row n holds q4[n, 2j] in its low nibble and
 * q4[n, 2j+1] in its high nibble, both two's complement.
 *   W        fp16 [N, K], K % 32 == 0
 *   Wp       uint8 [N, K/2]     (out)
 *   scale_w  fp32 [N]           (out) */
int pack_weight_int4(const w8a8_half *W, int N, int K, uint8_t *Wp,
                     float *scale_w, w8a8_stream_t stream);

/* Online per-token activation quantization ("INT8 TensorOps 커널 설계",
 * steps 1-2; mode table: INT8 per token).
 *   x        fp16 [M, K]
 *   xq       int8 [M, K]        (out)
 *   scale_a  fp32 [M, G]        (out) absmax / 127 per row (per group) */
int quantize_act_per_token(const w8a8_half *x, int M, int K, int group_size,
                           int8_t *xq, float *scale_a, w8a8_stream_t stream);

/* W8A8 GEMM with fused dequant ("INT8 TensorOps 커널 설계" steps 3-4;
 * "입도(Granularity)" for group_size > 0).  Exact INT32 (per-group) sums,
 * then the fp32 rescale and one fp16 rounding.
 *   xq       int8 [M, K],  scale_a fp32 [M, G]
 *   Wq       int8 [N, K],  scale_w fp32 [N, G]
 *   y        fp16 [M, N]        (out)
 * Any M >= 1 is accepted (M == 1 runs the matrix-vector kernel). */
int w8a8_gemm(const int8_t *xq, const float *scale_a, const int8_t *Wq,
              const float *scale_w, int M, int N, int K, int group_size,
              w8a8_half *y, w8a8_stream_t stream);

/* W8A8 matrix-vector product for decode (the SDK's INT8 MV kernel for
 * seq_len == 1, "cider 소개", section "cider의 동작 방식과 자동 경로 선택";
 * per channel or per group).  Same arguments as w8a8_gemm; M must be 1 (else
 * W8A8_ERR_INVALID_ARG).
 * Ordering: the matrix-vector kernel is launched with programmatic stream
 * serialization, and it may start reading Wq (only Wq) before the previous
 * kernel on the stream has finished when that kernel lets its dependents
 * start early (executes griddepcontrol.launch_dependents).  A kernel that does
 * so, and every kernel behind it that does so too, may still be running then.
 * So do not write Wq in such a kernel of your own, unless one that does not
 * (or an event, a copy, a synchronisation) lies between it and this call.
 * Every entry point of this library that gives codes in a weight's format
 * (INT8, packed INT4, e4m3), of weights or of activations, writes them without
 * letting dependents start early: they may be the Wq of any later call on the
 * stream.  The same holds for
 * w4a8_gemm and linear with M == 1. */
int w8a8_mv(const int8_t *xq, const float *scale_a, const int8_t *Wq,
            const float *scale_w, int M, int N, int K, int group_size,
            w8a8_half *y, w8a8_stream_t stream);

/* W4A8 GEMM ("cider 설치와 사용법": w4a8_linear; mode table: W4A8,
 * unpack -> INT8 matmul).  Per-channel INT4 weights packed as
 * pack_weight_int4 writes them, per-token INT8 activations.
 *   xq int8 [M, K], scale_a fp32 [M]; Wp uint8 [N, K/2], scale_w fp32 [N];
 *   y fp16 [M, N] (out); K % 32 == 0.  M == 1 runs the W4A8 matrix-vector
 *   kernel. */
int w4a8_gemm(const int8_t *xq, const float *scale_a, const uint8_t *Wp,
              const float *scale_w, int M, int N, int K, w8a8_half *y,
              w8a8_stream_t stream);

/* quantize_act_per_token with the INT8 codes written as fp16 values (every
 * code in [-127, 127] is an fp16 integer exactly): the operand format the
 * tensor-core GEMM reads without converting, which linear() uses for M > 1.
 *   x        fp16 [M, K]
 *   xq_h     fp16 [M, K]        (out) the codes q, as fp16
 *   scale_a  fp32 [M, G]        (out)
 * Ordering: the kernel lets the next kernel on the stream start early
 * (griddepcontrol.launch_dependents), which only matters to a kernel
 * launched with programmatic stream serialization; the library's GEMM is,
 * and it waits for this kernel to finish before reading any input. */
int quantize_act_per_token_h(const w8a8_half *x, int M, int K, int group_size,
                             w8a8_half *xq_h, float *scale_a, w8a8_stream_t stream);

/* The GEMM of w8a8_gemm (wbits 8) or w4a8_gemm (wbits 4, group_size 0) with
 * the activation codes given as fp16 values, as quantize_act_per_token_h
 * writes them.  Codes outside [-127, 127] or not integral are outside the
 * contract.  Always the tensor-core GEMM, for any M >= 1.
 *   xq_h fp16 [M, K], scale_a fp32 [M, G]; Wq int8 [N, K] or packed uint8
 *   [N, K/2]; scale_w fp32 [N, G]; y fp16 [M, N] (out)
 * The GEMM (any M, every GEMM entry point) is launched with programmatic
 * stream serialization: its set-up may overlap the previous kernel on the
 * stream, and it reads no input before that kernel has finished. */
int w8a8_gemm_h(const w8a8_half *xq_h, const float *scale_a, const void *Wq,
                const float *scale_w, int M, int N, int K, int group_size, int wbits,
                w8a8_half *y, w8a8_stream_t stream);

/* Bytes of workspace that linear() needs for M rows of K activations: the
 * activation codes (fp16 values for M > 1, INT8 for M == 1) and their fp32
 * scales, each region 256-byte aligned. */
size_t w8a8_linear_workspace_bytes(int M, int K, int group_size);

/* The whole layer, CiderLinear's forward ("cider 소개", section "cider의
 * 동작 방식과 자동 경로 선택": seq_len > 1 -> INT8 GEMM, seq_len == 1 ->
 * INT8 MV kernel).  M == 1: one kernel quantizes the row and runs the
 * matrix-vector product with the fused dequant.  2 <= M <= 8, per channel,
 * with the codes of the rows (padded to 2, 4 or 8) within 64 KB: one kernel
 * quantizes the rows and runs the few-row product on the same weight
 * stream.  In both, the workspace is checked but not written (see w8a8_mv
 * for the ordering rule of those kernels).  Otherwise: quantize x per token
 * into the workspace (quantize_act_per_token_h), then the GEMM
 * (w8a8_gemm_h) with the fused dequant.  Same quantization rule everywhere.
 *   x        fp16 [M, K]
 *   Wq       int8 [N, K] (wbits 8) or packed uint8 [N, K/2] (wbits 4)
 *   scale_w  fp32 [N, G] (wbits 4 requires group_size 0)
 *   workspace device buffer of at least w8a8_linear_workspace_bytes(M, K,
 *            group_size) bytes, 256-byte aligned, else W8A8_ERR_WORKSPACE
 *   y        fp16 [M, N] (out) */
int linear(const w8a8_half *x, const void *Wq, const float *scale_w, int M,
           int N, int K, int group_size, int wbits, void *workspace,
           size_t ws_bytes, w8a8_half *y, w8a8_stream_t stream);

/* linear() with no workspace argument, for callers that cannot allocate
 * device memory on their execution path (for example a serving runtime's
 * per-request path, where cudaMalloc may synchronize the device and fail
 * under memory pressure, or a plugin inside a host framework that owns all
 * device memory and exposes no allocator).  No counterpart on the method's
 * pages: an addition of this library.
 *   Arguments as linear(), minus workspace / ws_bytes.  The workspace is a
 *   fixed 8 MiB array in the library's device memory (held by every GPU that
 *   loads the library until the process exits); a problem whose
 *   w8a8_linear_workspace_bytes(M, K, group_size) exceeds 8 MiB returns
 *   W8A8_ERR_WORKSPACE and touches nothing.  Calls no allocator.
 *   All calls on a device share the array: calls whose kernels overlap on
 *   the GPU (unordered streams) race; calls on one stream are safe.  The
 *   first call on a device looks up the array's address, once per device;
 *   make it before any stream capture begins. */
int linear_noalloc(const w8a8_half *x, const void *Wq, const float *scale_w, int M,
                   int N, int K, int group_size, int wbits, w8a8_half *y,
                   w8a8_stream_t stream);

/* The weight-only product the method is measured against (W8A16 / W4A16:
 * "Apple Silicon의 AI 한계치는 당신의 생각보다 높습니다", the section on
 * MLX's weight-only quantization -- integer weights dequantized and
 * multiplied with fp16 activations; "cider 소개", mode table, W8A16 /
 * W4A16 rows, and the w8a16 / w4a16 columns of the latency table).  The
 * activations stay fp16: y = x . (q * s_w)^T, accumulated in fp32 on the
 * tensor cores (the integer codes are exact fp16 operands), then scaled by
 * s_w (per group: each group's sum scaled and added in ascending order) and
 * rounded once to fp16.  Not bit-exact against the double-precision
 * definition: within |dy| <= 2e-3 * max|y| + one fp16 ulp.
 *   x        fp16 [M, K]
 *   Wq       int8 [N, K] (wbits 8) or packed uint8 [N, K/2] (wbits 4, as
 *            pack_weight_int4 writes them; requires group_size 0)
 *   scale_w  fp32 [N, G]
 *   y        fp16 [M, N]       (out)
 * Any M >= 1 (the tensor-core GEMM, launched like w8a8_gemm_h). */
int weight_only_gemm(const w8a8_half *x, const void *Wq, const float *scale_w, int M, int N,
                     int K, int group_size, int wbits, w8a8_half *y, w8a8_stream_t stream);

/* Test export of step 3 alone ("INT8 TensorOps 커널 설계": INT32
 * accumulation): acc[m, n, g] = sum over k in group g of xq[m, k] *
 * Wq[n, k], exact, as int32 [M, N, G], through the same tensor-core
 * contraction the GEMM uses.  wbits 4 reads packed weights [N, K/2] and
 * needs group_size 0. */
int w8a8_gemm_i32(const int8_t *xq, const void *Wq, int M, int N, int K,
                  int group_size, int wbits, int32_t *acc,
                  w8a8_stream_t stream);

/* Test hook of the failure path (the method has no counterpart): sets, for
 * the launches of the tensor-core GEMM, of the cache attention and of the
 * 8-bit float products that follow (every entry point that runs them), the
 * limit of their bounded device-side waits in SM clock cycles (0 = the
 * default, about 2 s) and, with skip_first_copy = 1, leaves the first
 * weight-staging copy, or copy or hand-over of keys, of each CTA out, so that
 * the wait for it gives up: the kernel then returns early, its outputs are undefined, and
 * w8a8_check_status() reports W8A8_ERR_TIMEOUT.  No fault, trap or hang is
 * involved; the kernel still lets every copy it issued land before it
 * exits.  Process-wide; w8a8_test_set_fault(0, 0) restores normal
 * operation.  Returns W8A8_ERR_INVALID_ARG for a negative limit or a flag
 * other than 0 / 1. */
int w8a8_test_set_fault(long long wait_limit_cycles, int skip_first_copy);

/* ---- quantized key/value cache and attention over it -------------------
 *
 * What a decoder layer has between two linear() calls: the k and v of the
 * fused projection go into a paged cache in the library's number format
 * (symmetric, one fp32 scale per token and kv head: the per-token rule of
 * quantize_act_per_token over the head_dim elements of a head; INT8, or INT4
 * packed as pack_weight_int4 packs it), and attention reads it.  No
 * counterpart on the method's pages, which stop at the linear layer: an
 * addition of this library.
 *
 * The conventions at the top of this file hold, with these additions:
 *  - head_dim D is 64 or 128; page_size is a power of two from 16 to 1024;
 *    q_heads is a multiple of kv_heads (query head h reads kv head
 *    h / (q_heads / kv_heads)).
 *  - k, v and q are fp16 rows of D contiguous elements addressed by a token
 *    and a head stride in elements (so slices of a fused projection go in as
 *    they are): 16-byte aligned, strides non-negative multiples of 8.
 *  - Values that live on the device (slots, tables, lengths, offsets) cannot
 *    be checked by the host.  The kernels check them: what lies outside its
 *    range is left out (no access leaves a buffer), and
 *    w8a8_check_status() then reports W8A8_ERR_INDEX. */

/* A paged cache of one layer (device pointers, owned by the caller, 16-byte
 * aligned, contiguous).  Slot s is token s % page_size of page
 * s / page_size. */
typedef struct w8a8_kv_cache {
  void *k_codes;   /* [num_pages, kv_heads, page_size, D] int8 (bits 8) or
                      [num_pages, kv_heads, page_size, D/2] uint8 (bits 4) */
  void *v_codes;   /* the same */
  float *k_scale;  /* [num_pages, kv_heads, page_size] */
  float *v_scale;
  long long num_pages;
  int kv_heads, page_size, head_dim, bits;
} w8a8_kv_cache;

/* Quantizes T tokens' k and v into their slots.
 *   k, v   fp16 [T, kv_heads, D] by strides
 *   slots  int64 [T]; a negative slot is not stored (padding); two tokens
 *          with one slot race
 * Non-finite inputs are defined here: NaN is stored as 0, +-Inf as +-65504,
 * so a written cache holds finite values only. */
int kv_cache_write(const w8a8_half *k, long long k_token_stride, long long k_head_stride,
                   const w8a8_half *v, long long v_token_stride, long long v_head_stride,
                   const int64_t *slots, int T, const w8a8_kv_cache *cache,
                   w8a8_stream_t stream);

/* Reads T tokens back: k, v fp16 [T, kv_heads, D] contiguous (out),
 * fp16_rn((float)code * scale); zeros for a negative slot. */
int kv_cache_read(const int64_t *slots, int T, const w8a8_kv_cache *cache, w8a8_half *k,
                  w8a8_half *v, w8a8_stream_t stream);

/* Bytes of workspace of kv_cache_attention() for these sizes (0 for invalid
 * ones); grows with none of the device-side values. */
size_t kv_cache_attention_workspace_bytes(int T, int q_heads, int B, int max_q, int table_width,
                                          const w8a8_kv_cache *cache);

/* Attention of T query tokens over the cached tokens of B sequences.
 *   q           fp16 [T, q_heads, D] by strides
 *   q_offsets   int32 [B + 1]: sequence b has queries q_offsets[b] ..
 *               q_offsets[b + 1] - 1; NULL: one query per sequence (T == B)
 *   max_q       upper bound of the queries of one sequence (T is always
 *               one; a close bound makes a better launch)
 *   block_table int32 [B, table_width]: page ids of the sequence's tokens;
 *               table_width * page_size is at most 2^31 - 65536
 *   seq_lens    int32 [B]: tokens of the sequence in the cache, the queries'
 *               own included (write them first)
 *   softmax_scale  of the scores, 1 / sqrt(D) usually
 *   causal      1: query i of n sits at position seq_len - n + i and sees the
 *               keys up to its own; 0: every key of the sequence
 *   window      > 0 (causal only): it sees the last `window` of these
 *   workspace   at least kv_cache_attention_workspace_bytes(), 256-byte
 *               aligned, else W8A8_ERR_WORKSPACE; its content does not matter
 *   out         fp16 [T, q_heads, D] (out)
 *   lse         fp32 [T, q_heads] (out) natural log of the row's sum of
 *               exponentials, or NULL
 * S_j = softmax_scale * k_scale[j] * (q . code_k[j]) with the codes exact and
 * fp32 sums; out = sum_j softmax(S)_j * v_scale[j] * code_v[j], one fp16
 * rounding at the end.  A query that sees no key gets out 0 and lse -inf, and
 * so does a row that no sequence owns: before q_offsets[0], from q_offsets[B]
 * on (a batch padded to a fixed T), or beyond a sequence's first max_q (which
 * is reported, the others taken as if there were max_q).  Offsets out of
 * order are reported; the rows that they touch are then undefined.
 * Cache rows that no query sees (past seq_len, before every window) may hold
 * anything; of their pages only one that also holds a seen row has to be in
 * the cache.  Results do not depend on the order in which blocks run. */
int kv_cache_attention(const w8a8_half *q, long long q_token_stride, long long q_head_stride,
                       int T, int q_heads, const int32_t *q_offsets, int B, int max_q,
                       const int32_t *block_table, int table_width, const int32_t *seq_lens,
                       const w8a8_kv_cache *cache, float softmax_scale, int causal, int window,
                       void *workspace, size_t ws_bytes, w8a8_half *out, float *lse,
                       w8a8_stream_t stream);

/* ---- the norm in front of a layer --------------------------------------
 *
 * Root-mean-square norm of fp16 rows, with the residual's addition before it
 * and, instead of fp16 values, the 8-bit codes that the next layer reads:
 *   h = fp16_rn(x + residual)            (h = x without a residual)
 *   v = h * weight / sqrt(mean(h^2) + eps)
 * v is an fp32 value (h * weight is exact, the sums are fp32); it is rounded
 * once, to fp16 or to codes (INT8: 127 v / max|v|, rounded to the nearest; a
 * quotient within 2^-16 of a tie may go either way).  A row of zeros with eps 0
 * gives zeros.  No
 * counterpart on the method's pages, which start at the layer's input: an
 * addition of this library.  The conventions at the top of this file hold;
 * x, residual, weight and all outputs are 16-byte aligned, K is a multiple of
 * 16.
 *   x            fp16 [M, K]
 *   residual     fp16 [M, K], or NULL
 *   weight       fp16 [K]
 *   eps          >= 0, finite
 *   residual_out fp16 [M, K] (out) h; may be residual or x itself; NULL if
 *                and only if residual is NULL
 * Other overlaps of an output with an input are not allowed.
 * Ordering: with fp16 outputs (values, or codes as halves) the kernel lets the
 * next kernel on the stream start early, as quantize_act_per_token_h does. */

/* Code formats of rms_norm_quantize(). */
#define W8A8_CODES_INT8 0 /* int8, scales as quantize_act_per_token */
#define W8A8_CODES_HALF 1 /* the same codes as fp16 values, as quantize_act_per_token_h */
#define W8A8_CODES_FP8 2  /* e4m3, scales as quantize_act_fp8 */

/* y fp16 [M, K] (out). */
int rms_norm(const w8a8_half *x, const w8a8_half *residual, const w8a8_half *weight, int M, int K,
             float eps, w8a8_half *residual_out, w8a8_half *y, w8a8_stream_t stream);

/* Codes and scales of v.
 *   format     W8A8_CODES_INT8 / _HALF: group_size 0, 64 or 128 (K a multiple
 *              of it); q int8 or fp16 [M, K], scale fp32 [M, G].
 *              W8A8_CODES_FP8: group_size 128; q e4m3 [M, K], scale e8m0
 *              [M, ceil(K / 128)]. */
int rms_norm_quantize(const w8a8_half *x, const w8a8_half *residual, const w8a8_half *weight, int M,
                      int K, float eps, int format, int group_size, w8a8_half *residual_out, void *q,
                      void *scale, w8a8_stream_t stream);

/* ---- layers in 8-bit floats ---------------------------------------------
 *
 * The layer and a decoder's gated feed-forward block with e4m3 operands: the
 * tensor cores' 8-bit float rate is twice the fp16 rate that the INT8 layer
 * runs at on this GPU.  No counterpart on the method's pages: an addition of
 * this library.
 *
 * Format of a row of K elements (weights and activations alike): e4m3 codes
 * (1 byte: sign, 4 exponent bits, 3 mantissa bits, largest 448, no
 * infinities) and one e8m0 scale byte b, 2^(b - 127), for every 128
 * consecutive elements, the last group possibly shorter: ceil(K / 128) bytes.
 * The quantizers' scale is the smallest power of two s with max|x| / s <= 448,
 * 1 for a group of zeros and at least 2^-126; a code is e4m3_rn(x / s), ties
 * to even.  The products take any codes but NaN (0x7f, 0xff) and scale bytes
 * 1 .. 254.
 *
 * The conventions at the top of this file hold, with K (and F) a multiple of
 * 16, code pointers 16-byte aligned and scale pointers at any address.  Sums
 * are fp32 (the products of two codes are exact), rounded once to the output's
 * type.  Their order depends on N, K, the class of M (up to 16, 64, 128, 384,
 * 1024, 2560, 8192 rows, more) and, for the gated pair, on the form of the output
 * (fp16 or codes), not on timing: within a class a row's result does not depend
 * on the other rows of the batch.  No output may overlap an input. */

/* fp16 rows to codes and scales.
 *   x   fp16 [M, K];  xq e4m3 [M, K] (out);  scale_a e8m0 [M, ceil(K/128)] (out) */
int quantize_act_fp8(const w8a8_half *x, int M, int K, uint8_t *xq, uint8_t *scale_a,
                     w8a8_stream_t stream);
/* The same for weights [N, K] (a launch that no later kernel overlaps). */
int quantize_weight_fp8(const w8a8_half *W, int N, int K, uint8_t *Wq, uint8_t *scale_w,
                        w8a8_stream_t stream);

/* y[m, n] = fp16_rn(sum_k x[m, k] w[n, k]) over the values that the codes stand
 * for.
 *   xq e4m3 [M, K], scale_a e8m0 [M, ceil(K/128)]; Wq e4m3 [N, K], scale_w e8m0
 *   [N, ceil(K/128)]; y fp16 [M, N] (out)
 * All products here are launched with programmatic stream serialization, and
 * may read the weights (only these and their scales) before the previous kernel
 * on the stream has finished, under the rule of w8a8_mv: codes that any entry
 * point of this library wrote earlier on the stream may be the weights, so
 * products of two activations need nothing more. */
int fp8_gemm(const uint8_t *xq, const uint8_t *scale_a, const uint8_t *Wq, const uint8_t *scale_w,
             int M, int N, int K, w8a8_half *y, w8a8_stream_t stream);

/* Activations of the gated block. */
#define W8A8_GATE_SILU 0 /* g / (1 + exp(-g)); 0 for g below -87 */
#define W8A8_GATE_GELU 1 /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */

/* Both projections of a gated feed-forward block, the activation and the
 * product in one kernel: h[m, f] = act(x Wg^T)[m, f] * (x Wu^T)[m, f], an fp32
 * value, as fp16 (h) or as codes with scales (hq, scale_h).
 *   xq, scale_a  as fp8_gemm;  Wg, Wu e4m3 [F, K] with scale_g, scale_u
 *   h        fp16 [M, F] (out), or NULL for codes
 *   hq       e4m3 [M, F], scale_h e8m0 [M, ceil(F/128)] (out), both NULL with h;
 *            F a multiple of 16, at most 32768 (the K of a product to come) */
int fp8_gated_gemm(const uint8_t *xq, const uint8_t *scale_a, const uint8_t *Wg,
                   const uint8_t *scale_g, const uint8_t *Wu, const uint8_t *scale_u, int M, int F,
                   int K, int activation, w8a8_half *h, uint8_t *hq, uint8_t *scale_h,
                   w8a8_stream_t stream);

/* Bytes of workspace of fp8_linear() (0 for invalid sizes). */
size_t fp8_linear_workspace_bytes(int M, int K);

/* The whole layer: quantize_act_fp8 into the workspace, then fp8_gemm; for a few
 * rows one kernel that does both, which leaves the workspace alone (it is checked
 * all the same).  The result is that of the two calls, bit for bit.
 *   x fp16 [M, K]; Wq, scale_w as fp8_gemm; y fp16 [M, N] (out)
 *   workspace  at least fp8_linear_workspace_bytes(M, K), 256-byte aligned, else
 *              W8A8_ERR_WORKSPACE; its content does not matter */
int fp8_linear(const w8a8_half *x, const uint8_t *Wq, const uint8_t *scale_w, int M, int N, int K,
               void *workspace, size_t ws_bytes, w8a8_half *y, w8a8_stream_t stream);

/* Bytes of workspace of fp8_feed_forward() (0 for invalid sizes). */
size_t fp8_feed_forward_workspace_bytes(int M, int K, int F);

/* The whole gated feed-forward block: quantize_act_fp8, fp8_gated_gemm to codes,
 * fp8_gemm (the first two as one kernel for a few rows, with the same result): y = ((act(x Wg^T) * (x Wu^T)) as codes) Wd^T.
 *   x fp16 [M, K]; Wg, Wu e4m3 [F, K]; Wd e4m3 [N, F]; y fp16 [M, N] (out)
 *   workspace  at least fp8_feed_forward_workspace_bytes(M, K, F), 256-byte
 *              aligned, else W8A8_ERR_WORKSPACE; its content does not matter */
int fp8_feed_forward(const w8a8_half *x, const uint8_t *Wg, const uint8_t *scale_g,
                     const uint8_t *Wu, const uint8_t *scale_u, const uint8_t *Wd,
                     const uint8_t *scale_d, int M, int K, int F, int N, int activation,
                     void *workspace, size_t ws_bytes, w8a8_half *y, w8a8_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
