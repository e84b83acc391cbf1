/*
 * bsfp.h -- C ABI of libbsfp: block-scaled 4-bit (and 8-bit) quantization
 * and quantized matmul on AMD Instinct MI355X (gfx950).
 *
 * Formats (the contract; with b = bits, element k of a row sits at bit
 * b*(k % (32/b)) of uint32 word k/(32/b): for 4 bits nibble k%8 of word k/8,
 * low nibble first, for 8 bits byte k%4 of word k/4; every tensor row-major
 * and contiguous):
 *
 *   BSFP_NVFP4  bits 4, group 16.  codes: E2M1 (FP4) packed 8 per uint32.
 *               scales: uint8 E4M3 (OCP E4M3FN) per 16-element group.
 *               global_scale: optional fp32 g = amax/(448*6) per tensor.
 *               Value = E2M1(c) * E4M3(S) * g.
 *               (native NVFP4 is group 16 / bits 4: "feat(quant): backend
 *               quantization capability table ...", Gate impact; 448 and 6
 *               are F8E4M3_MAX and F4E2M1_MAX in "mlx 0.30.7.3 -> 0.30.7.6",
 *               qqmm_utils.cu.)
 *   BSFP_MXFP4  bits 4, group 32.  codes: E2M1.  scales: uint8 E8M0
 *               (2^(S-127)).  Value = E2M1(c) * 2^(S-127).
 *               (MX scale arm of the bits == 4 quantizer: "perf(cuda): enable
 *               hardware NVFP4/MXFP4 conversion on Blackwell builds",
 *               Current Behavior.)
 *   BSFP_AFFINE bits 4, group 64.  codes: unsigned 0..15.  scales, biases:
 *               bf16 per group.  Value = s*q + b.
 *               (affine 4-bit / group 64: "epic: NVIDIA Volta (sm_70)
 *               inference acceleration program", Baseline.)
 * Format variants ("feat(quant): backend quantization capability table
 * ...", Context: the affine 4/8-bit and mxfp8 modes a ROCm backend runs;
 * Gate impact: its GEMV groups 32, 64, 128):
 *   BSFP_AFFINE bits 4 or 8, group 32, 64 or 128.  codes unsigned
 *               0..2^bits-1.  Value = s*q + b.
 *   BSFP_MXFP8  bits 8, group 32.  codes: E4M3 (OCP E4M3FN) bytes.  scales:
 *               uint8 E8M0.  Value = E4M3(c) * 2^(S-127).
 *   Entry points: bsfp_quantize, bsfp_dequantize, bsfp_qmv (x of at most
 *   64 KB, M * K * 2 bytes) and bsfp_qmm_dense take every format;
 *   bsfp_qmm takes the three base formats, bsfp_quantize_sr NVFP4 and
 *   MXFP4.  Elsewhere a variant returns BSFP_ERR_UNSUPPORTED.
 *
 *   Codes and scales are uint32 [rows, cols*bits/32] and [rows, cols/group]; the
 *   packed shape follows quantize_input in "mlx 0.30.7.3 -> 0.30.7.6"
 *   (qqmm.cpp): last dim = cols*bits/32.  Scales are linear (not the tiled
 *   layout that file builds for cuBLASLt).
 *
 * Quantization rounds to nearest even and saturates (cvt.rn.satfinite.
 * e2m1x2.f32 in "perf(cuda): enable hardware NVFP4/MXFP4 conversion on
 * Blackwell builds", Problem / Background).  Block scales:
 *   NVFP4  S = E4M3(bamax / (6*g)), codes = E2M1(x * (1 / (E4M3(S)*g)))
 *   MXFP4  e = floor(log2 bamax) - 2, codes = E2M1(x * 2^-e), S = e + 127
 *   AFFINE s = bf16((max-min)/15), b = bf16(min), q = rint((x-b)/s) in 0..15
 *          (b bits: 2^b - 1 in place of 15)
 *   MXFP8  e = floor(log2 bamax) - 8, codes = E4M3(x * 2^-e) (saturating at
 *          448, sign bit kept), S = e + 127 (OCP MX v1.0 for E4M3 elements)
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE pointers of the current HIP device, 16-byte
 *     aligned; bf16 travels as uint16 bit patterns.  The caller owns and
 *     allocates every buffer (the library allocates no device memory, never
 *     frees, and never writes its inputs; the one exception is the static
 *     workspace of bsfp_qmm_noalloc, which lives in the library's code
 *     object on each GPU).
 *   - Work is enqueued on `stream` (a hipStream_t; NULL is the null stream)
 *     with no host synchronization.
 *   - Functions never throw and never abort.  Argument errors are detected on
 *     the host before anything is enqueued and return BSFP_ERR_ARG; a
 *     format outside the ones above returns BSFP_ERR_UNSUPPORTED; a failed
 *     launch returns BSFP_ERR_DEVICE.  bsfp_last_error() then describes it.
 *     (A C++ exception crossing a language bridge terminates the process, and
 *     an unsupported group size that throws aborts a whole test binary:
 *     "feat(quant): backend quantization capability table ...", Gate impact.)
 */
#ifndef BSFP_H
#define BSFP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BSFP_AFFINE = 0, BSFP_MXFP4 = 1, BSFP_NVFP4 = 2, BSFP_MXFP8 = 3 } bsfp_mode;

typedef enum {
    BSFP_OK = 0,
    BSFP_ERR_ARG = 1,          /* bad pointer, size, alignment or shape */
    BSFP_ERR_UNSUPPORTED = 2,  /* (mode, bits, group) outside the contract */
    BSFP_ERR_DEVICE = 3        /* launch failure reported by the runtime */
} bsfp_status;

/* Activation handling of bsfp_qmm. */
typedef enum {
    BSFP_ACT_BF16 = 0,  /* weight-only: y = x . dq(W)^T, x stays bf16 */
    BSFP_ACT_SAME = 1   /* qq: x is quantized with W's mode first, then
                           y = alpha * dq0(q(x)) . dq0(W)^T */
} bsfp_act;

/* NVFP4 global-scale handling of bsfp_quantize. */
typedef enum {
    BSFP_GS_NONE = 0,     /* no global scale: g = 1 */
    BSFP_GS_COMPUTE = 1,  /* amax over the tensor -> *amax, g = amax/2688 ->
                             *global_scale (both must be non-NULL) */
    BSFP_GS_GIVEN = 2     /* use the device fp32 *global_scale as g */
} bsfp_gs;

typedef void* bsfp_stream; /* hipStream_t */

/* A quantized tensor: logical bf16 shape [rows, cols]. */
typedef struct {
    int32_t mode;          /* bsfp_mode */
    int32_t bits;          /* 4 */
    int32_t group_size;    /* 16 NVFP4, 32 MXFP4, 64 AFFINE */
    int64_t rows, cols;    /* cols % group_size == 0; rows * cols <= 2^40 */
    uint32_t* codes;       /* [rows, cols/8] */
    void* scales;          /* NVFP4/MXFP4 uint8, AFFINE bf16: [rows, cols/group] */
    uint16_t* biases;      /* AFFINE bf16 [rows, cols/group]; NULL otherwise */
    float* global_scale;   /* NVFP4 g (device fp32) or NULL for none */
    float* amax;           /* NVFP4 tensor amax (device fp32), written by
                              BSFP_GS_COMPUTE; may be NULL otherwise */
} bsfp_qtensor;

/*
 * bsfp_amax: *amax_out = max |x_i| over the n bf16 values at x (device
 * fp32).  The source of the NVFP4 global scale (alpha = amax_x*amax_w /
 * (448*6)^2: "mlx 0.30.7.3 -> 0.30.7.6", qqmm_utils.cu,
 * compute_qqmm_pointers).  n >= 0 (n == 0 gives 0).  Exact and independent
 * of reduction order.
 */
bsfp_status bsfp_amax(const uint16_t* x, int64_t n, float* amax_out,
                      bsfp_stream stream);

/*
 * bsfp_quantize: bf16 x [q->rows, q->cols] -> q->codes, q->scales (and
 * q->biases for AFFINE; g and amax for NVFP4 per gs).  fp_quantize /
 * affine_quantize of "mlx 0.30.7.3 -> 0.30.7.6" (quantized.h, quantized.cpp
 * fast::Quantize::eval_gpu).  gs is a bsfp_gs value and is ignored unless
 * mode is NVFP4.  Codes and scales are bit-exact to the documented rules.
 */
bsfp_status bsfp_quantize(const uint16_t* x, const bsfp_qtensor* q, int32_t gs,
                          bsfp_stream stream);

/*
 * bsfp_quantize_sr: bsfp_quantize with stochastic rounding of the E2M1
 * codes, for NVFP4 and MXFP4 (the USE_SR variant of the 4-bit quantizer,
 * "perf(cuda): enable hardware NVFP4/MXFP4 conversion on Blackwell builds",
 * Current Behavior).  Scales, global scale and amax are exactly those of
 * bsfp_quantize.  Element k (row-major over [rows, cols]) takes the random
 * word rbits[k]: with its scaled value v between E2M1 grid magnitudes
 * lo < hi, the code is hi when (rbits[k] >> 8) * 2^-24 < (|v| - lo) /
 * (hi - lo), else lo (both sides exact in fp32); grid values stay, |v| >= 6
 * saturates, the sign bit follows v.  The rounding is unbiased up to 2^-24
 * of the grid spacing.  rbits: device pointer to q->rows * q->cols uint32,
 * 16-byte aligned, owned by the caller, read only; the caller chooses how
 * it is drawn.  AFFINE returns BSFP_ERR_UNSUPPORTED; other errors as for
 * bsfp_quantize.
 */
bsfp_status bsfp_quantize_sr(const uint16_t* x, const bsfp_qtensor* q, int32_t gs,
                             const uint32_t* rbits, bsfp_stream stream);

/*
 * bsfp_quantize_ws: bsfp_quantize (rbits == NULL) or bsfp_quantize_sr
 * (rbits != NULL, with its requirements) with a caller workspace.  For
 * NVFP4 with BSFP_GS_COMPUTE (the per-tensor global scale from the tensor
 * amax: fp_quantize with a global scale, "mlx 0.30.7.3 -> 0.30.7.6",
 * quantized.cpp and qqmm_utils.cu) the amax is reduced from per-workgroup
 * partial maxima kept in the workspace instead of an atomic maximum whose
 * accumulator a separate launch must zero first: two kernel launches
 * instead of three, and the same bits (a maximum is exact in any order).
 * Every other mode and gs ignores the workspace and behaves as
 * bsfp_quantize / bsfp_quantize_sr.
 *   workspace: device memory of at least BSFP_QUANTIZE_WS_BYTES bytes,
 *   4-byte aligned, owned by the caller; its contents on entry are ignored
 *   and undefined on return, and calls in flight at the same time need
 *   separate workspaces.  May be NULL where it is ignored.
 * Errors: those of bsfp_quantize / bsfp_quantize_sr, and BSFP_ERR_ARG for a
 * needed workspace that is NULL, misaligned or smaller than
 * BSFP_QUANTIZE_WS_BYTES.  Nothing is launched on an error.
 */
#define BSFP_QUANTIZE_WS_BYTES 1024
bsfp_status bsfp_quantize_ws(const uint16_t* x, const bsfp_qtensor* q, int32_t gs,
                             const uint32_t* rbits, void* workspace,
                             int64_t workspace_bytes, bsfp_stream stream);

/*
 * bsfp_dequantize: q -> bf16 out [q->rows, q->cols].  fp_dequantize /
 * affine_dequantize of "mlx 0.30.7.3 -> 0.30.7.6" (quantized.cpp).
 *   NVFP4  bf16((E2M1 * E4M3) * g)  (g = 1 when q->global_scale is NULL)
 *   MXFP4  bf16(E2M1 * 2^(S-127))
 *   AFFINE bf16(fma(s, q, b))
 */
bsfp_status bsfp_dequantize(const bsfp_qtensor* q, uint16_t* out,
                            bsfp_stream stream);

/*
 * bsfp_qmv: decode GEMV, y[m, n] = sum_k x[m, k] * dq(W)[n, k] for
 * m < M <= 8, with W = w [N = w->rows, K = w->cols] and x bf16 [M, K].
 * Weights are dequantized in registers and accumulated in fp32; y is bf16
 * [M, N] (round to nearest even).  NVFP4 includes W's global scale when
 * present.  ("epic: NVIDIA Volta (sm_70) inference acceleration program",
 * Diagnosis item 3: qmv must accumulate in float; fp_qmv(w, scales, x, out,
 * bits, group_size, M, N, K) in "mlx 0.30.7.3 -> 0.30.7.6", qqmm.cpp.)
 */
bsfp_status bsfp_qmv(const uint16_t* x, int64_t M, const bsfp_qtensor* w,
                     uint16_t* y, bsfp_stream stream);

/*
 * bsfp_qmv_batch: the decode GEMV of bsfp_qmv for `count` weight matrices
 * that share x, y_i[m, n] = sum_k x[m, k] * dq(W_i)[n, k] for i < count,
 * 1 <= count <= BSFP_QMV_BATCH_MAX.  A decoder's projections that read the
 * same activations (gate and up of an MLP) are such a set; the decode
 * weight stream the call serves is that of "epic: NVIDIA Volta (sm_70)
 * inference acceleration program", Baseline (measured), qmv per layer.
 * w[i] (host array of count descriptors) must share mode, bits, group size
 * and K (cols); rows may differ.  y[i] (host array of count device pointers)
 * is bf16 [M, w[i]->rows], 16-byte aligned.  With one row of x and a base
 * format the matrices run as one launch (their rows dealt over the CUs
 * together, so the launch's fixed start-up and drain are paid once); each
 * output row is computed exactly as bsfp_qmv computes it.  Otherwise the
 * matrices run one launch each.  Errors: BSFP_ERR_ARG for a count outside
 * 1..BSFP_QMV_BATCH_MAX, null arrays or entries, descriptors that differ in
 * mode, bits, group size or K, and everything bsfp_qmv rejects;
 * BSFP_ERR_UNSUPPORTED as bsfp_qmv.  Nothing is launched on an error.
 */
#define BSFP_QMV_BATCH_MAX 4
bsfp_status bsfp_qmv_batch(const uint16_t* x, int64_t M, const bsfp_qtensor* const* w,
                           int32_t count, uint16_t* const* y, bsfp_stream stream);

/*
 * bsfp_qmm_workspace_bytes: device scratch bytes that bsfp_qmm needs for
 * (mode, M, K, act): for BSFP_ACT_SAME, x's codes, scales and (NVFP4) amax
 * and g; 0 for BSFP_ACT_BF16.  Returns 0 for unsupported arguments.  The
 * quantized x is the intermediate that QQMatmul::eval_gpu allocates itself
 * before the GEMM (quantize_input with x's packed codes and scales, and the
 * NVFP4 scalars of create_nvfp4_scalars: "mlx 0.30.7.3 -> 0.30.7.6",
 * qqmm.cpp and qqmm_utils.cu); here the caller owns it, so that the library
 * allocates nothing.
 */
size_t bsfp_qmm_workspace_bytes(int32_t mode, int64_t M, int64_t K, int32_t act);

/*
 * bsfp_qmm: prefill GEMM on MFMA, y bf16 [M, N] with N = w->rows,
 * K = w->cols, x bf16 [M, K] row-major, W in the "transposed" MLX layout
 * [N, K] (QQMatmul::eval_gpu, w_transposed = true, lda = ldb = K:
 * "mlx 0.30.7.3 -> 0.30.7.6", qqmm.cpp).
 *   act == BSFP_ACT_BF16: y = x . dq(W)^T (bf16 MFMA; W's codes are staged
 *     in LDS and dequantized in registers, the global scale of NVFP4 applied
 *     to the fp32 sums).
 *   act == BSFP_ACT_SAME: x is quantized into `workspace` with W's mode
 *     (quantize_input in the same file), then y = alpha * dq0(q(x)) .
 *     dq0(W)^T, dq0 = dequantization without the global scale, alpha =
 *     g_x * g_w for NVFP4 with a global scale on W (g_x = amax_x/2688,
 *     computed here), else 1.  The pages' alpha = amax_x*amax_w/(448*6)^2
 *     (create_nvfp4_scalars) is the same quantity up to fp32 rounding.
 *     MXFP4 runs on the gfx950 scaled f8f6f4 MFMA; NVFP4 on fp16 MFMA with
 *     both operands dequantized exactly (E2M1 * E4M3 has at most 6
 *     significant bits, so fp16 holds it).  For M <= 8 (decode) the
 *     same product runs as the GEMV of bsfp_qmv on q(x) dequantized exactly
 *     to bf16, with alpha applied the same way (the M = 1 branch of
 *     QQMatmul, qqmm.cpp, with the global scale of w kept); when x is at
 *     most 64 KB the GEMV quantizes x itself, in one launch.
 * fp32 accumulation, bf16 (RNE) output.  `workspace` must hold
 * bsfp_qmm_workspace_bytes(...) bytes (16-byte aligned) and is overwritten.
 * x and y must be 16-byte aligned, w's scales and biases 4-byte aligned.
 * K must be a multiple of 64 and at most
 * 2^22, M and N at most 2^30 and M * N at most 2^33; BSFP_ACT_SAME needs
 * NVFP4 or MXFP4 weights.
 * Outside these limits the call returns BSFP_ERR_UNSUPPORTED and launches
 * nothing.
 */
bsfp_status bsfp_qmm(const uint16_t* x, int64_t M, const bsfp_qtensor* w,
                     int32_t act, void* workspace, size_t workspace_bytes,
                     uint16_t* y, bsfp_stream stream);

/*
 * Size of the workspace that bsfp_qmm_noalloc keeps in the library's own
 * device memory: 32 MiB per GPU.  It holds the qq workspace of
 * bsfp_qmm_workspace_bytes(...) up to that size, e.g. NVFP4 activations of
 * up to 2^24 elements (M = 3276 at K = 5120) or MXFP4 ones of up to about
 * 6.3 * 10^7.
 */
#define BSFP_NOALLOC_WORKSPACE_BYTES (32u << 20)

/*
 * bsfp_qmm_noalloc: bsfp_qmm for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc).  Same arguments, semantics, limits and errors as bsfp_qmm,
 * except that the workspace is not passed: the call uses a static device
 * array of BSFP_NOALLOC_WORKSPACE_BYTES inside the library, one per GPU,
 * held until the process ends (its address on a device is looked up on the
 * first call there).  The call allocates and frees nothing; the caller still
 * owns x, w and y.  A product whose workspace would exceed that size returns
 * BSFP_ERR_UNSUPPORTED and launches nothing.  Every call on one GPU shares
 * that GPU's array, and it keeps what the last call left there (every byte
 * a call reads it first writes, so nothing needs to start at zero): calls
 * that overlap on one GPU (other streams, other threads) race and must be
 * serialized by the caller.
 */
bsfp_status bsfp_qmm_noalloc(const uint16_t* x, int64_t M, const bsfp_qtensor* w,
                             int32_t act, uint16_t* y, bsfp_stream stream);

/*
 * bsfp_qmm_dense_scratch_bytes: bytes of the bf16 copy of a [rows, cols]
 * weight that bsfp_qmm_dense dequantizes into (rows * cols * 2); 0 for
 * negative arguments.
 */
size_t bsfp_qmm_dense_scratch_bytes(int64_t rows, int64_t cols);

/*
 * bsfp_qmm_dense: the dense prefill path of "mlx: opt-in dense GEMM for
 * nvfp4 prefill (dequantise to bf16 above a row threshold)": W is
 * dequantized to bf16 exactly as bsfp_dequantize does (NVFP4 with its global
 * scale, rounded once to bf16) into `scratch`, then y = x . scratch^T with
 * a dense bf16 GEMM (bf16 MFMA, fp32 accumulation, bf16 RNE output).  x bf16
 * [M, K], y bf16 [M, N], N = w->rows, K = w->cols, every mode.
 * `scratch` is caller-owned device memory of at least
 * bsfp_qmm_dense_scratch_bytes(N, K) bytes, 16-byte aligned, not
 * overlapping x or y; it is overwritten and may be reused for the next
 * layer once the call's stream has passed it, so the transient is bounded
 * by one layer's bf16 copy.  Picking this path above a row threshold is the
 * caller's policy (the binding's qmm(dense_rows=...)).  Same limits and
 * alignment rules as bsfp_qmm with BSFP_ACT_BF16; outside them the call
 * returns BSFP_ERR_UNSUPPORTED (or BSFP_ERR_ARG for bad pointers or a small
 * scratch) and launches nothing.
 */
bsfp_status bsfp_qmm_dense(const uint16_t* x, int64_t M, const bsfp_qtensor* w,
                           void* scratch, size_t scratch_bytes, uint16_t* y,
                           bsfp_stream stream);

/* ------------------------------------------------------------------------
 * A paged key/value cache held in 4 bits, and attention over it.
 *
 * One layer's cache is two quantized tensors, K and V, of one base 4-bit
 * format (NVFP4, MXFP4, AFFINE group 64).  Their rows are
 *     row = (page * kv_heads + head) * page_size + token in the page
 * and their columns the head dimension, so a page of one head is one
 * contiguous run of page_size quantized rows and bsfp_dequantize reads a
 * cache whole.  NVFP4 tensors may each carry a global scale (device fp32),
 * chosen before the first append and the same for all pages.
 *   A request r owns the pages block_table[r, 0 .. ceil(len / page_size)).
 * Its key at position t sits in page block_table[r, t / page_size], token
 * t % page_size; slot = page * page_size + t % page_size names the place.
 *   A step adds q_len[r] tokens to every request.  Their rows of q, k, v and
 * out follow each other by request: rows q_starts[r] .. q_starts[r + 1]
 * belong to request r.
 * Lengths, tables and starts are device memory (a step can be captured in a
 * HIP graph and replayed with other lengths): kernels check what they read
 * there, so a page id outside the cache or a length beyond the table is
 * never dereferenced.
 * ------------------------------------------------------------------------ */
typedef struct {
    const bsfp_qtensor* k;  /* [pages * kv_heads * page_size, head_dim] */
    const bsfp_qtensor* v;  /* the same shape and format */
    int64_t pages;          /* 0 .. 2^31 - 1 */
    int32_t kv_heads;       /* 1 .. 65535 */
    int32_t page_size;      /* tokens per page: 16, 32, 64, 128 or 256 */
} bsfp_kv_cache;

/*
 * bsfp_kv_plan: the tables of one step, built on the GPU from the request
 * lengths in one launch.
 *   in   past_lens [requests]  tokens each request has in the cache
 *        q_lens    [requests]  new tokens of this step (0 allowed)
 *        free_pages [free_count]  ids of free pages, taken in order from
 *                  entry *free_begin on (device int32)
 *   in/out block_table [requests, max_pages]: entries below
 *                  ceil(past / page_size) are read, the entries of pages
 *                  that this step begins are written, no others
 *   out  kv_lens [requests]       past + q
 *        q_starts [requests + 1]  running sum of q_lens, at most `tokens`
 *        slots [tokens] int64, positions [tokens]: of every new token, by
 *                  request; -1 past the last one
 *        state [2]: the free list's next begin; the number of refused
 *                  requests
 * A request takes ceil((past + q) / page_size) - ceil(past / page_size) new
 * pages; requests are served in order.  It is refused when a length is
 * negative, past + q exceeds max_pages * page_size, its tokens end beyond
 * `tokens`, or the free list does not hold the pages of this request and of
 * those before it.  A refused request takes no page, its kv_lens is 0 and
 * its slots and positions are -1, so the append skips its rows and its
 * attention rows are empty; what it has in the cache stays.  (A negative q
 * counts as 0 in q_starts.)
 *   The inputs are not changed, and no output may overlap an input or another
 * output (kv_lens is not past_lens of the same call): the same call again
 * writes the same values.  The caller carries state[0] over as the next step's
 * *free_begin and, as its past_lens, what each request then has in the cache:
 * kv_lens, but past_lens where the request was refused.  bsfp_kv_plan_carry
 * writes that too.
 * Errors: BSFP_ERR_ARG for null pointers, requests < 0, max_pages < 0,
 * tokens outside 0 .. 2^31 - 1, free_count outside 0 .. 2^31 - 1, a page
 * size that is not 16, 32, 64, 128 or 256, or buffers that overlap.
 */
bsfp_status bsfp_kv_plan(const int32_t* past_lens, const int32_t* q_lens, int32_t requests,
                         int32_t page_size, int32_t* block_table, int32_t max_pages,
                         const int32_t* free_pages, int64_t free_count,
                         const int32_t* free_begin, int64_t tokens, int32_t* kv_lens,
                         int32_t* q_starts, int64_t* slots, int32_t* positions, int32_t* state,
                         bsfp_stream stream);

/*
 * bsfp_kv_plan_carry: bsfp_kv_plan with one output more, next_lens [requests]:
 * past + q of an admitted request and past, as given, of a refused one.  It is
 * the next step's past_lens, so a refused request goes on where it stood once
 * there are pages for it.  Errors: those of bsfp_kv_plan.
 */
bsfp_status bsfp_kv_plan_carry(const int32_t* past_lens, const int32_t* q_lens, int32_t requests,
                               int32_t page_size, int32_t* block_table, int32_t max_pages,
                               const int32_t* free_pages, int64_t free_count,
                               const int32_t* free_begin, int64_t tokens, int32_t* kv_lens,
                               int32_t* q_starts, int64_t* slots, int32_t* positions,
                               int32_t* state, int32_t* next_lens, bsfp_stream stream);

/*
 * bsfp_kv_append: quantizes the rows k, v [tokens, kv_heads, head_dim] (bf16;
 * heads and columns contiguous, k_stride / v_stride elements from token to
 * token, so they may be columns of a fused projection's output) by the rules
 * of bsfp_quantize (NVFP4 with the tensor's global scale, BSFP_GS_GIVEN, or
 * none when it is NULL) and writes them at slots[token].  Tokens whose slot
 * is negative or beyond the cache are skipped; slots must differ from each
 * other.  One launch.  k and v 16-byte aligned, strides multiples of 8.
 * Errors: BSFP_ERR_ARG for bad pointers, shapes or strides,
 * BSFP_ERR_UNSUPPORTED for a format or head dimension outside the above
 * (head_dim 64, 128 or 256).
 */
bsfp_status bsfp_kv_append(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                           int64_t v_stride, int64_t tokens, const int64_t* slots,
                           const bsfp_kv_cache* cache, bsfp_stream stream);

/*
 * bsfp_kv_attention: softmax attention of the step's queries over the cache.
 * Row i of request r stands at position p = kv_lens[r] - q_len[r] + i and
 * sees the keys t of its request with 0 <= t <= p and, for window > 0,
 * t > p - window:
 *     s_t = scale * (q . K_t),  lse = log(sum_t exp(s_t)),
 *     out = sum_t exp(s_t - lse) V_t
 * with K, V the values the cache stands for.  Query head h reads kv head
 * h / (heads / kv_heads).  A row that sees no key gives out = 0 and
 * lse = -inf, and so do rows of `out` at or past q_starts[requests].  What
 * the pages hold beyond a request's keys has no effect, and a key none on the
 * rows that do not see it, NaN and infinities among its values included.
 *   q [tokens, heads, head_dim] bf16, q_stride elements from token to token
 *   out [tokens, heads, head_dim] bf16 contiguous; lse [tokens, heads] fp32
 *   or NULL
 *   max_q: no request has more new tokens than this (host knowledge that
 *   chooses and sizes the launches; rows of a request that has more may be
 *   left unwritten)
 *   workspace: bsfp_kv_attention_workspace_bytes(min(tokens, max_q), ...)
 *   bytes, 16-byte aligned, contents ignored; calls in flight at the same
 *   time need separate ones
 * Products run on the matrix cores with fp32 sums; maxima, sums and lse are
 * fp32, probabilities and values have 11 bits.  Probabilities below 2^-40 of a
 * row's largest count as zero, and so do MXFP4 and affine values below 2^-33 of
 * the largest in their quarter of the head dimension among the keys that the
 * row sees.  Results are the same on every call (no atomics).
 * Errors: BSFP_ERR_ARG for bad pointers, shapes, strides, max_q < 1, a scale
 * that is not positive or not finite times log2 e, or a small workspace;
 * BSFP_ERR_UNSUPPORTED for formats or head dimensions outside the above,
 * heads not a multiple of kv_heads, more than 2^31 - 1 rows, or a table of
 * more than 2^31 - 8192 keys (max_pages * page_size).
 */
bsfp_status bsfp_kv_attention(const uint16_t* q, int64_t q_stride, int64_t tokens, int32_t heads,
                              const bsfp_kv_cache* cache, const int32_t* block_table,
                              int32_t max_pages, const int32_t* kv_lens, const int32_t* q_starts,
                              int32_t requests, int32_t max_q, float scale, int32_t window,
                              uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                              bsfp_stream stream);

/*
 * Workspace bytes that suffice for every bsfp_kv_attention call with at most
 * these many tokens and requests, any lengths and any max_q; for calls whose
 * max_q is smaller than tokens it may be given as `tokens` (a decode step,
 * max_q = 1, needs far less).  0 for unsupported arguments.
 */
size_t bsfp_kv_attention_workspace_bytes(int64_t tokens, int32_t heads, int32_t kv_heads,
                                         int32_t head_dim, int32_t requests);

/*
 * bsfp_time_next_launch: measurement hook.  The main kernel of this
 * thread's next bsfp_qmv, bsfp_qmm or bsfp_qmm_dense call (the GEMV, or the
 * GEMM) is launched with hipExtLaunchKernelGGL, whose start and stop
 * events then carry that kernel's own begin and end times, with no extra
 * commands queued between kernels.  start_event and stop_event are hipEvent_t
 * handles the caller created (timing enabled) and still owns; either may be
 * NULL.  One-shot: the pair is cleared by the launch that uses it, and
 * passing two NULLs clears a pending pair; calls of other functions in between
 * leave it pending.  Always returns BSFP_OK.
 */
bsfp_status bsfp_time_next_launch(void* start_event, void* stop_event);

/* Thread-local description of the last non-OK status ("" if none). */
const char* bsfp_last_error(void);

/* Library version and the GPU architecture it was compiled for. */
const char* bsfp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BSFP_H */
