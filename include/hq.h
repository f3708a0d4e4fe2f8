/*
 * hq.h -- C ABI of the GB300 (sm_103a) quantized-weight matvec library (libhq.so).
 *
 * The library computes the bandwidth-bound decode product y = W_deq . x over
 * block-quantized weights, for 1..8 activation vectors in one pass, so that
 * every weight byte is streamed from HBM once per call.
 *
 * Sources (page title, section):
 *   - "One Native Stack for Private, Continuously-Learning AI", section "The
 *     Unified Quant Core": one quant-agnostic decode matvec over the ggml
 *     block formats Q8_0 (symmetric, 34 B per 32 weights) and Q4_0
 *     (symmetric, 18 B per 32 weights); the same core evaluates every routed
 *     MoE expert.  Section "The Central Efficiency Thesis", Lemma "QLoRA over
 *     the unified core is exact": y_i = sum_j What_ij x_j, What the CPU
 *     dequantization of the stored bytes, accumulated in f32.
 *   - "Economical Serving and the hanzo.ai Platform", subsection "The Roofline
 *     that Sets the Price": decode time per token is W/B (weight bytes over
 *     bandwidth); subsection "One Quant-Agnostic Core": per-format block
 *     decoder + traits record, reused by decode and MoE.
 *   - "Blue -- porting zen-nano (Qwen3-0.6B) to deterministic on-chain
 *     inference", section "Quantization recipe (validated)": per-output-channel
 *     symmetric int8 weights and gemmlowp requant
 *     (SaturatingRoundingDoublingHighMul, then RoundingDivideByPOT) to int8.
 *   - "DeepSeek-V4 on Hanzo Engine", section "A Fused Attention Kernel for
 *     512-Wide Latent Heads": speculative-verify widths q in [1, 8], hence
 *     n_vec in [1, 8].
 *
 * Conventions shared by every entry point
 *   - Pointers named W, x, y, ids, mult, shift, acc, out, scale are DEVICE
 *     pointers owned by the caller (cudaMalloc / PyTorch).  The library never
 *     allocates, frees or retains them, and keeps no state between calls other
 *     than a thread-local error string and a device fault word (below).
 *   - Every call is asynchronous and stream-ordered on `stream` (a
 *     cudaStream_t; NULL is the legacy default stream).  Arguments are
 *     validated on the host before any launch; a non-OK status means nothing
 *     was launched (except HQ_ERR_LAUNCH, which reports the launch failure).
 *     A fault inside a kernel surfaces at the caller's next synchronization.
 *     The matvec calls begin to read W (and an adapter's A) as soon as the
 *     kernel before them in the stream lets its programmatic dependents start,
 *     which without a trigger of its own is at its end: a kernel that writes
 *     weights must not trigger them before its last write.  No kernel of this
 *     library does.  The many-token calls read nothing before what precedes
 *     the call in the stream is done.
 *   - Row-major layouts.  Quantized rows are packed blocks with no padding:
 *     row i of a Q8_0 matrix is bytes [i*cols/32*34, (i+1)*cols/32*34).
 *   - Block layouts (little-endian): Q8_0 = { uint16 fp16 d; int8 q[32] },
 *     w_j = d*q_j.  Q4_0 = { uint16 fp16 d; uint8 qs[16] }, element j (0..15)
 *     is the low nibble of qs[j] and element j+16 the high nibble,
 *     w = d*(n - 8).
 *   - Float paths accumulate in fp32 and are deterministic run to run (fixed
 *     reduction order, no float atomics).  They match the f64 definition
 *     within |y - y_ref| <= 1e-3 * sum_j |w_deq x_j| + 1e-5 per output.
 *     The int8 path is bit-exact.
 *   - Shapes: rows >= 1, cols >= 32, cols % 32 == 0 (int8: cols >= 4 and
 *     cols % 4 == 0), 1 <= n_vec <= 8.  W and x must be 16-byte aligned.
 *     When cols % 256 == 0 (every decode shape) the TMA-staged kernel runs;
 *     other legal shapes run a plain-load kernel that gives the same results
 *     to the same tolerance.  There is no CPU fallback.
 */
#ifndef HQ_H_
#define HQ_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *hq_stream_t;   /* identical to cudaStream_t */

typedef enum {
    HQ_OK = 0,
    HQ_ERR_NULL = -1,         /* a required pointer is NULL                        */
    HQ_ERR_SHAPE = -2,        /* rows/cols/n_experts/n_active out of range         */
    HQ_ERR_ALIGN = -3,        /* W or x not 16-byte aligned (y: 4-byte)            */
    HQ_ERR_NVEC = -4,         /* n_vec not in [1, 8]                               */
    HQ_ERR_LAUNCH = -5,       /* the CUDA launch failed (see hq_last_error)        */
    HQ_ERR_UNSUPPORTED = -6,  /* no sm_100-family GPU, or a value not representable */
    HQ_ERR_DEVICE = -7        /* a kernel reported a fault word (hq_device_fault)  */
} hq_status;

/* Format codes taken by hq_debug_plan. */
#define HQ_FMT_Q8_0 8
#define HQ_FMT_Q4_0 4
#define HQ_FMT_Q4_K 75      /* 'K' */
#define HQ_FMT_I8 1

/* Library version (major*10000 + minor*100 + patch). */
int hq_version(void);

/* Message for the last non-OK status returned on this host thread ("" if none). */
const char *hq_last_error(void);

/*
 * hq_matvec_q8_0 -- y[v][i] = sum_j w_deq[i][j] * x[v][j] for v < n_vec, i < rows.
 *   W  : Q8_0 blocks, rows x (cols/32) x 34 bytes, 16-byte aligned.
 *   x  : fp32 [n_vec][cols], 16-byte aligned.
 *   y  : fp32 [n_vec][rows], overwritten (not accumulated).
 * Accumulation is fp32; |y - y_exact| <= 1e-3 * sum_j |w_deq[i][j] * x[v][j]| + 1e-5
 * for finite x with |x| < 2^100 (beyond that a block's partial sum may
 * overflow).  Every quant is decoded to its signed value exactly before it
 * multiplies x, so the rounding is relative to the products |w x| themselves:
 * the bound holds at every n_vec for sparse or outlier-dominated blocks and
 * for x of any sign pattern or mean.
 * Source: "One Native Stack ...", section "The Unified Quant Core" (Q8_0,
 * 34 B/32) and the Lemma of section "The Central Efficiency Thesis".
 */
hq_status hq_matvec_q8_0(const void *W, const float *x, float *y,
                         int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);

/*
 * hq_matvec_q4_0 -- as hq_matvec_q8_0 for Q4_0 blocks (rows x cols/32 x 18 B):
 * w = d * (n - 8), nibble order as in the conventions above; the same
 * accuracy and the same |x| < 2^100 precondition.
 * Source: "One Native Stack ...", section "The Unified Quant Core" (Q4_0, 18 B/32).
 */
hq_status hq_matvec_q4_0(const void *W, const float *x, float *y,
                         int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);

/*
 * hq_matvec_q4_k -- as hq_matvec_q8_0 for Q4_K super-blocks: W is
 * rows x (cols/256) x 144 bytes, 16-byte aligned, cols % 256 == 0
 * (HQ_ERR_SHAPE otherwise).  A super-block is { fp16 d, fp16 dmin, uint8
 * scales[12], uint8 qs[128] }: sub-block j (32 weights, j = 0..7) has a
 * six-bit scale sc_j and min m_j -- for j < 4, sc_j = scales[j] & 63 and
 * m_j = scales[j+4] & 63; for j >= 4, sc_j = (scales[j+4] & 15) |
 * (scales[j-4] >> 6) << 4 and m_j = (scales[j+4] >> 4) | (scales[j] >> 6) << 4
 * -- and its quants are the low (even j) or high (odd j) nibbles of
 * qs[32*(j/2) .. +31]; w = d*sc_j*q - dmin*m_j.  Each weight is formed in fp32
 * (one rounding) before it multiplies x, so the accuracy statement and the
 * |x| < 2^100 precondition of hq_matvec_q8_0 hold unchanged.
 * Source: "One Native Stack ...", sections "The Unified Quant Core" (Q4_K is
 * one of the native formats) and "Ported Versus Novel" (formats taken
 * verbatim from ggml, whose Q4_K super-block this is); "Economical Serving
 * ...", subsection "One Quant-Agnostic Core, Not a Kernel-per-Quant Zoo"
 * (the Q4_K decode kernel).
 */
hq_status hq_matvec_q4_k(const void *W, const float *x, float *y,
                         int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);


/*
 * hq_matvec_q8_0_lora, hq_matvec_q4_0_lora -- the float matvec of the same
 * format plus a QLoRA adapter over the frozen quantized base:
 *   y[v][i] = sum_j w_deq[i][j] x[v][j] + scale * sum_k B[i][k] (sum_j A[k][j] x[v][j]).
 *   lora_A    : bf16 [rank][cols] (raw bf16 bits), 16-byte aligned.
 *   lora_B    : bf16 [rows][rank], 2-byte aligned.
 *   scale     : alpha / r, finite.   rank : 1..64.
 *   workspace : caller-owned device memory of at least rank * n_vec floats,
 *               4-byte aligned; it receives u = A x (fp32 [n_vec][rank]) and
 *               must not be in use by other work until the call's kernels end.
 * W, x, y, rows, cols, n_vec and the accuracy are as for hq_matvec_q8_0; the
 * adapter term adds 1e-3 * |scale| * sum_k |B[i][k]| * sum_j |A[k][j] x[v][j]|
 * to the tolerance.  Two kernels run: the down projection u = A x, then the
 * matvec, which streams W once and adds scale * B u as it stores y.
 * Source: "One Native Stack ...", section "The Central Efficiency Thesis",
 * Lemma "QLoRA over the unified core is exact and base-weight-identical".
 */
hq_status hq_matvec_q8_0_lora(const void *W, const float *x, const uint16_t *lora_A,
                              const uint16_t *lora_B, float scale, int rank, float *workspace,
                              float *y, int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);
hq_status hq_matvec_q4_0_lora(const void *W, const float *x, const uint16_t *lora_A,
                              const uint16_t *lora_B, float scale, int rank, float *workspace,
                              float *y, int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);

/*
 * hq_matvec_q8_0_lora_noalloc -- hq_matvec_q8_0_lora without a workspace, for
 * callers that cannot allocate device memory.  Examples are code inside an
 * engine that hands all device memory to its own pre-sized pool, and a hot
 * path that must not call cudaMalloc / cudaFree, which may synchronize the
 * device.  Such a caller can pass no workspace for u = A x.
 *   Scratch: u lives in one file-scope array of 2 KB in the library's static
 *   device memory (64 x 8 fp32: the largest rank times the largest n_vec).
 *   Every GPU that loads the library holds it until the process exits.  A call
 *   with rank > 64 (or n_vec > 8) is rejected with HQ_ERR_SHAPE before any
 *   launch.  The call itself allocates nothing: no cudaMalloc, no cudaFree, no
 *   allocating library routine.
 *   Set-up: the library's first call on a device (this entry point or any
 *   other) looks up the scratch's device address with that device current.
 *   Make that first call before any stream capture.
 *   Sharing: every call on a device uses the same array, and nothing in it
 *   needs to start at zero (each call writes all of u before reading it).
 *   Calls of this entry point that overlap on the GPU (on different streams of
 *   one device) race on the array.  Calls on one stream are ordered and safe.
 * Arguments, validation, accuracy and kernels are those of hq_matvec_q8_0_lora.
 * Source: the paper has no counterpart (an allocation-free form of this
 * library's own QLoRA call).
 */
hq_status hq_matvec_q8_0_lora_noalloc(const void *W, const float *x, const uint16_t *lora_A,
                                      const uint16_t *lora_B, float scale, int rank, float *y,
                                      int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);

/*
 * hq_matvec_i8_requant -- per-output-channel int8 GEMV with gemmlowp requant:
 *   acc = sum_j W[o][j] * x[v][j]  (int32; the caller keeps it in range:
 *         |W|, |x| <= 127 and cols < 133,000 always fit),
 *   y[v][o] = clamp(RDivByPOT(SRDHM(acc, mult[o]), shift[o]), -128, 127).
 *   W     : int8 [rows][cols], 16-byte aligned.   x : int8 [n_vec][cols], 16-byte aligned.
 *   mult  : int32 [rows] (any value).             shift : int32 [rows], each in [0, 31].
 *   y     : int8 [n_vec][rows].
 * SRDHM(a,b) is the high word of 2ab rounded to nearest (ties toward +inf),
 * saturating only at a = b = INT32_MIN; RDivByPOT(x,e) is x/2^e rounded to
 * nearest with ties away from zero.  Bit-exact.  A shift outside [0,31] is a
 * precondition violation (the kernel clamps it to that range).
 * Source: "Blue -- porting zen-nano ...", section "Quantization recipe
 * (validated)" and section "Gaps vs the current toy engine", item 3.
 */
hq_status hq_matvec_i8_requant(const int8_t *W, const int8_t *x,
                               const int32_t *mult, const int32_t *shift, int8_t *y,
                               int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);

/*
 * hq_moe_matvec_q8_0 -- expert-indexed, grouped Q8_0 matvec for MoE decode.
 *   W_bank     : n_experts Q8_0 matrices of rows x cols, back to back
 *                (expert e starts at byte e*rows*cols/32*34), 16-byte aligned.
 *   expert_ids : int32 [n_vec][n_active], each in [0, n_experts).
 *   x          : fp32 [n_vec][cols] when x_per_slot == 0 (all slots of token t
 *                share x[t], as for gate/up), or [n_vec][n_active][cols] when
 *                x_per_slot == 1 (one input per slot, as for down).
 *   y          : fp32 [n_vec][n_active][rows]; y[t][k] = W_bank[ids[t][k]] . x(t,k).
 * Accuracy and the |x| < 2^100 precondition as for hq_matvec_q8_0.
 * Slots that pick the same expert are grouped so that each chosen expert's
 * bytes are streamed once per call.  No router weighting is applied (the
 * _combine variant below applies it).  An id
 * outside [0, n_experts) is a precondition violation: its outputs are set to
 * NaN and the device fault word gets HQ_FAULT_EXPERT_ID; nothing traps.
 * Source: "One Native Stack ...", section "The Unified Quant Core" (the MoE
 * path dispatches each routed expert through the same core); "Economical
 * Serving ...", subsection "The Roofline that Sets the Price" (MoE reads
 * only its active parameters).
 */
hq_status hq_moe_matvec_q8_0(const void *W_bank, const int32_t *expert_ids,
                             const float *x, int x_per_slot, float *y,
                             int64_t n_experts, int n_active, int64_t rows, int64_t cols,
                             int n_vec, hq_stream_t stream);

/*
 * hq_moe_matvec_q8_0_swiglu -- the grouped MoE matvec of an expert bank whose
 * gate and up matrices are stored as one matrix with their rows interleaved
 * (row 2i = gate row i, row 2i+1 = up row i; rows = 2 * intermediate, even),
 * with the SwiGLU gate applied as the outputs are stored:
 *   h[t][k][i] = silu(g) * u,  g = row 2i . x(t,k),  u = row 2i+1 . x(t,k),
 *   silu(z) = z / (1 + e^-z).
 *   h : fp32 [n_vec][n_active][rows / 2], 4-byte aligned; it is the x of the
 *       down projection (x_per_slot = 1).
 * Other arguments, grouping and the invalid-id behaviour (NaN outputs, fault
 * word) as for hq_moe_matvec_q8_0.  Accuracy: g and u are each within the
 * matvec tolerance e = 1e-3 * sum_j |w_deq * x| + 1e-5 of their exact values;
 * h is then within 1.1 * e_g * (|u| + e_u) + |silu(g)| * e_u, plus fp32
 * rounding, of silu(g) * u.
 * Source: "Blue -- porting zen-nano ...", section "Architecture" (each
 * layer's feed-forward is SwiGLU(gate, up, down)); the silu gate and the
 * row interleave are this library's readings.
 */
hq_status hq_moe_matvec_q8_0_swiglu(const void *W_bank, const int32_t *expert_ids, const float *x,
                                    int x_per_slot, float *h, int64_t n_experts, int n_active,
                                    int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);

/*
 * hq_moe_matvec_q8_0_combine -- the grouped MoE matvec with the router-weighted
 * sum over each token's slots applied in the same launch:
 *   y[t][i] = sum_k router_w[t][k] * (W_bank[ids[t][k]] . x(t,k))[i].
 *   router_w : fp32 [n_vec][n_active], the router's weights for the chosen
 *              experts (the router itself is the caller's), 4-byte aligned.
 *   y        : fp32 [n_vec][rows], 4-byte aligned.
 * A cluster of up to 8 CTAs (as many as one wave of the grid allows) owns
 * each 32-row tile and splits the tile's expert groups among its CTAs; each
 * CTA keeps its weighted per-token sums in shared memory and the cluster's
 * leader adds them over distributed shared memory.  No atomics and no workspace; the summation order is fixed, so y
 * is the same bits on every run.  A token with an invalid expert id gets
 * NaN rows (and the fault word HQ_FAULT_EXPERT_ID).  Accuracy: |y - y_ref|
 * <= 1e-3 * sum_k |router_w[t][k]| * sum_j |w_deq * x| + 1e-5.  Other
 * arguments as for hq_moe_matvec_q8_0.
 * Source: "Economical Serving ...", paragraph "MoE is the cheapest-per-quality
 * tier" (a sparsely gated mixture: the output is the gate-weighted sum of the
 * chosen experts' outputs).
 */
hq_status hq_moe_matvec_q8_0_combine(const void *W_bank, const int32_t *expert_ids, const float *x,
                                     int x_per_slot, const float *router_w, float *y, int64_t n_experts,
                                     int n_active, int64_t rows, int64_t cols, int n_vec, hq_stream_t stream);

/*
 * hq_moe_matvec_q8_0_ex -- the three MoE calls above in one entry point, with
 * flags.
 *   epilogue : HQ_MOE_EPI_NONE (as hq_moe_matvec_q8_0; router_w unused),
 *              HQ_MOE_EPI_SWIGLU (as hq_moe_matvec_q8_0_swiglu) or
 *              HQ_MOE_EPI_COMBINE (as hq_moe_matvec_q8_0_combine).
 *   flags    : 0, or HQ_MOE_IDS_READY: the caller guarantees that expert_ids
 *              were written by work that completed before the kernel that
 *              precedes this call in the stream -- e.g. the down projection of
 *              an MoE feed-forward, whose ids the router wrote before the
 *              gate|up launch.  The kernel then reads the ids and starts its
 *              weight copies while that kernel is still running, waiting for
 *              it only before it reads x or writes y.  Ids written by the
 *              immediately preceding kernel break the guarantee (the kernel
 *              may read stale ids).
 * All other arguments, results and errors as for the calls above; unknown
 * epilogues or flags give HQ_ERR_UNSUPPORTED.
 * Source: as hq_moe_matvec_q8_0 ("One Native Stack ...", section "The
 * Unified Quant Core": every routed expert through the same core; "Economical
 * Serving ...", subsection "The Roofline that Sets the Price").
 */
#define HQ_MOE_EPI_NONE 0
#define HQ_MOE_EPI_SWIGLU 1
#define HQ_MOE_EPI_COMBINE 2
#define HQ_MOE_IDS_READY 1
hq_status hq_moe_matvec_q8_0_ex(const void *W_bank, const int32_t *expert_ids, const float *x, int x_per_slot,
                                const float *router_w, float *y, int64_t n_experts, int n_active, int64_t rows,
                                int64_t cols, int n_vec, int epilogue, int flags, hq_stream_t stream);

/*
 * Quantizers (the one-off data-preparation step, on the GPU).
 * hq_quantize_q8_0: W fp32 [rows][cols] (device) -> out Q8_0 blocks (device):
 *   d = max|w|/127 in fp32, stored fp16 (round to nearest even);
 *   q = round(w/d) (fp32 division, half away from zero), clamped to [-127,127];
 *   an all-zero block stores d = 0 and q = 0.
 * hq_quantize_q4_0: d = m/-8 with m the block's largest-|w| element (first
 *   on ties, sign kept), stored fp16; n = min(15, floor(w/d + 8.5)) (fp32);
 *   an all-zero block stores d = -0 and n = 8.
 * hq_quantize_i8_rows: scale[o] = max|W[o,:]|/127 (fp32),
 *   Wq = round(W/scale) clamped to [-127,127]; with rows = 1 this is the
 *   static per-tensor activation quantizer.
 * Requires rows >= 1 and cols % 32 == 0 (i8: cols >= 1).  Alignment: Q8_0 and
 * Q4_0 take W 16-byte aligned and out 2-byte aligned; the int8 quantizer takes
 * W and scale 4-byte aligned.  HQ_ERR_ALIGN otherwise.
 * Source: "One Native Stack ...", section "The Unified Quant Core" (formats
 * taken verbatim from ggml); "Blue -- porting zen-nano ...", section
 * "Quantization recipe (validated)".
 */
hq_status hq_quantize_q8_0(const float *W, void *out, int64_t rows, int64_t cols,
                           hq_stream_t stream);
hq_status hq_quantize_q4_0(const float *W, void *out, int64_t rows, int64_t cols,
                           hq_stream_t stream);
hq_status hq_quantize_i8_rows(const float *W, int8_t *Wq, float *scale,
                              int64_t rows, int64_t cols, hq_stream_t stream);
/*
 * hq_quantize_q4_k -- fp32 W [rows][cols] (4-byte aligned) to Q4_K
 * super-blocks in out (rows x cols/256 x 144 B, 16-byte aligned), cols % 256
 * == 0.  The pages give no encoder; this one is a plain min/max reading, per
 * sub-block of 32: mn = min(0, min w), scale = (max w - mn)/15, min = -mn;
 * d = (largest scale)/63 and dmin = (largest min)/63 stored fp16 (RNE);
 * sc = round(scale * 63/largest scale), m likewise (at most 63); then with
 * a = d*sc and b = dmin*m from the stored values, q = round((w + b)/a)
 * clamped to [0, 15] (0 when a == 0).  All in fp32, half away from zero.
 * Source: "One Native Stack ...", section "Ported Versus Novel" (ggml's Q4_K).
 */
hq_status hq_quantize_q4_k(const float *W, void *out, int64_t rows, int64_t cols, hq_stream_t stream);

/*
 * The batched step: the products of any number of tokens with the same stored
 * weights, the probabilities of their logits, and the verification of drafted
 * tokens.  The matvec calls above stay the right ones for one request's 1..8
 * fp32 vectors; these serve prompts, and the verify step of many requests.
 *
 * Element types of x, y and logits in these calls (`dtype`): */
#define HQ_DT_F32 0
#define HQ_DT_F16 1
#define HQ_DT_BF16 2
/*
 * hq_weight_exponents -- set-up of the many-token products, once per weight:
 * w_exp[m] = e with every finite |weight| of matrix m below 2^(e + 14), read off the
 * block scales d (e + 14 = the exponent of 128 max|d| for Q8_0, 8 max|d| for
 * Q4_0, with max|d| = f 2^k, 0.5 <= f < 1, having exponent k; -14 when no d is finite and non-zero).  The products
 * multiply in 16-bit floats; weights times 2^-e use their range fully
 * whatever the scale of the matrix.
 *   fmt : HQ_FMT_Q8_0 or HQ_FMT_Q4_0 (HQ_ERR_UNSUPPORTED otherwise).
 *   W : n_mats matrices of rows x cols back to back, cols % 32 == 0, 16-byte aligned.
 *   w_exp : int32 [n_mats] (device).  n_mats in [1, 65535].
 * Source: none on the pages (a property of this implementation).
 */
hq_status hq_weight_exponents(int fmt, const void *W, int32_t *w_exp, int64_t n_mats, int64_t rows, int64_t cols,
                              hq_stream_t stream);

/*
 * hq_moe_matmul_q8_0 -- the expert-indexed Q8_0 product of any number of
 * tokens: y[t][k] = W_bank[ids[t][k]] . x(t,k), as hq_moe_matvec_q8_0_ex
 * computes for up to 8.  Slots are grouped by expert on the device (ragged
 * groups, no host synchronisation).
 *   W_bank, expert_ids, x_per_slot, router_w, epilogue : as for
 *       hq_moe_matvec_q8_0_ex; expert_ids is int32 [n_tokens][n_active].
 *   w_exp : int32 [n_experts], from hq_weight_exponents.
 *   x, y  : `dtype`, the layouts of hq_moe_matvec_q8_0_ex with n_tokens for
 *           n_vec; x 16-byte aligned, y aligned to its element.
 *   n_tokens : >= 0 (0 returns HQ_OK and launches nothing);
 *       n_tokens * n_active <= 2^27 (and fewer than 2^31 tiles of 16 of them and 128 rows); n_experts <= 8192.  cols % 256 == 0; HQ_MOE_EPI_SWIGLU
 *       needs an even number of rows; y may not overlap x.
 *   workspace : device memory of hq_moe_matmul_workspace() bytes, 256-byte
 *       aligned, not in use by other work until the call's kernels end.
 *       hq_moe_matmul_workspace is a HOST function; a negative result is the
 *       hq_status of arguments that the call itself would refuse.
 * Accuracy: f16 and bf16: each weight is rounded to 11 bits or within 2^-22 of its matrix's
 * largest, whichever is coarser; x is exact (bf16 elements below 2^-29
 * of their row's largest are rounded to multiples of 2^-39 of it), sums are fp32, y is rounded
 * once.  f32: both factors are split in two 11-bit terms and the
 * product of the two small terms is left out: relative error of a
 * product below 2^-20 (weights below 2^-17 of their matrix's largest: 2^-36 of that; elements of x below 2^-17 of
 * their row's largest: 2^-38 of that).
 * The fp32 sums of f32 leave the tensor core every 256 columns.
 * An infinity in x gives infinities of its weights' signs, and NaN where the weight (f16, bf16: rounded) is zero; it
 * and NaN stay in their own token's row.
 * HQ_MOE_EPI_SWIGLU, of the gate z = the product's result: z / (1 + e^-z) to a relative 2^-20, 0 below z = -88.7 (f32), or
 * to 2^-21 (1 + |z| / 4), 0 below z = -87 (f16, bf16).
 * Deterministic: the bits of a token's y do not depend on the other tokens, except through the
 * split of the columns over CTAs that the launch's sizes choose.
 * An id outside [0, n_experts): as for hq_moe_matvec_q8_0 (NaN, HQ_FAULT_EXPERT_ID).
 * Source: as hq_moe_matvec_q8_0; the pages' prefill core is the same
 * unified core ("One Native Stack ...", section "The Unified Quant Core").
 */
int64_t hq_moe_matmul_workspace(int64_t n_experts, int n_active, int64_t rows, int64_t cols, int64_t n_tokens,
                                int x_per_slot, int dtype, int epilogue);
hq_status hq_moe_matmul_q8_0(const void *W_bank, const int32_t *w_exp, const int32_t *expert_ids, const void *x,
                             int x_per_slot, const float *router_w, void *y, int64_t n_experts, int n_active,
                             int64_t rows, int64_t cols, int64_t n_tokens, int dtype, int epilogue,
                             void *workspace, int64_t workspace_bytes, hq_stream_t stream);

/*
 * hq_matmul_q8_0_adapters, hq_matmul_q4_0_adapters -- the shared projection
 * of many requests' tokens, each with its request's adapter:
 *   y[t][i] = sum_j w_deq[i][j] x[t][j]
 *             + scales[a] sum_k B[a][i][k] (sum_j A[a][k][j] x[t][j]),  a = adapter_ids[t].
 *   w_exp : int32 [1], from hq_weight_exponents.
 *   x : `dtype` [n_tokens][cols], 16-byte aligned.   y : `dtype` [n_tokens][rows].
 *   adapter_ids : int32 [n_tokens], each in [-1, n_adapters); -1: no adapter.
 *       Tokens of one request next to each other share the adapter's bytes.
 *   lora_A : bf16 [n_adapters][rank][cols], 16-byte aligned.
 *   lora_B : bf16 [n_adapters][rows][rank], 2-byte aligned.
 *   scales : fp32 [n_adapters], finite.   rank : 1..64 (adapters of smaller rank are padded with zeros).
 *   n_adapters : >= 0; with 0 the adapter arguments are not read (they may be NULL) and the
 *       call is the plain many-token product.
 *   n_tokens : 0..2^27 (0 launches nothing; fewer than 2^31 tiles of 16 of them and 128 rows).  cols % 256 == 0.
 *   workspace : hq_matmul_adapters_workspace() bytes, 256-byte aligned (a HOST
 *       function; negative: the hq_status of refused arguments).
 * Each token's row depends on its own adapter only: infinities and NaN of another's stay with that one's tokens.
 * An infinity or NaN in an adapter's A gives its tokens outputs that are infinite or NaN.
 * Accuracy of the base term as for hq_moe_matmul_q8_0; the adapter term takes x, A and B
 * exactly and sums in fp32, with A x in between rounded to 16 bits (f32: 24).  An id outside [-1, n_adapters) gives a NaN row of y and
 * HQ_FAULT_ADAPTER_ID.
 * Source: as hq_matvec_q8_0_lora (the Lemma "QLoRA over the unified core is
 * exact"), for a batch in which every request brings its own adapter.
 */
int64_t hq_matmul_adapters_workspace(int rank, int64_t rows, int64_t cols, int64_t n_tokens, int dtype);
hq_status hq_matmul_q8_0_adapters(const void *W, const int32_t *w_exp, const void *x, const int32_t *adapter_ids,
                                  const uint16_t *lora_A, const uint16_t *lora_B, const float *scales,
                                  int64_t n_adapters, int rank, void *y, int64_t rows, int64_t cols,
                                  int64_t n_tokens, int dtype, void *workspace, int64_t workspace_bytes,
                                  hq_stream_t stream);
hq_status hq_matmul_q4_0_adapters(const void *W, const int32_t *w_exp, const void *x, const int32_t *adapter_ids,
                                  const uint16_t *lora_A, const uint16_t *lora_B, const float *scales,
                                  int64_t n_adapters, int rank, void *y, int64_t rows, int64_t cols,
                                  int64_t n_tokens, int dtype, void *workspace, int64_t workspace_bytes,
                                  hq_stream_t stream);

/*
 * hq_softmax_rows -- probabilities of logits, one temperature per row:
 *   p[r][j] = exp((l[r][j] - max_j l[r][j]) / t_r) / sum_j exp(...),  t_r > 0;
 *   t_r <= 0 or NaN : greedy, p[r] is 1 at the first maximum and 0 elsewhere.
 *   logits : `dtype` [n_rows][vocab], aligned to its element.
 *   temperature : fp32 [n_rows], or NULL for 1.   p : fp32 [n_rows][vocab].
 *   n_rows : 0..2^28-1 (0 launches nothing).  vocab : 1..2^22.
 * Logits of -inf give 0, at an infinite temperature too (all others are then equal).  A row of nothing but -inf gives zeros (greedy too).  A row with
 * a NaN or +inf gives NaNs (greedy: the first maximum of what is not NaN; a row of nothing
 * but NaN and -inf gives zeros).  p may be the logits' own
 * memory when dtype is HQ_DT_F32.
 * Source: "DeepSeek-V4 on Hanzo Engine" (the verify rows whose
 * probabilities a speculative step compares).
 */
hq_status hq_softmax_rows(const void *logits, const float *temperature, float *p, int64_t n_rows, int64_t vocab,
                          int dtype, hq_stream_t stream);

/*
 * hq_verify_drafts -- speculative verification of n_req requests at once.
 * Request r drafted tokens drafts[off[r] .. off[r+1]); n_r = off[r+1] - off[r] >= 0.
 *   p  : fp32 [n_drafts + n_req][vocab], the target's probabilities: row off[r] + r + i
 *        is the target's distribution of request r's draft i, i = n_r the one after its last.
 *   q  : fp32 [n_drafts][vocab], the drafting probabilities, or NULL: drafts were certain (q = 1 at the draft).
 *   u_accept : fp32 [n_drafts], u_sample : fp32 [n_req], uniform numbers in [0, 1), the caller's.
 * Draft i is accepted while u_i * q_i(d_i) < p_i(d_i) (one fp32 product) and all before it were; a_r counts
 * them.  One more token is then sampled, from s = max(p - q, 0) (fp32) of the first refused draft, or from
 * s = p of the row after the last draft: s is taken as the integers S_j = floor(2^40 s_j), and the token is the
 * lowest j with S_0 + ... + S_j > floor(U sum S / 2^24), U = floor(2^24 u_sample[r]).  Integer sums have no
 * order, so the token is exact.  If the residual's integers are all zero, s = p is used; if those
 * are all zero too, the token is -1.
 *   n_accepted : int32 [n_req] = a_r.
 *   tokens     : int32 [n_drafts + n_req]; request r's at off[r] + r: the a_r accepted
 *                drafts, the sampled token, then -1 for each refused draft after the first.
 *   draft_offsets : int32 [n_req + 1] (device), from 0 to n_drafts.
 *   n_req : 0..2^24 (0 launches nothing); n_drafts >= 0 (0: drafts, q and u_accept are not read);
 *   n_drafts + n_req <= 2^30; vocab 1..2^22.
 * p and q are probabilities as hq_softmax_rows gives them.  Of other values: a draft whose p or q is NaN is refused, and s is
 * clamped to [0, 1], a NaN in it counting as 0.  A draft outside
 * [0, vocab) is refused and sets HQ_FAULT_DRAFT if all before it were accepted (those behind a refused one are not looked at).
 * Offsets that do not rise from 0 to n_drafts set it too (that request's outputs are then left unwritten).
 * Source: "DeepSeek-V4 on Hanzo Engine", the speculative-verify widths q in [1, 8].
 */
hq_status hq_verify_drafts(const float *p, const float *q, const int32_t *drafts, const int32_t *draft_offsets,
                           const float *u_accept, const float *u_sample, int32_t *n_accepted, int32_t *tokens,
                           int64_t n_req, int64_t n_drafts, int64_t vocab, hq_stream_t stream);

/*
 * The key/value cache: rows of the batched step's positions, quantized as they
 * are written, and the attention that reads them.
 *
 * A pool of n_pages pages holds page_size positions each, for all key/value
 * heads, as blocks of Q8_0 or Q4_0 (fmt HQ_FMT_Q8_0, HQ_FMT_Q4_0; 32 values along
 * the head, one fp16 scale).  It is device memory of
 * n_pages * hq_cache_page_bytes() bytes, 16-byte aligned, that need not be set to
 * anything.  Its inner layout is the library's:
 *   page  : [n_kv_heads][page_size / 16] cells of 16 positions
 *   cell  : quants of the keys, quants of the values, scales of the keys
 *           [16][head_dim / 32], scales of the values [8][head_dim / 32][2]
 *   quants: unsigned (q + 128, or the nibble n).  A key is [units][4][unit bytes]:
 *           lane c of 4 holds elements 8c .. 8c+7 of every block of 32 (Q4_0: a word
 *           a block, nibble i/2 + 4 (i mod 2) for element i).  The values of two
 *           neighbouring positions are [units][8][unit bytes]: lane g of 8 holds elements
 *           g, 8+g, 16+g and 24+g of every block, the halves of a word the two
 *           positions'.  A lane's bytes (head_dim / 8 for Q4_0, head_dim / 4 for Q8_0) are cut
 *           into units of 16 (8 where it has no more).
 *
 * Arguments that the calls share
 *   page_size    : 16, 32, 64, 128, 256, 512 or 1024.   n_pages : 1..2^31-1.
 *   page_table   : int32 [n_req][table_width] (device), table_width >= 1,
 *                  table_width * page_size <= 2^30: position p of request r is
 *                  in page page_table[r][p / page_size].  Entries behind a request's length are not read.
 *   offsets      : int32 [n_req + 1] (device): request r brings the tokens
 *                  offsets[r] .. offsets[r+1]-1 (none where they are equal).
 *   lengths      : int32 [n_req] (device), the positions of request r, its
 *                  tokens included: its token i of n is at position lengths[r] - n + i.
 *                  0 <= lengths[r] <= table_width * page_size.  A token at a negative position
 *                  (a length below n) has no place in the cache: it is not written, reads as zeros, and sees nothing
 *                  where attention is causal (where it is not, what every token of its request sees).
 *   n_req        : 0..2^20 (0 launches nothing).
 *   n_tokens     : 0..2^27 (0 launches nothing), the rows of the token tensors;
 *                  offsets[n_req] <= n_tokens.  Rows that are no request's (behind the last one's) stay as they are.
 *   n_kv_heads   : 1..1024.   head_dim : 64, 128 or 256.
 *   *_stride     : elements from one token to the next, a multiple of 16 bytes, at least
 *                  heads * head_dim; the heads of a token lie together.  So the
 *                  parts of one projection's rows can be passed as they are.  Token tensors are 16-byte aligned.
 *   dtype        : of the token tensors, HQ_DT_*.
 * Offsets and lengths outside these ranges set HQ_FAULT_CACHE, and that request is
 * left out (nothing of it is written); the others are served.  (Where offsets fall, requests in range may overlap:
 * a token's row is then either's, or parts of both.)  So does a page number outside [0, n_pages) that a call looks
 * up: nothing is written there, what is read there is NaN.
 */
/* HOST function: bytes of a page; negative: the hq_status of refused arguments. */
int64_t hq_cache_page_bytes(int fmt, int n_kv_heads, int head_dim, int page_size);

/*
 * hq_cache_write -- the tokens' key and value rows into the cache.
 *   k, v : `dtype` [n_tokens][n_kv_heads][head_dim].
 * Blocks are quantized as hq_quantize_q8_0 and hq_quantize_q4_0 do (fp32, correctly rounded
 * division), with two additions: the scale is at most the largest fp16 in
 * size, and a block with an infinity or a NaN is stored as a scale of NaN, so that all 32 read as NaN.
 * Two tokens for one place of the pool (shared pages) are the caller's to avoid.
 * Source: "One Native Stack ...", section "The Unified Quant Core" (the block
 * formats); "DeepSeek-V4 on Hanzo Engine" (the cache that decoding reads).
 */
hq_status hq_cache_write(int fmt, const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *pool,
                         int64_t n_pages, int page_size, const int32_t *page_table, int64_t table_width,
                         const int32_t *offsets, const int32_t *lengths, int64_t n_req, int64_t n_tokens,
                         int n_kv_heads, int head_dim, int dtype, hq_stream_t stream);

/*
 * hq_cache_read -- the values of the tokens' positions: d q or d (n - 8), rounded
 * once to `dtype`.  To take a whole cache out, offsets are the sums of the lengths.
 *   k, v : `dtype` [n_tokens][n_kv_heads][head_dim], written.
 */
hq_status hq_cache_read(int fmt, void *k, int64_t k_stride, void *v, int64_t v_stride, const void *pool,
                        int64_t n_pages, int page_size, const int32_t *page_table, int64_t table_width,
                        const int32_t *offsets, const int32_t *lengths, int64_t n_req, int64_t n_tokens,
                        int n_kv_heads, int head_dim, int dtype, hq_stream_t stream);

/*
 * hq_cache_attention -- attention of every request's tokens over its cached positions:
 *   out[t][h] = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale * (q[t][h] . k_p)),
 * k_p and v_p the stored values of key/value head h / (n_heads / n_kv_heads) at position p.
 *   q, out  : `dtype` [n_tokens][n_heads][head_dim]; out may be q itself (same stride), not overlap it otherwise.
 *   n_heads : a multiple of n_kv_heads, at most 4096.
 *   scale   : at most 2^100 in size.  Scores are fp32: they have to fit it, and a row of q whose largest element times
 *       scale passes 2^116 may come out as NaN.
 *   causal  : 1: a token sees the positions up to its own; 0: all of its request's.
 *   window  : w > 0: of those, the last w up to its own (needs causal 1; any size: past every position it is no window); 0: no window.
 *   workspace : hq_cache_attention_workspace() bytes, 256-byte aligned, not in
 *       use by other work until the call's kernels end (a HOST function;
 *       negative: the hq_status of refused arguments).  It is enough for batches of fewer tokens or requests too, and
 *       does not grow with them without end: at most 39 MiB.
 * A token that sees no position gets zeros.  Positions that a token does not see do
 * not touch it, whatever they hold.  One whose key has a NaN or infinite scale makes the rows that
 * see it NaN; a value block's makes that block's 32 elements NaN.
 * Accuracy: scores, maxima, sums and outputs are fp32.  f32 tokens: quants are exact, q and the weights
 * times the values' scales are taken in two 11-bit terms.  bf16 up to 16 rows and f16 up to 32 a key/value head of the mean
 * request (n_tokens / n_req, rounded up, times n_heads / n_kv_heads): the weights times their value block's scale are rounded to 11 bits; scores are off by up to 2^-22 of the position's
 * largest key element times the sum of |q|.  f16 and bf16, more rows: the weights are rounded to 11 bits; the
 * stored keys and values to 11 bits with bf16 tokens, with f16 ones to 14 (Q8_0) or not at all (Q4_0); or to 2^-17 (Q4_0) or 2^-20 (Q8_0) of the
 * largest that 32 neighbouring positions can hold (8 or 127 times their largest scale) where that is coarser.  q is exact,
 * but for elements below 2^-24 of their row's largest.
 * Deterministic: the same call gives the same bits.  Between batches a token's bits may differ, within the accuracy above: the rest of the
 * batch decides the split of the positions over CTAs, and n_tokens / n_req (rows behind the last request and requests without tokens
 * count) decides which of the two kernels runs, and with it the rounding of f16 and bf16 tokens.
 * Source: "DeepSeek-V4 on Hanzo Engine", section "A Fused Attention Kernel
 * for 512-Wide Latent Heads" (attention over the decode cache, one to eight
 * verified rows a request; its heads of 512 are wider than those here).
 */
int64_t hq_cache_attention_workspace(int fmt, int page_size, int64_t table_width, int64_t n_req, int64_t n_tokens,
                                     int n_heads, int n_kv_heads, int head_dim, int dtype);
hq_status hq_cache_attention(int fmt, const void *q, int64_t q_stride, const void *pool, int64_t n_pages, int page_size,
                             const int32_t *page_table, int64_t table_width, const int32_t *offsets,
                             const int32_t *lengths, int64_t n_req, int64_t n_tokens, int n_heads, int n_kv_heads,
                             int head_dim, float scale, int causal, int64_t window, void *out, int64_t out_stride,
                             int dtype, void *workspace, int64_t workspace_bytes, hq_stream_t stream);

/*
 * hq_requant_params -- HOST function: real multipliers M[i] in (0, 1) to
 * (mult, shift) with M ~= mult * 2^-31 * 2^-shift: M = f * 2^-shift with
 * f in [0.5, 1), mult = round(f * 2^31) (half away from zero; 2^31 becomes
 * 2^30 with shift - 1).  M, mult, shift are HOST arrays of n elements.
 * Returns HQ_ERR_UNSUPPORTED if some M is outside (0,1) or needs shift > 31.
 * Source: "Blue -- porting zen-nano ...", section "Quantization recipe
 * (validated)" (the requant multiplier s_a*s_w[o]/s_out as an integer pair).
 */
hq_status hq_requant_params(const double *M, int64_t n, int32_t *mult, int32_t *shift);

/*
 * hq_requant_i32_debug -- applies the device requant epilogue of
 * hq_matvec_i8_requant to arbitrary int32 accumulators, so that values the
 * GEMV cannot reach (INT32_MIN, INT32_MAX) are tested bit-exactly:
 * y[i] = requant(acc[i], mult[i % rows], shift[i % rows]).  Device pointers;
 * acc, y have n elements, mult, shift have rows elements.
 * Source: as hq_matvec_i8_requant.
 */
hq_status hq_requant_i32_debug(const int32_t *acc, const int32_t *mult, const int32_t *shift,
                               int8_t *y, int64_t n, int64_t rows, hq_stream_t stream);

/*
 * Device fault word.  Kernels never trap: a bounded wait that gives up (a
 * TMA transfer that never completes) or an out-of-range id sets a bit
 * in a per-device word, whatever it holds already, and the kernel finishes
 * without the missing data (the many-token products run on over whatever their
 * buffers hold, at the call's own addresses: after a time-out their
 * outputs are wrong).  hq_device_fault() synchronizes the current device, returns the word
 * in *fault (0 = none) and clears it; it returns HQ_ERR_DEVICE if the word
 * was non-zero.  Bits 0..7 are the HQ_FAULT_* flags; when the first fault of
 * the word was a timeout, bits 9..31 hold the index of the CTA that gave up
 * and bit 8 is set if the waiter was a consumer warp (clear: the producer).
 */
#define HQ_FAULT_WAIT_TIMEOUT 1u   /* an mbarrier wait exceeded its time limit */
#define HQ_FAULT_EXPERT_ID    2u   /* an expert id outside [0, n_experts)      */
#define HQ_FAULT_ADAPTER_ID   4u   /* an adapter id outside [-1, n_adapters)   */
#define HQ_FAULT_DRAFT        8u   /* draft offsets that do not rise from 0 to n_drafts, or a draft outside [0, vocab) */
#define HQ_FAULT_CACHE       16u   /* a cache's offsets, lengths or page numbers out of range */
hq_status hq_device_fault(uint32_t *fault);

/*
 * hq_selftest_wait_timeout -- test-only exercise of the failure path: one CTA
 * of one warp waits on an mbarrier that nothing arrives on, with the matvec
 * kernels' bounded wait but a limit of `cycles` SM clock cycles
 * (1 <= cycles <= 4e9).  The wait gives up, sets HQ_FAULT_WAIT_TIMEOUT in the
 * fault word with CTA 0 and the consumer bit recorded, and the kernel returns:
 * nothing faults, traps or hangs, and the context stays usable.  Read the
 * result with hq_device_fault().
 * Source: none on the pages (a property of this implementation's waits).
 */
hq_status hq_selftest_wait_timeout(int64_t cycles, hq_stream_t stream);

/*
 * hq_selftest_wait -- test-only, the same for each kind of bounded wait, with a
 * fault word that is not empty.
 *   wait  : HQ_WAIT_MATVEC (as hq_selftest_wait_timeout), HQ_WAIT_CLUSTER (on
 *           arrivals of another CTA of a cluster), HQ_WAIT_MATMUL and
 *           HQ_WAIT_MATMUL_GO (the many-token products': whose result is
 *           tested, and whose is not; the latter counts sleeps of about
 *           65536 cycles).
 *   fault : HQ_FAULT_* flags of data faults that are in the word before; the
 *           time-out's flag has to join them.
 * Source: none on the pages (a property of this implementation's waits).
 */
#define HQ_WAIT_MATVEC 0
#define HQ_WAIT_CLUSTER 1
#define HQ_WAIT_MATMUL 2
#define HQ_WAIT_MATMUL_GO 3
hq_status hq_selftest_wait(int wait, uint32_t fault, int64_t cycles, hq_stream_t stream);

/*
 * hq_launch_count -- the number of kernels the library has launched (or
 * recorded into a stream capture) in this process, on every device: a
 * monotone host-side counter for callers that account for launches.
 * Source: none on the pages (introspection of this implementation).
 */
uint64_t hq_launch_count(void);

/*
 * hq_debug_plan -- test-only: the launch geometry the library would choose for
 * a dense matvec of `rows` x `cols` at `n_vec` vectors, on a device with
 * `num_sms` SMs and `smem_optin` bytes of opt-in shared memory per CTA, for a
 * kernel of `regs` registers per thread.  Pure host arithmetic: no device is
 * touched, so it also runs on a machine without a GPU.
 *   fmt : 8 (Q8_0), 4 (Q4_0), 75 (Q4_K) or 1 (int8).  cols : a multiple of 256 (int8:
 *         128), the shapes the TMA-staged kernel serves.
 *   out : int64 [out_len >= HQ_PLAN_FIELDS], caller-owned host memory,
 *         filled with { policy (0 one owner per stage, 1 Q8_0 short rows,
 *         4 column-split stages; 2 and 3 are not used),
 *         consumer warps per CTA,
 *         rows per tile, grid (CTAs), K split (CTAs per cluster), ring stages,
 *         dynamic shared memory bytes, CTAs per SM of the launch bound,
 *         CTA slots (SMs x CTAs per SM the plan assumed), row tiles }.
 * Errors: HQ_ERR_NULL, HQ_ERR_SHAPE, HQ_ERR_NVEC, HQ_ERR_UNSUPPORTED (fmt).
 * Source: none on the pages (introspection of this implementation).
 */
#define HQ_PLAN_FIELDS 10
hq_status hq_debug_plan(int fmt, int n_vec, int64_t rows, int64_t cols, int num_sms, int smem_optin, int regs,
                        int64_t *out, int out_len);

#ifdef __cplusplus
}
#endif

#endif /* HQ_H_ */
