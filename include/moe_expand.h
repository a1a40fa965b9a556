/*
 * moe_expand.h -- C ABI of libmoe_expand.so: one expert-parallel rank's MoE
 * expert computation on the expanded dispatch layout, for AMD Instinct
 * MI355X (gfx950).
 *
 * The path, in call order (all on one HIP stream, no host synchronisation,
 * no host read of device data):
 *
 *   moe_expand_layout     received fp8 tokens + top-k ids/weights
 *                          -> per-(token, expert) rows grouped by expert,
 *                             each expert block padded to `align` rows,
 *                             row->expert labels, slot->row map, psum
 *   moe_grouped_gemm_fp8  gate_up projection (w13), bf16 out
 *   moe_act_quant         SiLU(gate)*up, per-1x128 fp8 quantisation, and
 *                          (fp32 scales) the top-k weight folded into the
 *                          down projection's input scale
 *   moe_grouped_gemm_fp8  down projection (w2), bf16 out
 *   moe_gather            each token's expert rows summed back into one
 *                          bf16 row (weighted here under UE8M0 scales)
 *
 * The standard (non-EP) path [P3 pre_permute_standard_to_deep_gemm,
 * post_permute_deep_gemm_to_standard] uses the same calls, entering with
 * moe_expand_layout_bf16 (bf16 token rows, quantised per 1x128 group while
 * they are scattered) and leaving through moe_gather with the top-k weights
 * and the routed scaling factor.
 *
 * Around the experts of a layer (before either standard path):
 *   moe_layer_norm        the norm of the residual stream, the branch before it added
 *   moe_grouped_gemm_bf16 the gate's logits, as one group
 *   moe_router            each token's experts and weights, as the layout takes them
 * and back, with the gradients that the training calls leave: moe_router_backward,
 * the grouped gradients of the gate, moe_layer_norm_backward.
 * moe_grouped_gemm_w4 takes the place of moe_grouped_gemm_bf16 for experts' weights of
 * 4 bits (int4 or MXFP4).
 *
 * The decode path's masked slab [P1 "Why decode stays on V1 low_latency";
 * P3 pre_permute_deepep_v2_to_deep_gemm / post_permute_deep_gemm_to_
 * deepep_v2, masked branches; _run_masked_gemm] runs after moe_expand_layout:
 *   moe_expand_to_masked_slab    expanded rows -> fixed-height slab
 *                                [num_experts, max_m, hidden], masked_m
 *   moe_grouped_gemm_fp8_masked  gate_up on each expert's masked_m rows
 *   moe_act_quant_masked         SiLU(gate)*up + per-1x128 quantisation
 *   moe_grouped_gemm_fp8_masked  down
 *   moe_masked_slab_to_expand    back to the expanded rows, times the top-k
 *                                weights
 *   moe_gather                   combine with weight 1
 *
 * Training the bf16 path: after the forward calls (moe_expand_layout_bf16,
 * moe_grouped_gemm_bf16, moe_silu_mul_bf16, moe_grouped_gemm_bf16,
 * moe_gather, whose intermediate buffers the caller keeps), in call order:
 *   moe_gather_backward          d out -> d of the down rows and of the
 *                                top-k weights
 *   moe_grouped_wgrad_bf16       d w2 from the down rows' d and SiLU*up
 *   moe_grouped_dgrad_bf16       d of SiLU*up
 *   moe_silu_mul_bf16_backward   d of the gate_up rows
 *   moe_grouped_wgrad_bf16       d w13 from them and the expanded rows
 *   moe_grouped_dgrad_bf16       d of the expanded rows
 *   moe_gather                   (weights NULL, factor 1) d of the tokens
 *   moe_adamw                    AdamW over all the weights at once
 * Alignment pad rows and rows past the total may hold anything: they are
 * never written, and what they hold enters no result.  Pad rows may be read
 * (moe_silu_mul_bf16_backward loads every row below min(status[0], capacity)
 * before it knows which ones are live).  A captured sequence may be replayed on new
 * routings: every row count, the step number and the learning rate are read
 * on the device.
 *
 * Sources, by page and section:
 *  [P1] SGLang pull request 37261, "feat(deepep_v2): expanded (do_expand=True)
 *       prefill dispatch for DeepEP-V2": Modifications/Core (row labels from
 *       the device psum with no cumsum, host copy or sentinel; the weight
 *       fold into down_proj's fp32 input scale and the UE8M0 fallback), the
 *       SGLANG_DEEPEP_V2_PREFILL_DO_EXPAND section (expanded rows grouped by
 *       expert), and the review thread's note on the expand-mode psum
 *       (psum[e] = align(psum[e-1]) + count[e]; total rows = align(psum[E-1])).
 *  [P2] vLLM pull request 54109, PaddedStandard activation format:
 *       Motivation (inactive rows carry -1 in every top-k slot; the real /
 *       padding boundary psum_recv_per_rank lives on the device; prefill
 *       alignment gaps are zeroed) and Design (the kernel must skip inactive
 *       rows or make them safe to discard, and honour -1 markers rather than
 *       trust row contents).
 *  [P3] SGLang moe_runner/deep_gemm.py source page: _run_contiguous_gemm
 *       (gate_up GEMM, SiLU*up, per-token-group fp8 quant, down GEMM),
 *       _get_compact_all_tokens (capacity bound), _cast_to_e8m0_with_
 *       rounding_up (UE8M0 rule), pre_permute_deepep_v2_to_deep_gemm and
 *       post_permute_deep_gemm_to_deepep_v2 (expanded branch),
 *       pre_permute_standard_to_deep_gemm (bf16 rows quantised per token
 *       group, then scattered into 128-aligned expert blocks) and
 *       post_permute_deep_gemm_to_standard (top-k weights and the routed
 *       scaling factor in the reduction).
 *
 * Conventions for every call:
 *  - Pointers named as device buffers are device memory the caller owns
 *    (allocated, e.g., by PyTorch).  The library never allocates or frees
 *    device memory, copies between host and device, synchronises, or reads
 *    device data on the host.  `stream` is a hipStream_t (NULL = the default stream); work
 *    is enqueued asynchronously on it.
 *  - Host-detectable errors (null pointers, bad sizes, misaligned buffers,
 *    unsupported combinations) are returned as a moe_status before anything
 *    is launched, and nothing is written.  MOE_ERR_LAUNCH reports a failed
 *    kernel launch.
 *  - Device-detected conditions are OR-ed into status[1] by
 *    moe_expand_layout (MOE_FLAG_*); later calls clamp to what is valid.
 *  - fp8 is OCP E4M3 ("fn": bias 7, max 448, no infinities).  bf16 buffers
 *    hold raw 16-bit patterns.  fp32 scales are IEEE float; UE8M0 scales are
 *    one unsigned exponent byte per group, value 2^(b-127).
 *  - Scales: one per 1x128 activation group, one per 128x128 weight block.
 *    The received rows' x_scale is row-major [rows, K/128].  The expanded
 *    activation scales that moe_expand_layout and moe_act_quant write and
 *    moe_grouped_gemm_fp8 reads are K-block-major ("MN-major")
 *    [K/128, capacity]: the scale of expanded row m, K block b sits at
 *    b * capacity + m, so one K block's scales for consecutive rows are one
 *    contiguous run (the GEMM of [P3 _run_contiguous_gemm] likewise takes its
 *    activation scales transposed: TMA-aligned, or mn-major under UE8M0).
 *    Weight scales are [E, N/128, K/128].
 *  - Calls are stateless and reentrant; calls that share output buffers
 *    must be ordered by the caller's streams.
 *  - A buffer that a call writes shares no memory with another of its buffers
 *    unless the call's comment allows it.  The training calls refuse it
 *    (MOE_ERR_UNSUPPORTED).
 */
#ifndef MOE_EXPAND_H
#define MOE_EXPAND_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_NULL = 1,         /* a required pointer is NULL                 */
  MOE_ERR_SHAPE = 2,        /* a size is out of range or inconsistent     */
  MOE_ERR_ALIGNMENT = 3,    /* a pointer or stride is not 16-byte aligned */
  MOE_ERR_UNSUPPORTED = 4,  /* valid in principle, not supported          */
  MOE_ERR_WORKSPACE = 5,    /* workspace missing or too small             */
  MOE_ERR_LAUNCH = 6,       /* a kernel launch (or, for
                               moe_expand_layout_noalloc, the lookup of its
                               scratch address) failed                    */
  MOE_ERR_SCRATCH = 7       /* moe_expand_layout_noalloc: the sizes need
                               more workspace than its static scratch
                               (MOE_NOALLOC_SCRATCH_BYTES) holds          */
} moe_status;

typedef enum {
  MOE_SCALE_F32 = 0,        /* fp32 scale per group                       */
  MOE_SCALE_UE8M0 = 1,      /* one power-of-two exponent byte per group   */
  MOE_SCALE_NONE = 2,       /* moe_expand_layout_bf16 only: keep the rows in
                               bf16, no quantisation, no scales (the bf16-
                               weight path)                               */
  MOE_SCALE_MXFP8 = 3       /* MXFP8: one UE8M0 byte per 1x32 group along K,
                               for activations and for every weight row
                               [P3 DeepGemmMoeQuantInfo: block [1, 32]];
                               activation scales [rows, K/32] bytes
                               (x_scale_stride in bytes, a multiple of 4),
                               expanded ones as one 4-byte word per
                               (128-wide K block, row): the block's four
                               bytes in K order, K-block-major; weight
                               scales [E, N, K/32] bytes.  Supported by
                               moe_expand_layout, moe_grouped_gemm_fp8 (at
                               most 256 experts), moe_act_quant (no fold)  */
} moe_scale_fmt;

typedef enum {
  MOE_GRAD_BF16 = 0,        /* gradients in bf16                          */
  MOE_GRAD_F32 = 1          /* gradients in fp32                          */
} moe_grad_fmt;

typedef enum {
  MOE_STATE_F32 = 0,        /* optimiser states in fp32                   */
  MOE_STATE_FP8 = 1         /* optimiser states as fp8 codes with an fp32
                               scale per group of MOE_STATE_GROUP values  */
} moe_state_fmt;

typedef enum {
  MOE_FLOAT_BF16 = 0,       /* bf16 values                                */
  MOE_FLOAT_F32 = 1         /* fp32 values                                */
} moe_float_fmt;

typedef enum {
  MOE_NORM_LAYER = 0,       /* about the mean                             */
  MOE_NORM_RMS = 1          /* about zero                                 */
} moe_norm_kind;

typedef enum {
  MOE_SCORE_SOFTMAX = 0,
  MOE_SCORE_SIGMOID = 1
} moe_score;

typedef enum {
  MOE_W4_INT4 = 0,          /* two's complement codes -8..7, a bf16 scale
                               per group of 32, 64 or 128 along K         */
  MOE_W4_MXFP4 = 1          /* MXFP4: E2M1 codes (bit 3 the sign; 0, 0.5, 1,
                               1.5, 2, 3, 4, 6), a UE8M0 byte per 32      */
} moe_w4_fmt;

/* Bits of status[1] written by moe_expand_layout. */
#define MOE_FLAG_CAPACITY_OVERFLOW 1 /* total rows > capacity: rows at or past
                                        the capacity were dropped (their slots
                                        get -1)                               */
#define MOE_FLAG_EXPERT_ID_RANGE 2   /* a valid row held an id >= num_experts;
                                        that slot was skipped                 */
#define MOE_FLAG_SLAB_OVERFLOW 4     /* (moe_expand_to_masked_slab) an expert
                                        had more than max_m live rows; rows
                                        past max_m were dropped               */

/* Limits of this build. */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOPK 32
#define MOE_MIN_ALIGN 16
#define MOE_MAX_ALIGN 1024
#define MOE_STATE_GROUP 128
/* Size of moe_expand_layout_noalloc's static per-GPU scratch: calls with
 * moe_expand_workspace_bytes(rows, topk, num_experts) above it are refused
 * (roughly rows * num_experts <= 15 million). */
#define MOE_NOALLOC_SCRATCH_BYTES (4u << 20)

/* Text for a moe_status value (static storage; never NULL). */
const char* moe_status_string(int status);

/* Host, pure.  Largest padded row total over every routing of rows*topk
 * assignments onto num_experts experts with blocks rounded up to `align`
 * rows: align * (n + (rows*topk - n) / align), n = min(rows*topk, E)
 * [P3 _get_compact_all_tokens].  Use it to size the expanded buffers
 * without reading the device-side row count.  Returns -1 on bad input. */
int64_t moe_expand_capacity(int64_t rows, int topk, int num_experts, int align);

/* Host, pure.  Bytes of device workspace moe_expand_layout needs for
 * `rows` receive-buffer rows.  Returns 0 on bad input. */
size_t moe_expand_workspace_bytes(int64_t rows, int topk, int num_experts);

/*
 * Expanded layout [P1 Core + psum note; P2 Motivation/Design; P3
 * pre_permute_deepep_v2_to_deep_gemm].
 *
 * Inputs (device):
 *   x              [rows, x_stride] bytes, fp8 token rows (hidden bytes used)
 *   x_scale        [rows, x_scale_stride] fp32 or UE8M0 bytes (by fmt)
 *   topk_ids       [rows, topk] int32; id < 0 = not for this rank / inactive;
 *                  id >= num_experts is skipped and flagged
 *   topk_weights   [rows, topk] fp32; may be NULL only if row_weight is NULL
 *   psum_recv_per_rank [num_src_ranks] int32 inclusive prefix sum of rows
 *                  received per source rank; its last entry is the number of
 *                  valid rows R_v (clamped to [0, rows]).  NULL: R_v = rows.
 *                  Rows >= R_v are never read as routing.
 * Sizes: hidden % 128 == 0; 1 <= topk <= MOE_MAX_TOPK; 1 <= num_experts <=
 *   MOE_MAX_EXPERTS; align a power of two in [16, 1024]; capacity a multiple
 *   of align (moe_expand_capacity gives one that cannot overflow);
 *   x_stride % 16 == 0 and x 16-byte aligned.
 * Outputs (device, caller-allocated):
 *   ex             [capacity, hidden] fp8 expanded rows
 *   ex_scale       [hidden/128, capacity] K-block-major scales (same
 *                  format as x_scale): row m, block b at b * capacity + m
 *   psum           [num_experts] int32, psum[e] = align(psum[e-1]) + count[e]
 *   m_indices      [capacity] int32: expert of each expanded row, alignment
 *                  pads included; -1 from the total to the capacity
 *   src2dst        [rows, topk] int32: expanded row of each live slot, -1
 *                  otherwise (all slots of rows >= R_v are -1)
 *   row_weight     [capacity] fp32 top-k weight of each expanded row (0 on
 *                  pads); may be NULL
 *   status         [2] int32: status[0] = total expanded rows
 *                  align(psum[E-1]) (may exceed capacity: see the flag),
 *                  status[1] = MOE_FLAG_* bits
 * Rows of one expert are in ascending (row, k) order.  Alignment pad rows
 * get fp8 zero, scale 0 and weight 0.  Rows from the total up to the
 * capacity are left untouched.
 * workspace: device, >= moe_expand_workspace_bytes(rows, topk, num_experts)
 *   bytes, 256-byte aligned, no initialisation needed.
 */
moe_status moe_expand_layout(
    const void* x, int64_t x_stride, const void* x_scale,
    int64_t x_scale_stride, moe_scale_fmt fmt,
    const int32_t* topk_ids, const float* topk_weights,
    const int32_t* psum_recv_per_rank, int num_src_ranks,
    int64_t rows, int hidden, int topk, int num_experts, int align,
    int64_t capacity,
    void* ex, void* ex_scale, int32_t* psum, int32_t* m_indices,
    int32_t* src2dst, float* row_weight, int32_t* status,
    void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_expand_layout with no workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation.  Every other argument, output and error
 * is as moe_expand_layout's; the call allocates and frees nothing.
 *
 * The workspace is a static device array of MOE_NOALLOC_SCRATCH_BYTES inside
 * the library: each GPU the library runs on holds its own copy until the
 * process ends.  Its address is looked up on the first call on each device
 * (that call must have the device current, as every call must).  Sizes whose
 * workspace (moe_expand_workspace_bytes) exceeds the array return
 * MOE_ERR_SCRATCH before anything is launched; a failed address lookup
 * returns MOE_ERR_LAUNCH.  All calls on one GPU share the array: calls that
 * may run concurrently on one GPU (unordered streams) race and must not be
 * issued; calls ordered on one stream are safe, and nothing needs clearing
 * between them.
 */
moe_status moe_expand_layout_noalloc(
    const void* x, int64_t x_stride, const void* x_scale,
    int64_t x_scale_stride, moe_scale_fmt fmt,
    const int32_t* topk_ids, const float* topk_weights,
    const int32_t* psum_recv_per_rank, int num_src_ranks,
    int64_t rows, int hidden, int topk, int num_experts, int align,
    int64_t capacity,
    void* ex, void* ex_scale, int32_t* psum, int32_t* m_indices,
    int32_t* src2dst, float* row_weight, int32_t* status, void* stream);

/*
 * Expanded layout of bf16 token rows, quantised on the way [P3
 * pre_permute_standard_to_deep_gemm: per-token-group fp8 quantisation of the
 * hidden states, then the scatter into the aligned expert blocks].
 *
 * As moe_expand_layout, except:
 *   x          [rows, x_stride] bf16 token rows (x_stride in elements,
 *              >= hidden; x_stride * 2 % 16 == 0, x 16-byte aligned); there
 *              is no x_scale.  Each valid row with a live slot is read once,
 *              quantised per 1x128 group and written to every destination:
 *                amax = max(max |x| over the group, 1e-10)
 *                fp32:  scale = amax / 448, q = fp8_rne(x * (448 / amax))
 *                UE8M0: b = smallest exponent byte with 2^(b-127) >= amax/448,
 *                       q = fp8_rne(x * 2^(127-b))
 *              (each operation rounded in fp32; the same rule as
 *              moe_act_quant's).  Rows without a live slot are not read.
 *              fmt MOE_SCALE_NONE (the bf16-weight path): the rows are kept
 *              in bf16 and copied as they are; ex is then [capacity, hidden]
 *              bf16, ex_scale is not used (may be NULL), pad rows are 0.
 * Errors, ownership and every other argument: as moe_expand_layout.
 */
moe_status moe_expand_layout_bf16(
    const void* x, int64_t x_stride, moe_scale_fmt fmt,
    const int32_t* topk_ids, const float* topk_weights,
    const int32_t* psum_recv_per_rank, int num_src_ranks,
    int64_t rows, int hidden, int topk, int num_experts, int align,
    int64_t capacity,
    void* ex, void* ex_scale, int32_t* psum, int32_t* m_indices,
    int32_t* src2dst, float* row_weight, int32_t* status,
    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Contiguous grouped fp8 GEMM, "NT": out[m, :] = A[m, :] . W[e]^T for every
 * expanded row m of expert e [P3 _run_contiguous_gemm; P1 Core].
 *
 *   a        [capacity, k] fp8 (row stride k), a_scale [k/128, capacity]
 *            K-block-major (row m, block b at b * capacity + m)
 *   w        [num_experts, n, k] fp8 (k contiguous), w_scale
 *            [num_experts, n/128, k/128]; a_scale and w_scale in `fmt`
 *   psum, status  as written by moe_expand_layout
 *   out      [capacity, n] bf16
 * Expert e owns rows [align(psum[e-1]), align(psum[e])) -- exactly the rows
 * moe_expand_layout labels e in m_indices -- so the kernel reads the layout
 * from the device psum (no per-row labels needed).  For every such row
 * m < min(status[0], capacity):
 *   out[m,j] = bf16( sum_kb sa[m,kb] * sw[e,j/128,kb] *
 *                    sum_{t in kb} a[m,t] * w[e,j,t] )
 * accumulated in fp32 (UE8M0: the exponents are applied by the matrix
 * cores).  Row groups made only of alignment padding (rows >= psum[e]) may
 * be skipped and left unwritten; rows past the total are never written.
 * Sizes: n % 128 == 0, k % 128 == 0, k / 128 <= 511 (else
 * MOE_ERR_UNSUPPORTED), align as for the layout, capacity a multiple of
 * align.  Alignment: a, w, out 16 bytes; a_scale 16 bytes (fp32) or 4
 * (UE8M0); w_scale 4 bytes.  UE8M0 scale arrays are read in aligned 4-byte
 * words, so their allocations must extend to a multiple of 4 bytes.
 */
moe_status moe_grouped_gemm_fp8(
    const void* a, const void* a_scale, moe_scale_fmt fmt,
    const void* w, const void* w_scale,
    const int32_t* psum, const int32_t* status,
    int64_t capacity, int n, int k, int num_experts, int align,
    void* out, void* stream);

/*
 * SiLU(gate)*up with per-1x128 fp8 quantisation [P3 _run_contiguous_gemm,
 * _situ_mul_quant_contig_kernel (quantisation rule), _cast_to_e8m0_with_
 * rounding_up; P1 Core (fold)].
 *
 *   gate_up   [capacity, 2*inter] bf16: gate = first half, up = second
 *   m_indices, psum, status  as written by moe_expand_layout
 *   fold_weight  [capacity] fp32 (the layout's row_weight) or NULL.  Only
 *                with MOE_SCALE_F32 (UE8M0 + fold -> MOE_ERR_UNSUPPORTED).
 *   out       [capacity, inter] fp8; out_scale [inter/128, capacity] in fmt,
 *             K-block-major (row m, group g at g * capacity + m)
 * For each live row m (m < min(status[0], capacity), m < psum[e]):
 *   y = g / (1 + exp(-g)) * u in fp32; per group amax = max(|y|, 1e-10);
 *   F32:   s = amax / 448, q = fp8_rne(y * (448 / amax)), s *= fold_weight[m]
 *   UE8M0: b = smallest power-of-two exponent byte with 2^(b-127) >= amax/448,
 *          q = fp8_rne(y * 2^(127-b))
 * Alignment pad rows (psum[e] <= m < align(psum[e])) get q = 0, scale 0.
 * Sizes: inter % 128 == 0; gate_up and out 16-byte aligned.
 */
moe_status moe_act_quant(
    const void* gate_up, const int32_t* m_indices, const int32_t* psum,
    const int32_t* status, int64_t capacity, int inter, int num_experts,
    int align, moe_scale_fmt fmt, const float* fold_weight,
    void* out, void* out_scale, void* stream);

/*
 * Weighted gather back to token rows [P3 post_permute_deep_gemm_to_deepep_v2
 * and ep_gather's use in post_permute_deep_gemm_to_deepep_normal; P1 Core
 * (UE8M0 weighting of the down output); P3 post_permute_deep_gemm_to_standard
 * (the routed scaling factor)].
 *
 *   expert_out   [capacity, hidden] bf16 (down projection output)
 *   src2dst      [rows, topk] int32 as written by moe_expand_layout;
 *                entries outside [0, capacity) are treated as -1
 *   topk_weights [rows, topk] fp32, or NULL when the weights were folded
 *   routed_scaling_factor  multiplies each row's sum (1 on the expand path;
 *                the model's factor on the standard path); a NaN or infinite
 *                factor is MOE_ERR_UNSUPPORTED
 *   psum_recv_per_rank / num_src_ranks  as for the layout (R_v)
 *   out          [rows, hidden] bf16
 * For r < R_v: out[r] = bf16( f * sum over k ascending with src2dst[r,k] >= 0
 *   of c_k * float(expert_out[src2dst[r,k]]) ), c_k = topk_weights[r,k] or 1,
 * f = routed_scaling_factor, each product and sum rounded to fp32 in that
 * order.  Valid rows with no live slot become 0.  Rows >= R_v are not
 * written.
 * Sizes: hidden % 128 == 0 and hidden <= 8192 (else MOE_ERR_UNSUPPORTED);
 * buffers 16-byte aligned.
 */
moe_status moe_gather(
    const void* expert_out, const int32_t* src2dst, const float* topk_weights,
    float routed_scaling_factor, const int32_t* psum_recv_per_rank, int num_src_ranks,
    int64_t rows, int hidden, int topk, int64_t capacity,
    void* out, void* stream);

/*
 * Expanded rows -> the decode path's masked slab [P1 "Why decode stays on V1
 * low_latency": the fixed-height slab and the bridge into it; P3
 * pre_permute_deepep_v2_to_deep_gemm, masked branch].
 *
 *   ex, ex_scale   as written by moe_expand_layout (scales [hidden/128,
 *                  capacity] K-block-major), psum and status likewise
 *   slab           [num_experts * max_m, hidden] fp8: row e * max_m + i =
 *                  expanded row align(psum[e-1]) + i for i < masked_m[e]
 *   slab_scale     [hidden/128, num_experts * max_m] K-block-major
 *   masked_m       [num_experts] int32 = min(live rows of e, max_m)
 * Slab rows past masked_m[e] are not written.  An expert with more than
 * max_m live rows sets MOE_FLAG_SLAB_OVERFLOW in status[1] (written here:
 * status is read-write) and its rows past max_m are dropped.
 * Sizes: max_m >= 16 and a multiple of 16; num_experts * max_m <= 2^30.
 */
moe_status moe_expand_to_masked_slab(
    const void* ex, const void* ex_scale, moe_scale_fmt fmt, const int32_t* psum,
    int32_t* status, int64_t capacity, int hidden, int num_experts, int align, int max_m,
    void* slab, void* slab_scale, int32_t* masked_m, void* stream);

/*
 * Contiguous grouped bf16 GEMM, "NT" [P3 _run_bf16_contiguous_gemm,
 * grouped_gemm_nt_bf16_contig]: as moe_grouped_gemm_fp8 with bf16 operands
 * and no scales.
 *   a    [capacity, k] bf16, w [num_experts, n, k] bf16 (k contiguous)
 *   out  [capacity, n] bf16: the fp32 sum of the bf16 products rounded once
 * Sizes: n % 128 == 0, k % 64 == 0; buffers 16-byte aligned.
 */
moe_status moe_grouped_gemm_bf16(
    const void* a, const void* w, const int32_t* psum, const int32_t* status,
    int64_t capacity, int n, int k, int num_experts, int align, void* out,
    void* stream);

/*
 * SiLU(gate)*up to bf16 for every live expanded row [P3
 * _run_bf16_contiguous_gemm: silu_and_mul between the bf16 GEMMs]:
 *   gate_up  [capacity, 2*inter] bf16 -> out [capacity, inter] bf16,
 *   y = bf16_rne(silu(g) * u) with silu(g) = g / (1 + exp(-g)), in fp32.
 * Alignment pad rows are not written (the GEMM never reads them).
 */
moe_status moe_silu_mul_bf16(
    const void* gate_up, const int32_t* m_indices, const int32_t* psum,
    const int32_t* status, int64_t capacity, int inter, int num_experts,
    int align, void* out, void* stream);

/*
 * Masked grouped fp8 GEMM [P3 _run_masked_gemm]: as moe_grouped_gemm_fp8 on
 * the slab, expert e's rows being [e * max_m, e * max_m + masked_m[e]).
 *   a        [num_experts * max_m, k] fp8, a_scale [k/128, num_experts * max_m]
 *   w, w_scale as moe_grouped_gemm_fp8
 *   out      [num_experts * max_m, n] bf16; rows past masked_m[e] unwritten
 * Sizes: max_m a multiple of 16; n, k multiples of 128.
 */
moe_status moe_grouped_gemm_fp8_masked(
    const void* a, const void* a_scale, moe_scale_fmt fmt, const void* w,
    const void* w_scale, const int32_t* masked_m, int max_m, int n, int k,
    int num_experts, void* out, void* stream);

/*
 * SiLU(gate)*up and per-1x128 fp8 quantisation of the slab's live rows
 * [P3 _run_masked_gemm's activation; the rule of moe_act_quant, no fold]:
 *   gate_up  [num_experts * max_m, 2*inter] bf16
 *   out      [num_experts * max_m, inter] fp8, out_scale [inter/128,
 *            num_experts * max_m] K-block-major
 * Rows past masked_m[e] are neither read nor written.
 */
moe_status moe_act_quant_masked(
    const void* gate_up, const int32_t* masked_m, int max_m, int inter,
    int num_experts, moe_scale_fmt fmt, void* out, void* out_scale, void* stream);

/*
 * The slab's down rows back to the expanded layout [P1 "Why decode stays on
 * V1 low_latency"; P3 post_permute_deep_gemm_to_deepep_v2, masked branch:
 * the top-k weights are applied here, the expanded combine takes none].
 *   slab_out    [num_experts * max_m, hidden] bf16
 *   masked_m, max_m  as written / used by moe_expand_to_masked_slab
 *   psum, status, m_indices  from moe_expand_layout
 *   row_weight  [capacity] fp32 top-k weight of each expanded row, or NULL
 *   out         [capacity, hidden] bf16: for every expanded row m below the
 *               total, of expert e at i = m - align(psum[e-1]):
 *               bf16(row_weight[m] * slab_out[e * max_m + i]) if i <
 *               masked_m[e] (fp32 product, one rounding; a copy when
 *               row_weight is NULL); 0 for rows the slab height dropped
 *               (masked_m[e] <= i < psum[e] - align(psum[e-1])).  Alignment
 *               pad rows and rows past the total are not written.
 */
moe_status moe_masked_slab_to_expand(
    const void* slab_out, const int32_t* masked_m, int max_m, const int32_t* psum,
    const int32_t* status, const int32_t* m_indices, const float* row_weight,
    int64_t capacity, int hidden, int num_experts, int align, void* out, void* stream);

/*
 * Input gradient of moe_grouped_gemm_bf16: for every live expanded row m of
 * expert e (m < psum[e], m < min(status[0], capacity))
 *   dx[m, t] = bf16( sum_j dy[m, j] * w[e, j, t] )
 * accumulated in fp32.  n and k are those of the forward call: dy is the
 * gradient of its output.
 *   dy   [capacity, n] bf16, w [num_experts, n, k] bf16 as in the forward
 *        call (not transposed), psum, status as there
 *   dx   [capacity, k] bf16; rows that are not live are not written
 * Rows of dy that are not live do not enter any result.
 * Sizes, alignment and errors as moe_grouped_gemm_bf16 (n % 128 == 0,
 * k % 64 == 0, and n / 64, k / 64 <= 511).
 */
moe_status moe_grouped_dgrad_bf16(
    const void* dy, const void* w, const int32_t* psum, const int32_t* status,
    int64_t capacity, int n, int k, int num_experts, int align, void* dx,
    void* stream);

/*
 * Host, pure.  Bytes of device workspace moe_grouped_wgrad_bf16 needs (0 for
 * most sizes: only few, long reductions are split over workgroups and joined
 * through it).  Returns 0 on bad input.
 */
size_t moe_grouped_wgrad_workspace_bytes(int64_t capacity, int n, int k, int num_experts);

/*
 * Weight gradient of moe_grouped_gemm_bf16: for every expert e
 *   dw[e, j, t] = sum over the live rows m of e of dy[m, j] * x[m, t]
 * accumulated in fp32 (the order of the sum depends on the sizes and the
 * rows of e only: equal calls give equal bits) and rounded once to `fmt`.
 * accumulate != 0: the sum is added to dw's value in fp32 first (dw holds
 * the gradients of earlier calls).  An expert without live rows gets 0, or
 * keeps its values when accumulating.
 *   dy   [capacity, n] bf16, x [capacity, k] bf16 (the forward call's a)
 *   dw   [num_experts, n, k] in `fmt`
 * Rows that are not live do not enter any result, whatever they hold.
 * workspace: device, >= moe_grouped_wgrad_workspace_bytes(...) bytes,
 * 256-byte aligned, no initialisation needed; may be NULL when that is 0.
 * Calls that may overlap need a workspace each.
 * Sizes and errors as moe_grouped_dgrad_bf16; a short workspace is
 * MOE_ERR_WORKSPACE.  Buffers 16-byte aligned.
 */
moe_status moe_grouped_wgrad_bf16(
    const void* dy, const void* x, const int32_t* psum, const int32_t* status,
    int64_t capacity, int n, int k, int num_experts, int align, moe_grad_fmt fmt,
    int accumulate, void* dw, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of moe_silu_mul_bf16, for every live expanded row:
 *   gate_up    [capacity, 2*inter] bf16: g = first half, u = second, as given
 *              to the forward call
 *   dy         [capacity, inter] bf16
 *   d_gate_up  [capacity, 2*inter] bf16: with s = 1 / (1 + exp(-g)) in fp32
 *              d g = dy * u * (s * (1 + g * (1 - s))),  d u = dy * (g * s),
 *              each rounded once to bf16
 * Rows that are not live are not written.  d_gate_up may be gate_up itself
 * (each value is read before its place is written).
 * Sizes and errors as moe_silu_mul_bf16.
 */
moe_status moe_silu_mul_bf16_backward(
    const void* gate_up, const void* dy, const int32_t* m_indices, const int32_t* psum,
    const int32_t* status, int64_t capacity, int inter, int num_experts, int align,
    void* d_gate_up, void* stream);

/*
 * Gradient of moe_gather (out[r] = f * sum_k c[r,k] * expert_out[src2dst[r,k]]):
 *   dout            [rows, hidden] bf16
 *   expert_out, src2dst, topk_weights, routed_scaling_factor,
 *   psum_recv_per_rank, num_src_ranks  as given to the forward call;
 *                   src2dst names each expanded row at most once, as
 *                   moe_expand_layout writes it
 *   d_expert_out    [capacity, hidden] bf16: for each live slot (r, k),
 *                   r < R_v, row src2dst[r,k] = bf16( (f * c[r,k]) * dout[r] ),
 *                   c = 1 when topk_weights is NULL; other rows are not written
 *   d_topk_weights  [rows, topk] fp32: f * sum_h dout[r,h] *
 *                   expert_out[src2dst[r,k], h], summed in fp32; 0 for the
 *                   slots of valid rows that are not live; rows >= R_v are
 *                   not written.  May be NULL (expert_out is then not read
 *                   and may be NULL too).
 * Sizes and errors as moe_gather.
 */
moe_status moe_gather_backward(
    const void* dout, const void* expert_out, const int32_t* src2dst,
    const float* topk_weights, float routed_scaling_factor,
    const int32_t* psum_recv_per_rank, int num_src_ranks, int64_t rows, int hidden,
    int topk, int64_t capacity, void* d_expert_out, float* d_topk_weights, void* stream);

/* One tensor of moe_adamw (device pointers, 16-byte aligned; grad in the
 * given format; all hold numel values in the same order). */
typedef struct {
  float* master;            /* fp32 parameters, updated                     */
  const void* grad;         /* gradient, bf16 or fp32                       */
  void* m;                  /* first moment: fp32, or fp8 codes             */
  void* v;                  /* second moment: fp32, or fp8 codes of its root */
  void* param;              /* bf16 copy of the updated master, or NULL     */
  float* m_scale;           /* MOE_STATE_FP8: [ceil(numel/128)] fp32        */
  float* v_scale;           /* MOE_STATE_FP8: [ceil(numel/128)] fp32        */
  int64_t numel;
  moe_grad_fmt grad_fmt;
  moe_state_fmt state_fmt;
} moe_adamw_tensor;

/*
 * One AdamW step over num_tensors tensors (host array, read before the call
 * returns), with decoupled weight decay.  With t = *step (the number of this
 * step, from 1), in fp32 (m and v: each operation rounded by itself; the
 * quotients of the step within a few fp32 steps):
 *   g = grad * *grad_scale                       (grad_scale NULL: g = grad)
 *   m = m * beta1 + g * (1 - beta1)
 *   v = v * beta2 + (g * g) * (1 - beta2)
 *   master -= *lr * (m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps)
 *                    + weight_decay * master)
 *   param = bf16(master)
 * step (int64), lr and grad_scale (fp32) are device scalars: a captured call
 * takes their values at each replay.
 * MOE_STATE_FP8: m and r = sqrt(v) are kept per group of 128 consecutive
 * values as E4M3 codes and a scale: amax = max(max |x| over the group,
 * 2^-100), scale = amax * fl(1/448), code = fp8_rne(x * (fl(1/amax) * 448));
 * a positive r gets at least the smallest positive code (2^-9), since a second
 * moment of 0 would let the step divide by eps alone.  The step itself uses m and v
 * before they are coded.  An infinite value spoils its group.
 * A state whose beta is above 31/32 moves by far less than the codes' distance
 * (6 to 12 %) in a step and would keep its nearest code for good.  It gets one
 * of its two neighbouring codes instead, the expected one being its value: with
 * 32-bit h = (m_bits ^ rotl(r_bits, 11)) * 0x9e3779b9 + t * 0xbb67ae85,
 * h = (h ^ h >> 16) * 0x9e3779b9, h = (h ^ h >> 15) * 0x6a09e667, h ^= h >> 16,
 * the upper (m) or lower (r) 20 bits of h, as a fraction of the distance, are
 * added to the magnitude before it is cut off to a code.  Equal calls give equal
 * codes.  A single root is then off by 15 to 20 % in the mean square (nearest
 * codes at smaller betas: 8 %), without a bias.
 * The last group of a tensor may be short.
 * Errors: numel < 0 or > 2^33, num_tensors < 0, hyperparameters
 * out of range (beta in [0, 1), eps 0 or at least 2^-126, weight_decay >= 0,
 * all finite):
 * MOE_ERR_SHAPE; unknown formats, or an array that is written (master, m, v,
 * param, the scales) and shares memory with any other of the call's arrays or
 * scalars: MOE_ERR_UNSUPPORTED.  Gradients may be shared.  Tensors with numel
 * 0 are skipped.
 */
moe_status moe_adamw(
    const moe_adamw_tensor* tensors, int num_tensors, const int64_t* step,
    const float* lr, const float* grad_scale, double beta1, double beta2, double eps,
    double weight_decay, void* stream);

/*
 * The norm of the residual stream in front of a layer, with the branch before
 * it (attention's, or the last layer's output) added on the way:
 *   h = x + branch                      (branch NULL: h = x)
 *   mu = mean(h), rstd = 1 / sqrt(mean((h - mu)^2) + eps)
 *                                       (MOE_NORM_RMS: mu = 0)
 *   y = (h - mu) * rstd * weight + bias (bias NULL: none)
 * in fp32, the variance about the mean.  With a branch, h is first rounded to
 * the stream's type x_fmt: the norm is of the stream as it is kept.
 *   x       [rows, x_stride] bf16 or fp32 (x_fmt), hidden columns used
 *   branch  [rows, hidden] bf16 or NULL
 *   weight, bias  [hidden] in w_fmt; bias may be NULL
 *   sum     [rows, hidden] in x_fmt: h; may be NULL, and must be without a
 *           branch; may be x itself where x_stride is hidden
 *   y       [rows, hidden] bf16
 *   mean, rstd  [rows] fp32, what the backward pass takes; may be NULL (mean:
 *           0 for MOE_NORM_RMS)
 *   psum_recv_per_rank / num_src_ranks  as for the layout (R_v)
 * Rows >= R_v are neither read nor written.  A row whose h holds a NaN gets NaN
 * throughout, and one with an infinity, too, but for MOE_NORM_RMS: its rstd is 0, and
 * y the NaN of 0 times infinity there and bias (or 0) beside it.  So is, in fp32, a
 * row whose sum of squares passes the largest value, without the NaN.
 * Sizes: hidden % 8 == 0 and hidden <= 8192 (else MOE_ERR_UNSUPPORTED);
 * hidden <= x_stride <= 2^30, rows of x 16-byte aligned; 0 <= eps < infinity; buffers
 * 16-byte aligned, mean and rstd 4-byte.  A buffer that is written and shares
 * memory with another (but for sum and x, above): MOE_ERR_UNSUPPORTED.
 */
moe_status moe_layer_norm(
    const void* x, int64_t x_stride, moe_float_fmt x_fmt, const void* branch,
    const void* weight, const void* bias, moe_float_fmt w_fmt, moe_norm_kind kind, float eps,
    const int32_t* psum_recv_per_rank, int num_src_ranks, int64_t rows, int hidden, void* sum,
    void* y, float* mean, float* rstd, void* stream);

/* Host, pure.  Bytes of device workspace moe_layer_norm_backward needs where
 * it writes dweight or dbias.  Returns 0 on bad input. */
size_t moe_layer_norm_backward_workspace_bytes(int64_t rows, int hidden);

/*
 * Gradient of moe_layer_norm.  With d = dy + dy2, xh = (x - mean) * rstd and
 * g = d * weight, in fp32:
 *   dx = rstd * (g - mean(g) - xh * mean(g * xh)) + dsum
 *                                       (MOE_NORM_RMS: without mean(g))
 *   dweight = sum over rows of d * xh,  dbias = sum over rows of d
 *   dy      [rows, hidden] bf16; dy2 the same, of a second reader of y (the
 *           gate beside the experts), or NULL
 *   x       [rows, x_stride] in x_fmt: the forward call's h (its sum, or x
 *           where it had no branch)
 *   mean, rstd  [rows] as the forward call wrote them; mean is not read for
 *           MOE_NORM_RMS (may be NULL)
 *   dsum    [rows, hidden] in x_fmt: the gradient that reaches h along the
 *           residual stream, or NULL
 *   dx      [rows, hidden] in x_fmt: the gradient of h, which is x's and the
 *           branch's; may be dsum itself
 *   dweight, dbias  [hidden] in grad_fmt; either may be NULL.  accumulate != 0:
 *           the sums are added to what they hold, in fp32, and rounded once.
 *           Without a valid row they become 0 (or stay, accumulating).
 * Equal calls give equal bits.  Rows >= R_v enter no result, and their dx is
 * not written.
 * workspace: device, >= moe_layer_norm_backward_workspace_bytes(rows, hidden)
 * bytes, 256-byte aligned, no initialisation needed; not used without dweight
 * and dbias (may be NULL then).  Calls that may overlap need one each.
 * Sizes and errors as moe_layer_norm; a short workspace is MOE_ERR_WORKSPACE.
 */
moe_status moe_layer_norm_backward(
    const void* dy, const void* dy2, const void* x, int64_t x_stride, moe_float_fmt x_fmt,
    const void* weight, moe_float_fmt w_fmt, moe_norm_kind kind, const float* mean,
    const float* rstd, const void* dsum, const int32_t* psum_recv_per_rank, int num_src_ranks,
    int64_t rows, int hidden, void* dx, void* dweight, void* dbias, moe_grad_fmt grad_fmt,
    int accumulate, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The router: each token's experts and their weights from the gate's logits,
 * in the form that the layout takes.
 *   logits  [rows, logits_stride] bf16 or fp32, num_experts columns used
 *   bias    [num_experts] fp32 or NULL: added to the scores for the choice only
 *   score   s = softmax(logits) or 1 / (1 + exp(-logits))
 *   num_groups, topk_groups  1, 1: any expert.  Otherwise the experts are
 *           num_groups runs of equal length, and only the topk_groups groups
 *           with the largest sum of their two largest s + bias are chosen from
 *   topk_ids      [rows, topk] int32: the topk largest s + bias, falling; the
 *           lowest expert (group) first among equals
 *   topk_weights  [rows, topk] fp32: s of each, or s / (sum of the chosen s)
 *           with normalize != 0
 *   psum_recv_per_rank / num_src_ranks  as for the layout (R_v)
 * A logit (or bias) of -inf or NaN is an expert that is not available: it is
 * never chosen, and a NaN or -inf logit has score 0.  +inf counts as the
 * largest finite fp32 value.  Slots for which no expert is left (all of them
 * in a row without any) get id -1 and weight 0.  Without a bias and groups
 * the experts are compared by their logits (-0 and +0 are equal), otherwise by fp64
 * scores (and sums of scores), which are told apart down to fp64's own rounding: logits
 * whose scores fp64 holds as one number are equal then.  A bias of the lowest
 * fp32 value is a key like others; only -inf and NaN exclude an expert.  Rows >= R_v
 * are neither read nor written.
 * Sizes: 1 <= topk <= min(num_experts, MOE_MAX_TOPK), num_experts <=
 * MOE_MAX_EXPERTS, num_groups <= 64 and a divisor of num_experts,
 * logits_stride >= num_experts; buffers aligned to their elements.  An output
 * that shares memory with another buffer: MOE_ERR_UNSUPPORTED.
 */
moe_status moe_router(
    const void* logits, int64_t logits_stride, moe_float_fmt fmt, const float* bias,
    moe_score score, int num_groups, int topk_groups, int normalize,
    const int32_t* psum_recv_per_rank, int num_src_ranks, int64_t rows, int num_experts,
    int topk, int32_t* topk_ids, float* topk_weights, void* stream);

/*
 * Gradient of moe_router's weights (the choice has none):
 *   topk_ids        [rows, topk] as the forward call wrote them; slots outside
 *                   [0, num_experts) or of an expert that is not available
 *                   are passed over (their d_topk_weights is not read into any result)
 *   d_topk_weights  [rows, topk] fp32
 *   d_logits        [rows, d_logits_stride] in fmt, num_experts columns
 *                   written: with w the weights, g their gradients and sums
 *                   over the row's slots,
 *     softmax             d x_j = w_j g_j - s_j * sum(w g)    (every expert)
 *     softmax, normalize  d x_j = w_j (g_j - sum(w g))        (0 if not chosen)
 *     sigmoid             d x_j = w_j (1 - s_j) g_j
 *     sigmoid, normalize  d x_j = w_j (1 - s_j) (g_j - sum(w g))
 *                   An expert that is not available gets 0; one that is named
 *                   twice gets the sum of its slots.
 * Rows >= R_v are neither read nor written.  Sizes and errors as moe_router.
 */
moe_status moe_router_backward(
    const void* logits, int64_t logits_stride, moe_float_fmt fmt, moe_score score, int normalize,
    const int32_t* topk_ids, const float* d_topk_weights, const int32_t* psum_recv_per_rank,
    int num_src_ranks, int64_t rows, int num_experts, int topk, void* d_logits,
    int64_t d_logits_stride, void* stream);

/*
 * Contiguous grouped GEMM with 4-bit weights, "NT": as moe_grouped_gemm_bf16,
 * for every live expanded row m of expert e (m < psum[e], m < min(status[0],
 * capacity))
 *   out[m, j] = bf16( sum over groups g of s[e, j, g] *
 *                     sum over t in g of a[m, t] * q[e, j, t] )
 * accumulated in fp32.
 *   a        [capacity, k] bf16
 *   w        [num_experts, n, k/2] bytes of two codes each, the lower k in the
 *            low four bits
 *   w_scale  [num_experts, n, k/group]: bf16 (MOE_W4_INT4; group 32, 64 or
 *            128) or UE8M0 bytes (MOE_W4_MXFP4; group 32).  MXFP4 weights are
 *            exact for scale bytes 2..252 and NaN for byte 255; other bytes make weights
 *            outside bf16's normal range.
 *   out      [capacity, n] bf16; rows that are not live are not written
 * Rows of a that are not live do not enter any result.  Equal calls give equal bits; a
 * row's last bit may depend on how many rows there are beside it (sums over k are formed
 * in parts for few rows and in one for many).  MOE_W4_INT4 forms sums of a (8 + q) and
 * of 8 a: infinities in a row give NaN, and values beyond 2^120 may.
 * Sizes: n % 128 == 0, k % 128 == 0 and n / 64, k / 64 <= 511 (else
 * MOE_ERR_UNSUPPORTED), align and capacity as for the layout; buffers
 * 16-byte aligned.  out sharing memory with another buffer:
 * MOE_ERR_UNSUPPORTED.
 */
moe_status moe_grouped_gemm_w4(
    const void* a, const void* w, const void* w_scale, moe_w4_fmt fmt, int group,
    const int32_t* psum, const int32_t* status, int64_t capacity, int n, int k, int num_experts,
    int align, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPAND_H */
