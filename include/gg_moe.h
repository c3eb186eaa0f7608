/*
 * gg_moe.h -- C ABI of libgg_moe: grouped GEMMs of the MoE expert backward
 * pass on AMD Instinct MI355X (gfx950).
 *
 * The entry points, each defined on an NVIDIA cuDNN frontend documentation
 * page (the pages describe the method; this library is an independent
 * implementation for CDNA4):
 *
 *   gg_wgrad   "Grouped GEMM + WGrad (Unified)", section "Operation":
 *              Wgrad[e] = A[:, begin:end] @ B[begin:end, :] over the token
 *              slice of expert e, accumulate or overwrite.
 *   gg_wgrad_mx  the same, section "Block-scaled contract", on MXFP8
 *              operands.
 *   gg_dglu    "Grouped GEMM + dGLU (SM100)", section "BF16 contract /
 *              Tensors, layouts, and equation": R_g = alpha_g^2 A_g B_g^T
 *              fused with the dSwiGLU / dGeGLU backward over 32-wide
 *              interleaved blocks of X_g = beta_g C_g, a dprob row reduction
 *              and an optional per-expert dbias.
 *   gg_dglu_mx "Grouped GEMM + dGLU (SM100)", section "Block-scaled
 *              contract / Equations": the same fused op on MXFP8 operands,
 *              R_g = alpha_g^2 deq(A_g) deq(B_g)^T, with the per-expert amax
 *              of the input and gate halves of D ("Shapes": (L, 2, 1)).
 *   gg_dsrelu  "Grouped GEMM + dsReLU (SM100)", section "Equations":
 *              G = alpha_g deq(A) deq(B)^T on MXFP8 operands,
 *              D_row = prob * 2 * C * relu(G), dprob = sum_n C relu(G)^2,
 *              plus the per-expert Amax of section "Shapes".
 *
 * and, defined here, what stands before and after them in a training step:
 *
 *   gg_route, gg_route_bwd   the router: top-k choice, weights, tokens per
 *              expert, balance loss; the gradient of its logits.
 *   gg_plan, gg_permute, gg_combine, gg_combine_bwd   tokens to the rows of
 *              the grouped GEMMs, and back.
 *   gg_grad_norm, gg_grad_clip   the 2-norm over many gradients, and
 *              clipping by it.
 *
 * and the forward pass of the experts, with weights in 4 bits:
 *
 *   gg_mx4_quant, gg_mx4_dequant   rows to MXFP4 and back.
 *   gg_glu     the gated activation whose backward gg_dglu computes.
 *   gg_gemm_mx4   the grouped product of MXFP4 rows and weights.
 *   gg_moe_few   a whole layer for up to 64 tokens, bf16 or MXFP4 weights.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers are device pointers unless marked [host].  Every buffer is
 *   owned by the caller; the library allocates no memory.  Its scratch space
 *   is the caller's `workspace` (size from the matching *_workspace_size),
 *   which makes the calls safe to capture into a HIP graph.
 * - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *   stream).  Pointer arrays and the memory they point to must stay alive
 *   and unmoved until the stream has finished the call ("Output modes" of
 *   the wgrad page; the pointer-array note of the dGLU page).  Two calls that
 *   may overlap must not share a workspace (wgrad page, "Block-scaled
 *   contract", on the descriptor workspace).
 * - Every entry point returns a gg_status.  All argument checks run on the
 *   host, before any device work is queued; on failure nothing is launched
 *   and gg_last_error() holds a message.
 * - The values of offsets / padded_offsets live in device memory and are not
 *   read by the host (the pages' traced paths cannot host-validate them
 *   either).  The kernels clamp every range they derive from them, so a
 *   malformed array never causes an out-of-bounds access; the violation is
 *   recorded in the workspace's error word, readable with gg_device_error().
 *   GG_FLAG_VALIDATE_OFFSETS instead copies the array to the host, waits
 *   for `stream`, and rejects a malformed array with GG_ERR_OFFSETS.
 */
#ifndef GG_MOE_H
#define GG_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GG_ABI_VERSION 3

typedef enum {
    GG_OK = 0,
    GG_ERR_NULL = 1,         /* a required pointer is NULL                       */
    GG_ERR_SHAPE = 2,        /* a size is out of range or inconsistent           */
    GG_ERR_DTYPE = 3,        /* unsupported dtype or dtype pairing               */
    GG_ERR_LAYOUT = 4,       /* unsupported major / stride                       */
    GG_ERR_ALIGN = 5,        /* a base pointer or row pitch is not 16-B aligned  */
    GG_ERR_MODE = 6,         /* not exactly one output (wgrad) / weight mode     */
    GG_ERR_WORKSPACE = 7,    /* workspace NULL or smaller than required          */
    GG_ERR_UNSUPPORTED = 8,  /* valid per the pages but outside this library     */
    GG_ERR_DEVICE = 9,       /* no gfx950 device current                         */
    GG_ERR_HIP = 10,         /* a HIP runtime call failed                        */
    GG_ERR_OFFSETS = 11,     /* offsets rejected by GG_FLAG_VALIDATE_OFFSETS     */
    GG_ERR_VALUE = 12        /* a scalar parameter is outside its domain         */
} gg_status;

typedef enum {
    GG_BF16 = 0,
    GG_F16 = 1,
    GG_F32 = 2,
    GG_F8E4M3 = 3,           /* OCP E4M3 ("float8_e4m3fn"): max 448, no inf     */
    GG_F8E5M2 = 4,           /* OCP E5M2 ("float8_e5m2"): max 57344, inf / NaN  */
    GG_MXFP4 = 5             /* OCP E2M1 codes, two a byte, with E8M0 scales: the
                                weights of gg_moe_few                           */
} gg_dtype;

typedef enum {
    GG_MAJOR_K = 0,          /* the reduction axis is contiguous                  */
    GG_MAJOR_M = 1,          /* the M axis (rows of the product) is contiguous    */
    GG_MAJOR_N = 2           /* the N axis (columns of the product) is contiguous */
} gg_major;

/* GG_DSITUGLU is defined for the block-scaled contract only (gg_dglu_mx). */
typedef enum { GG_DSWIGLU = 0, GG_DGEGLU = 1, GG_DSITUGLU = 2 } gg_act;

/* What gg_route makes of a logit. */
typedef enum { GG_SOFTMAX = 0, GG_SIGMOID = 1 } gg_score;

enum {
    /* dGLU: in each 64-column pair of C and D the gate block comes first.
     * Default (flag clear): the input block comes first, as the dGLU page's
     * "interleaved input/gate" C and its interleave of [dinput, dgate] say. */
    GG_FLAG_GATE_FIRST = 1u,
    /* dGeGLU: use 0/1 indicator filters (the derivative of the clamped
     * activation) instead of the page's value-bearing filters, which carry
     * the raw gate / input value inside the clamp range. */
    GG_FLAG_GEGLU_MASK_FILTER = 2u,
    /* Copy offsets / padded_offsets to the host, wait for `stream`, and
     * return GG_ERR_OFFSETS unless they are non-decreasing, every group is a
     * multiple of 256, and the last value equals tokens_sum (wgrad) or is at
     * most m_rows (dgrad).  Off by default: it synchronises the stream. */
    GG_FLAG_VALIDATE_OFFSETS = 4u,
    /* wgrad: K-major operands are stored "tensor_ragged" (the wgrad page's
     * input_order): expert e's (rows, count_e) block is K-contiguous, with
     * row pitch count_e, and the blocks are concatenated in expert order, so
     * that block e starts at element rows * offsets[e-1] (0 for e = 0).
     * M-/N-major operands hold each token contiguously either way, so the
     * flag leaves them as they are. */
    GG_FLAG_TENSOR_RAGGED = 8u,
    /* Static scheduling (the pages' use_dynamic_sched=False, dGLU page
     * "Class API").  The persistent bf16 wgrad kernel then walks its items in
     * a fixed order -- workgroup j of an XCD's W workgroups takes that XCD's
     * items j, j + W, j + 2W, ... -- instead of taking them from the XCD's
     * atomic work queue in finish order.  The results are identical.  The
     * other kernels launch one workgroup per tile, dispatched by the
     * hardware in a fixed order, so for them both settings are the same
     * schedule and the flag is accepted with no effect. */
    GG_FLAG_STATIC_SCHED = 16u,
    /* Block-scaled entries (gg_wgrad_mx, gg_dglu_mx, gg_dsrelu): the FP8
     * codes of A and B are E5M2 rather than E4M3 -- the other MXFP8 ab_dtype
     * of the dGLU page's "Data Types" table; A and B always share one format
     * ("Additional Type Constraints").  The dgrad entries take it with an
     * FP8 d_dtype only (the same section pairs FP8 operands with FP8
     * outputs), else GG_ERR_UNSUPPORTED; gg_wgrad_mx with any wgrad_dtype. */
    GG_FLAG_AB_E5M2 = 32u,
    /* gg_route, gg_route_bwd: the chosen experts' weights are divided by
     * their sum. */
    GG_FLAG_NORMALIZE = 64u
};

/*
 * FP8 outputs of the block-scaled dgrad entries (gg_dglu_mx, gg_dsrelu) when
 * d_dtype is GG_F8E4M3 or GG_F8E5M2 ("Grouped GEMM + dGLU (SM100)",
 * "Block-scaled contract / Equations", step 3, and its "Data Types" d_dtype
 * column; the dsReLU page's FP8 D_row / D_col with SFD_row / SFD_col).  W is
 * the width of D (2n for dGLU, n for dsReLU).  Blocks of 32 values -- 32
 * columns of a row for d_row, 32 rows of a column for d_col -- share one
 * E8M0 scale SFD = 2^e, e the smallest integer with
 *   2^e >= fp32(fp32(norm_const * max|D|) * fp32(1/fmax))
 * fmax the format's largest value (448 for E4M3, 57344 for E5M2; the page's
 * norm_const * max|D| * rcp_max, rounded up to a power of two, which keeps
 * every code within fmax; e in [-127, 127], -127 for an all-zero block), and
 * each value is stored as fp8(D * norm_const / 2^e), clamped to +-fmax,
 * round to nearest even.  D here is the fp32 result before any rounding;
 * d_row and d_col share the one format.
 * A plain layout replaces the pages' MMA-interleaved scale tensors; the
 * column scales of one group occupy its own row-block range of every column
 * (groups are multiples of 256 rows, so no block straddles two).
 */
typedef struct {
    void* d_col;               /* (m_rows, W) FP8 column-quantized D, row-major, 16-B
                                  aligned; or NULL for no column output             */
    uint8_t* sfd_row;          /* (m_rows, W/32): row m, block b at m*(W/32) + b      */
    uint8_t* sfd_col;          /* (W, P), P = ceil(m_rows/32): column c, rows 32j ..
                                  32j+31 at c*P + j; NULL exactly when d_col is NULL */
    const float* norm_const;   /* float[1], device memory                              */
} gg_fp8_out;

/* Bits of the device error word (see gg_device_error). */
enum {
    GG_DEVERR_DECREASING = 1,   /* an offset is smaller than its predecessor   */
    GG_DEVERR_GRANULE = 2,      /* a group size is not a multiple of 256       */
    GG_DEVERR_LAST = 4,         /* last offset != tokens_sum / > m_rows        */
    GG_DEVERR_SKIPPED = 8,      /* a group was too malformed to compute        */
    GG_DEVERR_IDS = 16          /* gg_plan: an id outside -1 .. E-1, or twice
                                   in its token                                */
};

/* ABI version of the loaded library (GG_ABI_VERSION of its build).  It changes
 * when a call or a structure that was there does; a call that has come since
 * is found by its name. */
int gg_abi_version(void);

/* Message for the last non-GG_OK status returned on this thread ("" if
 * none).  Valid until the next gg_* call on the same thread. */
const char* gg_last_error(void);

/* Waits for `stream`, then stores into *code [host] the device error word
 * that the last call using `workspace` left (0 = no violation; otherwise an
 * OR of GG_DEVERR_*).  The word is cleared by the next call on the
 * workspace. */
gg_status gg_device_error(const void* workspace, void* stream, int32_t* code);

/* ------------------------------------------------------------------------ */
/* Grouped wgrad                                                             */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_wgrad needs for num_experts experts. */
size_t gg_wgrad_workspace_size(int32_t num_experts);

/*
 * Wgrad[e] = A[:, begin:end] @ B[begin:end, :] for every expert e, with
 * begin = 0 for e = 0, begin = offsets[e-1] otherwise, end = offsets[e]
 * ("Grouped GEMM + WGrad (Unified)", "Operation"); fp32 accumulation.
 *
 * a          A, logical shape (hidden, tokens_sum), bf16 ("BF16 contract"):
 *              a_major GG_MAJOR_K: element (h,t) at a[h*tokens_sum + t]
 *              a_major GG_MAJOR_M: element (h,t) at a[t*hidden + h]
 * b          B, logical shape (tokens_sum, intermediate), bf16:
 *              b_major GG_MAJOR_K: element (t,i) at b[i*tokens_sum + t]
 *              b_major GG_MAJOR_N: element (t,i) at b[t*intermediate + i]
 * offsets    int32[num_experts], non-decreasing cumulative token ends; every
 *            count a multiple of 256 and offsets[E-1] == tokens_sum ("BF16
 *            contract").  Counts that are multiples of 8 but not of 256 are
 *            computed exactly and flagged (GG_DEVERR_GRANULE); a group whose
 *            bounds are not multiples of 8 is skipped (GG_DEVERR_SKIPPED).
 * num_experts 1..1024.  tokens_sum >= 0, a multiple of 8.
 * hidden, intermediate  multiples of 64, >= 64; at most 2^28 output tiles
 *            of 256 x 256 over all experts (GG_ERR_UNSUPPORTED beyond).
 * Output, exactly one of ("Output modes"):
 * wgrad_dense  (num_experts, hidden, intermediate) row-major, or NULL;
 * wgrad_ptrs   int64[num_experts] device array of 16-B-aligned, non-NULL
 *              addresses, one (hidden, intermediate) row-major matrix per
 *              expert; or NULL.
 * wgrad_dtype  GG_BF16, GG_F16 or GG_F32.
 * accumulate   nonzero: out = round(old + result) (the caller initialises
 *              every output); zero: out = round(result), an empty expert
 *              gives exact zeros.  Rounding is to nearest even.
 * flags        OR of GG_FLAG_VALIDATE_OFFSETS, GG_FLAG_TENSOR_RAGGED
 *              ("input_order": the K-major operands' storage, see the flag)
 *              and GG_FLAG_STATIC_SCHED.
 * workspace    >= gg_wgrad_workspace_size(num_experts) bytes, 256-B aligned.
 *              Besides the error word and the experts' rank table it holds the
 *              work-queue counters of the kernel's scheduler, reset by every
 *              call; calls that may overlap must not share it.
 */
gg_status gg_wgrad(const void* a, gg_major a_major, const void* b, gg_major b_major,
                   const int32_t* offsets, int32_t num_experts, int64_t tokens_sum,
                   int32_t hidden, int32_t intermediate,
                   void* wgrad_dense, const int64_t* wgrad_ptrs, gg_dtype wgrad_dtype,
                   int32_t accumulate, uint32_t flags,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * gg_wgrad without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Every argument has gg_wgrad's meaning;
 * the scratch the kernels use (error word, work-queue counters, expert
 * rank table) is a static array of 16640 bytes inside the library, one per
 * GPU, held until the process ends, which limits num_experts to 1024 (beyond:
 * GG_ERR_WORKSPACE; gg_wgrad's own limit is the same).  No path of the call
 * allocates memory, host or device.
 *   - All calls on one GPU share that GPU's scratch: calls that may overlap
 *     on one GPU (different streams, or host threads) race and must not be
 *     issued.  Each call clears what it needs before its kernels run.
 *   - The device error word lives in that scratch and is not readable by
 *     the caller; use GG_FLAG_VALIDATE_OFFSETS to have malformed offsets
 *     rejected (GG_ERR_OFFSETS), or gg_wgrad with a workspace to read it.
 */
gg_status gg_wgrad_noalloc(const void* a, gg_major a_major, const void* b, gg_major b_major,
                           const int32_t* offsets, int32_t num_experts, int64_t tokens_sum,
                           int32_t hidden, int32_t intermediate,
                           void* wgrad_dense, const int64_t* wgrad_ptrs, gg_dtype wgrad_dtype,
                           int32_t accumulate, uint32_t flags, void* stream);

/*
 * The same operation on block-scaled operands ("Grouped GEMM + WGrad
 * (Unified)", "Block-scaled contract"), MXFP8: E4M3 codes (E5M2 with
 * GG_FLAG_AB_E5M2) with one E8M0 scale per 32 consecutive tokens of a row,
 * deq(q, s) = fp8(q) * 2^(s-127), fp32 accumulation.  The reduction axis is
 * contiguous in both operands:
 * a_fp8      A (hidden, tokens_sum) K-major: (h,t) at a[h*tokens_sum + t];
 * sfa        (hidden, tokens_sum/32): sfa[h*(tokens_sum/32) + t/32];
 * b_fp8      B (tokens_sum, intermediate) stored K-major, as an
 *            (intermediate, tokens_sum) array: (t,i) at b[i*tokens_sum + t];
 * sfb        (intermediate, tokens_sum/32): sfb[i*(tokens_sum/32) + t/32].
 *            With GG_FLAG_TENSOR_RAGGED all four hold per-expert blocks
 *            instead: expert e's codes at a[hidden*begin + h*count + t-begin]
 *            and scales at sfa[(hidden*begin + h*count + t-begin)/32]
 *            (likewise b, sfb with intermediate).
 * tokens_sum a multiple of 128, as is every expert's count (the pages ask
 *            for 256; a count that is not a multiple of 128 is skipped and
 *            flagged GG_DEVERR_SKIPPED, one of 128 but not 256 computed and
 *            flagged GG_DEVERR_GRANULE).
 * flags      as for gg_wgrad, and GG_FLAG_AB_E5M2.
 * Codes 16-byte, scales 4-byte aligned.  Every other argument as for
 * gg_wgrad; the pages' global scales belong to formats other than MXFP8 and
 * are not taken.
 */
gg_status gg_wgrad_mx(const void* a_fp8, const uint8_t* sfa, const void* b_fp8, const uint8_t* sfb,
                      const int32_t* offsets, int32_t num_experts, int64_t tokens_sum,
                      int32_t hidden, int32_t intermediate,
                      void* wgrad_dense, const int64_t* wgrad_ptrs, gg_dtype wgrad_dtype,
                      int32_t accumulate, uint32_t flags,
                      void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Grouped dgrad + dSwiGLU / dGeGLU                                          */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_dglu needs for L experts and compact width n. */
size_t gg_dglu_workspace_size(int32_t L, int32_t n, int32_t generate_dbias);

/*
 * For the rows m of group g (po[g-1] <= m < po[g], po[-1] = 0) and compact
 * columns n ("Grouped GEMM + dGLU (SM100)", "BF16 contract"):
 *   R[m,n] = alpha_g^2 * sum_k A[m,k] B_g[n,k]          (fp32 accumulation)
 *   X = beta_g * C[m,:]  (one fp32 product per element)
 *   compact column n lies in block pair p = n/32 at j = n%32; its input
 *   column is 64p + j and its gate column 64p + 32 + j (GG_FLAG_GATE_FIRST
 *   swaps them).
 *   dSwiGLU, s = sigmoid(gate):
 *     D[input] = R prob gate s
 *     D[gate]  = R prob input s (1 + gate (1 - s))
 *     dprob   += R gate s input
 *   dGeGLU, gc = min(gate, clamp_max), uc = clamp(input, clamp_min,
 *   clamp_max), s = sigmoid(geglu_alpha gc), filters
 *   fg = gate if gate <= clamp_max else 0, fu = input if clamp_min <= input
 *   <= clamp_max else 0 (1 instead of the raw value with
 *   GG_FLAG_GEGLU_MASK_FILTER):
 *     D[gate]  = R prob (uc + linear_offset) s (1 + geglu_alpha gc (1 - s)) fg
 *     D[input] = R prob gc s fu
 *     dprob   += R gc s (uc + linear_offset)
 *   dbias[g, c] += sum over the group's rows of D[m, c] (before rounding).
 *
 * a          A (m_rows, k) bf16, K-major: a[m*k + kk].
 * m_rows     rows of A, C, D, prob, dprob; >= valid_m = padded_offsets[L-1].
 *            Rows at or past valid_m are neither read for output nor written.
 * k          reduction size, a multiple of 64, at most 2^21.
 * b_dense    dense weights, the pages' (N, K, L) tensor with strides
 *            (K, 1, N*K): expert g's (n, k) element at b[g*n*k + n*k + kk].
 * b_ptrs     or: int64[L] device array, expert g's (n, k) bf16 matrix at
 *            b_ptrs[g]; K-major (element at n*k + kk) when b_major is
 *            GG_MAJOR_K, N-major (element at kk*n + nn) when GG_MAJOR_N.
 *            Exactly one of b_dense / b_ptrs is non-NULL; b_dense requires
 *            GG_MAJOR_K.
 * n          compact gradient width N, a multiple of 32, at most 2^20
 *            (GG_ERR_UNSUPPORTED beyond either limit).
 * c          forward activation (m_rows, 2n), row-major, dtype c_dtype
 *            (GG_BF16, GG_F16 or GG_F32).
 * padded_offsets  int32[L] cumulative group ends, each group a multiple of
 *            256 (m_aligned).  L in 1..1024.
 * alpha, beta  float[L];  prob  float[m_rows].
 * d_row      output (m_rows, 2n), row-major, d_dtype (GG_BF16, GG_F16 or
 *            GG_F32), rounded to nearest even.
 * dprob      float[m_rows], caller-zeroed, accumulated into ("must be
 *            zero-initialized").
 * dbias      bf16 (L, 2n) row-major, caller-zeroed and accumulated into
 *            (one rounding of old + sum), or NULL for no dbias.
 * act        GG_DSWIGLU or GG_DGEGLU; geglu_alpha, clamp_min, clamp_max,
 *            linear_offset are the dGeGLU constants (the pages' defaults:
 *            1.702, -7, 7, 1); ignored for dSwiGLU.
 * flags      OR of GG_FLAG_GATE_FIRST, GG_FLAG_GEGLU_MASK_FILTER,
 *            GG_FLAG_VALIDATE_OFFSETS, GG_FLAG_STATIC_SCHED.
 * workspace  >= gg_dglu_workspace_size(L, n, dbias != NULL), 256-B aligned.
 */
gg_status gg_dglu(const void* a, int64_t m_rows, int32_t k,
                  const void* b_dense, const int64_t* b_ptrs, gg_major b_major, int32_t n,
                  const void* c, gg_dtype c_dtype,
                  const int32_t* padded_offsets, int32_t L,
                  const float* alpha, const float* beta, const float* prob,
                  void* d_row, gg_dtype d_dtype, float* dprob, void* dbias,
                  gg_act act, float geglu_alpha, float clamp_min, float clamp_max,
                  float linear_offset, uint32_t flags,
                  void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Grouped dgrad + dSwiGLU / dGeGLU on MXFP8 operands                        */
/* ------------------------------------------------------------------------ */

/*
 * For the rows m of group g ("Grouped GEMM + dGLU (SM100)", "Block-scaled
 * contract / Equations"):
 *   R[m,n] = alpha_g^2 * sum_k deq(A[m,k]) deq(B_g[n,k])   (fp32 accumulation)
 * with deq(q, s) = e4m3(q) * 2^(s - 127), one E8M0 scale byte per 32
 * consecutive K values of a row (MXFP8: "sf_vec_size 32" in the page's
 * data-type table), followed by exactly the dSwiGLU / dGeGLU, dprob and dbias
 * steps documented for gg_dglu.  In addition ("Shapes": amax (L, 2, 1) for
 * a bf16 / fp16 D):
 *   amax[2g + 0] = max |D| over the group's input-gradient columns,
 *   amax[2g + 1] = max |D| over its gate-gradient columns,
 * taken before rounding (0 for an empty group).
 *
 * a_fp8      A (m_rows, k) FP8 codes (E4M3, or E5M2 with GG_FLAG_AB_E5M2),
 *            K-major: a[m*k + kk].
 * sfa        E8M0 scales (m_rows, k/32), row-major: sfa[m*(k/32) + kk/32]
 *            (a plain layout; the pages' MMA-interleaved scale layout is not
 *            used).
 * m_rows     as for gg_dglu.  k: a multiple of 128, at most 2^21.
 * b_fp8,sfb  dense weights (L, n, k) FP8 (A's format), element at
 *            b[g*n*k + nn*k + kk] (GG_MAJOR_K) or b[g*n*k + kk*n + nn]
 *            (GG_MAJOR_N), and scales (L, n, k/32) at
 *            sfb[(g*n + nn)*(k/32) + kk/32] for either major;
 * b_ptrs, sfb_ptrs  or: int64[L] device arrays of per-expert (n, k) codes
 *            and (n, k/32) scales with the same in-matrix layout (the page's
 *            discrete b_ptrs / sfb_ptrs).  Exactly one of the dense pair /
 *            the pointer pair is given.
 * b_major    GG_MAJOR_K or GG_MAJOR_N ("Parameters / Input tensor B (dense
 *            mode)": K-major or N-major), for dense and discrete B alike;
 *            else GG_ERR_LAYOUT.
 * n          compact width, a multiple of 32, at most 2^20
 *            (GG_ERR_UNSUPPORTED beyond either limit).
 * c_dtype    as for gg_dglu, or GG_F8E4M3 / GG_F8E5M2 (the dGLU page's
 *            "Input tensor C" dtypes): an FP8 C is read as its exact value.
 * c, padded_offsets, L, alpha, beta, prob, d_row, dprob, dbias, geglu_alpha,
 * clamp_min, clamp_max, linear_offset
 *            as for gg_dglu.
 * act        GG_DSWIGLU, GG_DGEGLU, or GG_DSITUGLU: the page's dSiTU-GLU
 *            ("Block-scaled contract / Equations") on gate G and input U of
 *            X = beta_g C, b1 = situ_beta1, b2 = situ_beta2 (the page's
 *            defaults: 4 and 25; both positive and finite, else
 *            GG_ERR_VALUE; ignored for the other activations):
 *              T_g = b1 tanh(G/b1) sigmoid(G),   T_u = b2 tanh(U/b2)
 *              D[gate]  = R prob T_u ((1 - tanh^2(G/b1)) sigmoid(G)
 *                         + b1 tanh(G/b1) sigmoid(G) (1 - sigmoid(G)))
 *              D[input] = R prob T_g (1 - tanh^2(U/b2))
 *              dprob   += R T_g T_u
 * amax       float[2L] ((L, 2) row-major), written by the call (the library
 *            clears it first), or NULL.
 * d_dtype    as for gg_dglu, or GG_F8E4M3 / GG_F8E5M2: d_row then holds
 *            the row-quantized FP8 D ((m_rows, 2n), 16-B aligned) and
 *            fp8_out [host] the rest of the FP8 output (see gg_fp8_out);
 *            fp8_out is ignored for the other dtypes.
 * flags      as for gg_dglu, and GG_FLAG_AB_E5M2 (with an FP8 d_dtype).
 * workspace  >= gg_dglu_workspace_size(L, n, dbias != NULL), 256-B aligned.
 */
gg_status gg_dglu_mx(const void* a_fp8, const uint8_t* sfa, int64_t m_rows, int32_t k,
                     const void* b_fp8, const uint8_t* sfb,
                     const int64_t* b_ptrs, const int64_t* sfb_ptrs, gg_major b_major, int32_t n,
                     const void* c, gg_dtype c_dtype,
                     const int32_t* padded_offsets, int32_t L,
                     const float* alpha, const float* beta, const float* prob,
                     void* d_row, gg_dtype d_dtype, float* dprob, void* dbias, float* amax,
                     const gg_fp8_out* fp8_out, gg_act act, float geglu_alpha, float clamp_min, float clamp_max,
                     float linear_offset, float situ_beta1, float situ_beta2, uint32_t flags,
                     void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Grouped dgrad + dsReLU on MXFP8 operands                                  */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_dsrelu needs for L experts. */
size_t gg_dsrelu_workspace_size(int32_t L);

/*
 * For the rows m of group g ("Grouped GEMM + dsReLU (SM100)", "Equations"):
 *   G[m,n]     = alpha_g * sum_k deq(A[m,k]) deq(B_g[n,k])   (fp32 accumulation)
 *   D_row[m,n] = prob[m] * 2 * C[m,n] * relu(G[m,n])
 *   dprob[m]  += sum_n C[m,n] * relu(G[m,n])^2
 *   amax[g]    = max |D_row| over the group, before rounding (0 if empty)
 * with deq(q, s) = fp8(q) * 2^(s - 127): MXFP8, one E8M0 scale byte per 32
 * consecutive K values of a row ("sf_vec_size 32" for MXFP8 on the dGLU
 * page's data-type table), the codes E4M3, or E5M2 with GG_FLAG_AB_E5M2 (A
 * and B alike).
 *
 * a_fp8      A (m_rows, k) FP8 codes, K-major: a[m*k + kk].
 * sfa        E8M0 scales (m_rows, k/32), row-major: sfa[m*(k/32) + kk/32].
 *            (A plain row-major layout; the pages' 6-D MMA-interleaved scale
 *            layout is not used.)
 * m_rows     as for gg_dglu.  k: a multiple of 128, at most 2^21.
 * b_fp8,sfb  dense weights (L, n, k) FP8 (A's format), element at
 *            b[g*n*k + nn*k + kk] (GG_MAJOR_K) or b[g*n*k + kk*n + nn]
 *            (GG_MAJOR_N), and scales (L, n, k/32) at
 *            sfb[(g*n + nn)*(k/32) + kk/32] for either major;
 * b_ptrs, sfb_ptrs  or: int64[L] device arrays of per-expert (n, k) codes
 *            and (n, k/32) scales with the same in-matrix layout.
 *            Exactly one of the dense pair / the pointer pair is given.
 * b_major    GG_MAJOR_K or GG_MAJOR_N (the page's "Layouts" allow an
 *            N-major B for FP8 operands), else GG_ERR_LAYOUT.
 * n          a multiple of 32, at most 2^21 (GG_ERR_UNSUPPORTED beyond either
 *            limit).
 * c          (m_rows, n) row-major, c_dtype GG_BF16, GG_F16, GG_F32,
 *            GG_F8E4M3 or GG_F8E5M2 (the dsReLU page's "Input tensor C"
 *            dtypes; an FP8 C is read as its exact value).
 * padded_offsets, L  as for gg_dglu.
 * alpha      float[L];  prob  float[m_rows].
 * d_row      (m_rows, n) row-major, d_dtype GG_BF16, GG_F16 or GG_F32; or
 *            GG_F8E4M3 / GG_F8E5M2, the row-quantized D, with fp8_out [host]
 *            giving the rest of the FP8 output (see gg_fp8_out; ignored
 *            otherwise).
 * dprob      float[m_rows], caller-zeroed, accumulated into.
 * amax       float[L], written by the call (the library clears it first), or
 *            NULL.
 * flags      OR of GG_FLAG_VALIDATE_OFFSETS, GG_FLAG_STATIC_SCHED and
 *            GG_FLAG_AB_E5M2 (with an FP8 d_dtype).
 * workspace  >= gg_dsrelu_workspace_size(L), 256-B aligned.
 */
gg_status gg_dsrelu(const void* a_fp8, const uint8_t* sfa, int64_t m_rows, int32_t k,
                    const void* b_fp8, const uint8_t* sfb,
                    const int64_t* b_ptrs, const int64_t* sfb_ptrs, gg_major b_major, int32_t n,
                    const void* c, gg_dtype c_dtype,
                    const int32_t* padded_offsets, int32_t L,
                    const float* alpha, const float* prob,
                    void* d_row, gg_dtype d_dtype, float* dprob, float* amax,
                    const gg_fp8_out* fp8_out, uint32_t flags,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* The router                                                                */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_route needs. */
size_t gg_route_workspace_size(int64_t tokens, int32_t num_experts);

/*
 * The choice of experts, their weights, tokens per expert and the balance
 * loss.  Per token t, with x its logits:
 *   key_e   = x_e + bias_e                     (one fp32 addition; with
 *             GG_SIGMOID too the bias is on the logit, not on the score:
 *             sigmoid(x_e) + bias_e is another order, which this call does
 *             not have)
 *   ids     = the top_k experts of the largest keys, largest first, ties to
 *             the lower index.  -0 and +0 are equal; a NaN of either sign is
 *             above +inf.  A logit, bias or key of -inf is never chosen:
 *             where fewer than top_k experts are left, the rest of ids is -1
 *             and of prob 0.
 *   scores  = softmax(x) over all experts (GG_SOFTMAX) or sigmoid(x)
 *             (GG_SIGMOID), without the bias
 *   prob    = scale * score of the chosen; with GG_FLAG_NORMALIZE
 *             scale * softmax over the chosen experts' logits (GG_SOFTMAX),
 *             scale * s / (sum of the chosen s + 1e-20) (GG_SIGMOID)
 *   counts_e = tokens that chose e;  N = routed = tokens with a choice
 *   balance = num_experts * sum_e (counts_e / (top_k N)) (1/N) sum_t p_te,
 *             over the N tokens, p the softmax, or s / (sum over all experts
 *             of s + 1e-20); 0 if N is 0
 * A NaN or +inf logit makes NaN of what the formulas say it enters.
 * fp32 arithmetic: a weight is good to some 16 units of 2^-24 of itself at
 * logits of any size (softmax: besides the rounding of x minus the largest).
 * The loss's probabilities are off by up to |x| units each and added up in
 * fp32 within a block, in fp64 over the blocks, in an order that depends on
 * the sizes alone, so equal calls give equal bits.
 *
 * logits     (tokens, num_experts), dtype GG_BF16, GG_F16 or GG_F32, element
 *            (t, e) at logits[t*ld + e], ld >= num_experts; aligned to its
 *            element.
 * tokens     0 .. 2^23.  num_experts 1..1024.
 * bias       float[num_experts], or NULL for none; +inf and NaN count as the
 *            largest finite value.
 * top_k      1 .. min(32, num_experts).  scale: finite.
 * ids, prob  (tokens, top_k) int32 / float outputs.
 * counts     int32[num_experts], routed int32[1]: outputs.
 * balance    float[1] output, or NULL: the loss is not computed.
 * flags      0 or GG_FLAG_NORMALIZE.
 * workspace  >= gg_route_workspace_size(tokens, num_experts), 256-B aligned.
 */
gg_status gg_route(const void* logits, gg_dtype dtype, int64_t ld, int64_t tokens,
                   int32_t num_experts, const float* bias, int32_t top_k, gg_score score,
                   float scale, uint32_t flags, int32_t* ids, float* prob, int32_t* counts,
                   int32_t* routed, float* balance,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * The gradient of gg_route's logits:
 *   dlogits = d/dlogits (sum_tj dprob_tj prob_tj + dbalance balance)
 * at the choice `ids` (the choice and the counts have no gradient).  Rows of
 * a token without a choice are 0.  A NaN or +inf logit that was not chosen
 * enters where the formulas have all experts: the balance loss, and GG_SOFTMAX
 * without GG_FLAG_NORMALIZE.
 *
 * logits, dtype, ld, tokens, num_experts, top_k, score, scale, flags, ids,
 * counts, routed   as given to and made by gg_route.  An id outside
 *            0 .. num_experts-1 is no choice; the ids of a token differ.
 * dprob      float (tokens, top_k) if row_of is NULL; otherwise float[m_rows],
 *            the gradient by expert row that gg_dglu and gg_dsrelu write, and
 *            choice (t, j) takes dprob[row_of[t*top_k + j]]: 0 where row_of
 *            is outside 0 .. m_rows-1 (a dropped choice).
 * dbalance   float[1] in device memory, or NULL for no balance loss.
 * dlogits    output (tokens, num_experts), dtype, contiguous, not
 *            overlapping logits; aligned to its element; fp32 arithmetic,
 *            rounded once (exponentials as in gg_route's weights for GG_F32,
 *            as in its loss for the 16-bit types).
 */
gg_status gg_route_bwd(const void* logits, gg_dtype dtype, int64_t ld, int64_t tokens,
                       int32_t num_experts, int32_t top_k, gg_score score, float scale,
                       uint32_t flags, const int32_t* ids, const int32_t* counts,
                       const int32_t* routed, const float* dprob, const int32_t* row_of,
                       int64_t m_rows, const float* dbalance, void* dlogits, void* stream);

/* ------------------------------------------------------------------------ */
/* Dispatch to the expert-sorted rows, and back                              */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_plan needs. */
size_t gg_plan_workspace_size(int64_t tokens, int32_t num_experts);

/* The most rows that gg_plan can need, whatever the ids are: with n = tokens
 * * top_k, n + (granule-1) * min(num_experts, n) down to a multiple of
 * granule.  0 for arguments out of gg_plan's ranges. */
int64_t gg_plan_max_rows(int64_t tokens, int32_t top_k, int32_t num_experts, int32_t granule);

/*
 * The rows of every token's choices in the layout the grouped GEMMs take:
 * expert after expert, tokens in order within an expert, every group padded
 * to a multiple of `granule` rows (256 for this library's GEMMs).
 *   counts_e  = tokens that chose e
 *   padded_offsets_e = sum of the padded counts of experts 0 .. e
 *   row_of[t, j] = padded_offsets_{e-1} + number of tokens t' < t that chose
 *                  e = ids[t, j]; -1 where there is no row
 *   prob_rows[row_of[t, j]] = prob[t, j], 0 in the padding
 * An id of -1 has no row; nor has one outside -1 .. num_experts-1 or a
 * second use of an expert by a token, which set GG_DEVERR_IDS.  Groups are
 * cut off at m_rows (down to a multiple of granule): choices past it have
 * no row, counts and padded_offsets hold what is left, GG_DEVERR_LAST is set.
 *
 * ids        (tokens, top_k) int32; tokens 0 .. 2^23, top_k 1..32,
 *            num_experts 1..1024, granule a power of two in 1..256.
 * m_rows     rows there is room for, 0 .. 2^31-1; gg_plan_max_rows suffices.
 * prob       (tokens, top_k) float and prob_rows float[m_rows], or both NULL.
 *            Rows at or past padded_offsets[E-1] are not written.
 * counts, padded_offsets  int32[num_experts], row_of (tokens, top_k) int32:
 *            outputs.
 * workspace  >= gg_plan_workspace_size(tokens, num_experts), 256-B aligned;
 *            its error word is read with gg_device_error.
 */
gg_status gg_plan(const int32_t* ids, int64_t tokens, int32_t top_k, int32_t num_experts,
                  int32_t granule, int64_t m_rows, const float* prob, int32_t* counts,
                  int32_t* padded_offsets, int32_t* row_of, float* prob_rows,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * x_rows[row_of[t, j], :] = x[t, :] for every choice with a row (row_of
 * within 0 .. m_rows-1), and zeros in every group's padding rows,
 * padded_offsets[e-1] + counts[e] .. padded_offsets[e]-1.  Copies: any value
 * keeps its bits.
 *
 * x          (tokens, width), element (t, c) at x[t*ldx + c], ldx >= width;
 *            GG_BF16, GG_F16, GG_F32, GG_F8E4M3 or GG_F8E5M2 (rows of bytes:
 *            the E8M0 scales of MXFP8 rows too), aligned to its element.
 * width      1 .. 2^20.
 * row_of, counts, padded_offsets  as made by gg_plan.
 * x_rows     output (m_rows, width), contiguous; other rows are not written.
 * The gradient of x is gg_combine of x_rows' gradient with no weights.
 */
gg_status gg_permute(const void* x, gg_dtype dtype, int64_t ldx, int64_t tokens, int32_t width,
                     const int32_t* row_of, int32_t top_k, const int32_t* counts,
                     const int32_t* padded_offsets, int32_t num_experts, int64_t m_rows,
                     void* x_rows, void* stream);

/*
 * out[t, :] = sum_j weights[t, j] * y_rows[row_of[t, j], :] over the choices
 * with a row, in fp32 in the order of j, rounded once; 0 for a token with
 * none.
 *
 * y_rows     (m_rows, width) contiguous, GG_BF16, GG_F16 or GG_F32.
 * weights    (tokens, top_k) float, or NULL for 1.
 * out        (tokens, width), y_rows' dtype, element (t, c) at out[t*ldo + c].
 */
gg_status gg_combine(const void* y_rows, gg_dtype dtype, int64_t m_rows, int32_t width,
                     const int32_t* row_of, int64_t tokens, int32_t top_k, const float* weights,
                     void* out, int64_t ldo, void* stream);

/*
 * The gradients of gg_combine:
 *   dy_rows[row_of[t, j], :] = weights[t, j] * dout[t, :]  (rounded once;
 *                              zeros in the padding rows, as gg_permute)
 *   dweights[t, j] = sum_c dout[t, c] * y_rows[row_of[t, j], c]   (fp32; 0
 *                              for a choice without a row)
 * dout (tokens, width) with row pitch ldd; y_rows, dy_rows (m_rows, width)
 * contiguous, not overlapping; all of one dtype.  weights, dweights
 * (tokens, top_k) float.
 */
gg_status gg_combine_bwd(const void* dout, gg_dtype dtype, int64_t ldd, int64_t tokens,
                         int32_t width, const void* y_rows, int64_t m_rows, const float* weights,
                         const int32_t* row_of, int32_t top_k, const int32_t* counts,
                         const int32_t* padded_offsets, int32_t num_experts, void* dy_rows,
                         float* dweights, void* stream);

/* ------------------------------------------------------------------------ */
/* Gradient norm and clipping                                                */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_grad_norm needs. */
size_t gg_grad_workspace_size(void);

/*
 * sumsq = (accumulate ? sumsq : 0) + sum of the squares of every element of
 * n tensors, in fp64, in an order that depends on the sizes alone.
 *
 * ptrs       int64[n] device array: the tensors' addresses, aligned to their
 *            elements; not read for an empty tensor.
 * ends       int64[n] device array: cumulative element counts (tensor i has
 *            ends[i] - ends[i-1] elements), non-decreasing.
 * dtypes     int32[n] device array: GG_BF16, GG_F16 or GG_F32 each (a tensor
 *            of any other value is left out).
 * n          0 .. 2^24.  total: elements of all tensors, ends[n-1] [host],
 *            up to 2^40; elements past it are left out.
 * sumsq      double[1], device memory, 8-byte aligned: ranks that share the
 *            parameters add theirs up before gg_grad_clip.
 * workspace  >= gg_grad_workspace_size() bytes, 256-B aligned.
 */
gg_status gg_grad_norm(const int64_t* ptrs, const int64_t* ends, const int32_t* dtypes, int32_t n,
                       int64_t total, double* sumsq, int32_t accumulate,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * norm   = sqrt(sumsq)
 * factor = min(1, max_norm / (norm + eps))    (1 if max_norm >= norm + eps,
 *          whatever the quotient; NaN if norm is NaN, and only then)
 * every element g becomes g * factor (one fp32 product, rounded once to its
 * type).
 *
 * ptrs, ends, dtypes, n, total  as for gg_grad_norm.
 * sumsq      double[1], device memory.
 * max_norm   >= 0 and not NaN; eps >= 0 and finite.
 * norm       float[2] output: norm and factor.
 * out_ptrs   int64[n] device array of the results' addresses, in ptrs' types,
 *            or NULL: in place, and where the factor is exactly 1 nothing is
 *            written.  A result is its own tensor or does not overlap any.
 */
gg_status gg_grad_clip(const int64_t* ptrs, const int64_t* ends, const int32_t* dtypes, int32_t n,
                       int64_t total, const double* sumsq, float max_norm, float eps, float* norm,
                       const int64_t* out_ptrs, void* stream);

/* ------------------------------------------------------------------------ */
/* MXFP4: quantisation                                                       */
/* ------------------------------------------------------------------------ */

/*
 * MXFP4 (OCP Microscaling): blocks of 32 consecutive values of a row, one E2M1
 * code of 4 bits a value -- sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6 for 0 .. 7 --
 * and one E8M0 scale byte s a block: value = code * 2^(s - 127), s = 255: the
 * block is NaN.
 * codes      (rows, width/2): value 2j of a row in the low half of its byte j,
 *            value 2j + 1 in the high half.
 * scales     (rows, width/32).
 *
 * gg_mx4_quant: s - 127 = e is the smallest e >= -127 with max|x| of the block
 * <= 6 * 2^e (-127 for a block of zeros), so that no value is clamped; each
 * code is x / 2^e rounded to the nearest, ties to the even code, keeping the
 * sign of zeros.  A block with a NaN or an infinity has scale 255 and codes 0.
 * (The values' gradient, taken straight through, is the gradient of x.)
 *
 * x          (rows, width), GG_BF16, GG_F16 or GG_F32, element (r, c) at
 *            x[r*ldx + c], ldx >= width; aligned to its element.
 * rows       0 .. 2^30.  width: a multiple of 32, at most 2^20.
 * codes, scales  outputs, contiguous, of any alignment (gg_gemm_mx4 and
 *            gg_moe_few read codes at 16-byte alignment).
 * end        int32[1] in device memory, or NULL: rows at or past *end are
 *            neither read nor written (padded_offsets + E - 1 for a dispatched
 *            batch).
 */
gg_status gg_mx4_quant(const void* x, gg_dtype dtype, int64_t ldx, int64_t rows, int32_t width,
                       uint8_t* codes, uint8_t* scales, const int32_t* end, void* stream);

/*
 * out = the values that codes and scales stand for, rounded once to dtype
 * (bf16 and fp32 hold every one but those past their largest, which become
 * infinities).
 *
 * out        (rows, width), GG_BF16, GG_F16 or GG_F32, element (r, c) at
 *            out[r*ldo + c], ldo >= width; aligned to its element.
 * rows, width, codes, scales, end  as for gg_mx4_quant.
 */
gg_status gg_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t width,
                         void* out, gg_dtype dtype, int64_t ldo, const int32_t* end, void* stream);

/* ------------------------------------------------------------------------ */
/* The gated activation                                                      */
/* ------------------------------------------------------------------------ */

/*
 * The forward pass of what gg_dglu and gg_dglu_mx differentiate (at beta 1):
 * compact column n of a row lies in block pair p = n/32 at j = n%32, its input
 * u in column 64p + j of c and its gate g in 64p + 32 + j (GG_FLAG_GATE_FIRST
 * swaps them).
 *   GG_DSWIGLU   y = prob g sigmoid(g) u
 *   GG_DGEGLU    y = prob gc sigmoid(geglu_alpha gc) (uc + linear_offset),
 *                gc = min(g, clamp_max), uc = clamp(u, clamp_min, clamp_max)
 *   GG_DSITUGLU  y = prob b1 tanh(g/b1) sigmoid(g) b2 tanh(u/b2)
 * fp32 arithmetic, rounded once; a sigmoid below 2^-126 may count as 0.  A NaN
 * gate or input gives NaN.
 *
 * c          (rows, 2n), GG_BF16, GG_F16 or GG_F32, row pitch ldc >= 2n.
 * prob       float[rows], or NULL for 1.
 * rows       0 .. 2^30.  n: a multiple of 32, at most 2^20.
 * y          output (rows, n), GG_BF16, GG_F16 or GG_F32, row pitch ldy >= n.
 * c and y aligned to their elements; no element of y is one of c.
 * act and its constants  as for gg_dglu_mx.
 * flags      0 or GG_FLAG_GATE_FIRST.
 * end        as for gg_mx4_quant.
 */
gg_status gg_glu(const void* c, gg_dtype c_dtype, int64_t ldc, const float* prob, int64_t rows,
                 int32_t n, void* y, gg_dtype y_dtype, int64_t ldy, gg_act act, float geglu_alpha,
                 float clamp_min, float clamp_max, float linear_offset, float situ_beta1,
                 float situ_beta2, uint32_t flags, const int32_t* end, void* stream);

/* ------------------------------------------------------------------------ */
/* The grouped product of MXFP4 rows and weights                             */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_gemm_mx4 needs. */
size_t gg_gemm_mx4_workspace_size(void);

/*
 * For the rows m of group g (offsets[g-1] <= m < offsets[g], offsets[-1] = 0):
 *   d[m, n] = alpha_g * sum_k deq(a[m, k]) deq(b_g[n, k]) + bias[g, n]
 * with MXFP4 operands (above), fp32 accumulation, rounded once to d_dtype.
 *
 * a_fp4, sfa  codes (m_rows, k/2) and scales (m_rows, k/32).
 * k          a multiple of 128, at most 2^21.  n: a multiple of 32, at most
 *            2^21 (GG_ERR_UNSUPPORTED beyond either limit).
 * b_fp4, sfb  dense weights: codes (L, n, k/2), scales (L, n, k/32);
 * b_ptrs, sfb_ptrs  or: int64[L] device arrays of the experts' codes (n, k/2)
 *            and scales (n, k/32).  Exactly one of the two pairs is given.
 * offsets    int32[L] cumulative group ends, non-decreasing, at most m_rows;
 *            groups of any size, empty ones among them (gg_plan's
 *            padded_offsets at any granule).  An end below an earlier one or 0
 *            makes an empty group and sets GG_DEVERR_DECREASING, one past
 *            m_rows is cut off and sets GG_DEVERR_LAST.  L in 1..1024.
 * m_rows     0 .. 2^31-1.  Rows of d at or past the last end are not written.
 *            (m_rows/256 + min(m_rows, L)) * ceil(n/256), the tiles that there
 *            may be, are limited to 2^23 (GG_ERR_UNSUPPORTED).
 * alpha      float[L], or NULL for 1.  bias: float (L, n), or NULL.
 * d          output (m_rows, n) contiguous, GG_BF16, GG_F16 or GG_F32.
 * Codes and d 16-byte, scales, alpha and bias 4-byte aligned.
 * flags      0.
 * workspace  >= gg_gemm_mx4_workspace_size() bytes, 256-B aligned: the error
 *            word, read with gg_device_error.
 */
gg_status gg_gemm_mx4(const uint8_t* a_fp4, const uint8_t* sfa, int64_t m_rows, int32_t k,
                      const uint8_t* b_fp4, const uint8_t* sfb, const int64_t* b_ptrs,
                      const int64_t* sfb_ptrs, int32_t n, const int32_t* offsets, int32_t L,
                      const float* alpha, const float* bias, void* d, gg_dtype d_dtype,
                      uint32_t flags, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* A whole layer for a few tokens                                            */
/* ------------------------------------------------------------------------ */

/* Bytes of workspace gg_moe_few needs (0 for arguments out of its ranges). */
size_t gg_moe_few_workspace_size(int32_t tokens, int32_t top_k, int32_t hidden, int32_t inner);

/*
 * For up to 64 tokens, e = ids[t, j]:
 *   h    = prob[t, j] * act(w1_e x[t] + bias1_e)
 *   y[t] = sum_j (w2_e h + prob[t, j] * bias2_e)
 * act as for gg_glu, on rows of w1 in 32-wide blocks of inputs and gates.  An
 * id outside 0 .. num_experts-1 is no choice (its prob is not used); a token
 * without any gives 0; an expert may be chosen twice by a token.  Products with
 * fp32 accumulation; h is held as the sum of two bf16 values (16 bits), for an
 * fp32 y of three (24 bits; none finer than 2^-133), and the choices are added
 * up in fp32 in a fixed order, so equal calls give equal bits.  Only the chosen
 * experts' weights are read.
 *
 * x          (tokens, hidden) bf16, row pitch ldx >= hidden, a multiple of 8, at
 *            most 2^23.
 * tokens     0 .. 64.  hidden, inner: multiples of 32, at most 2^16.
 *            num_experts 1..1024, top_k 1..32.
 * ids, prob  (tokens, top_k) int32 / float, as made by gg_route.
 * w_dtype    GG_BF16: w1 (num_experts, 2 inner, hidden) and w2 (num_experts,
 *            hidden, inner) row-major, sf1 and sf2 NULL; or GG_MXFP4: codes
 *            (num_experts, 2 inner, hidden/2), (num_experts, hidden, inner/2)
 *            and scales sf1 (num_experts, 2 inner, hidden/32), sf2 (num_experts,
 *            hidden, inner/32).  A value past bf16's largest is an infinity.
 * bias1      float (num_experts, 2 inner), or NULL;  bias2: float
 *            (num_experts, hidden), or NULL.
 * y          output (tokens, hidden), GG_BF16, GG_F16 or GG_F32, row pitch
 *            ldy >= hidden; aligned to its element.
 * x, w1, w2 16-byte, every other array 4-byte aligned (scales: any).
 * act and its constants  as for gg_dglu_mx.  flags: 0 or GG_FLAG_GATE_FIRST.
 * workspace  >= gg_moe_few_workspace_size(...) bytes, 256-B aligned.
 */
gg_status gg_moe_few(const void* x, int64_t ldx, int32_t tokens, int32_t hidden, const int32_t* ids,
                     const float* prob, int32_t top_k, int32_t num_experts, const void* w1,
                     const uint8_t* sf1, const float* bias1, const void* w2, const uint8_t* sf2,
                     const float* bias2, gg_dtype w_dtype, int32_t inner, void* y, gg_dtype y_dtype,
                     int64_t ldy, gg_act act, float geglu_alpha, float clamp_min, float clamp_max,
                     float linear_offset, float situ_beta1, float situ_beta2, uint32_t flags,
                     void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GG_MOE_H */
