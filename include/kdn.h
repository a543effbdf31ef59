/*
 * kdn.h -- C ABI of the MI355X (gfx950) Kalman Delta Network mixer library.
 *
 * The library computes the KDN sequence-mixer forward pass in its two
 * scan-compatible approximations, Diagonal KDN (d_k variance scalars per
 * head) and Isotropic KDN (one variance scalar per head), and the single-token
 * decode step.  The method is defined on the KDN reading notes (page
 * "Kalman Delta Networks: 不确定性感知的关联记忆"), method part:
 *   - exact filter it approximates: §2, Eq. (12)-(17);
 *   - Diagonal KDN predict/gain: §4, Eq. (23)-(30);
 *   - information scaling mu: §5, Eq. (60)-(65) (gain uses the predicted
 *     variance; mu only shapes the variance carried to the next token);
 *   - Moebius form of the variance recurrence and the affine memory scan:
 *     §6, Eq. (32)-(39), with the Appendix D chunking summarised there;
 *   - Isotropic KDN: §7, Eq. (40) and Appendix C;
 *   - parameters alpha (decay), omega (process noise), r (observation
 *     noise) as inputs, and "scanned training == token-by-token inference":
 *     §8.
 *
 * Per token t and head, with D_t = diag(alpha_t):
 *   Diagonal:  p^ = alpha^2 (.) p + omega;  z = sum_i p^_i k_i^2;
 *              kappa = p^ (.) k / (r + z);
 *              p <- p^ / (1 + (mu/r) k (.) k (.) p^)
 *   Isotropic: a = mean_i alpha_i^2;  b^ = a b + omega;  n = |k|^2;
 *              kappa = b^ k / (r + b^ n);  b <- b^ / (1 + mu n b^ / (d_k r))
 *   Memory (both): S <- D S;  delta = v - S^T k;  S <- S + kappa delta^T;
 *              o = S^T q   (read after this token's write)
 *
 * CONVENTIONS (every entry point)
 *   - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *     never frees caller memory and allocates nothing on the forward or step
 *     paths; scratch space, where a regime needs it, is the caller's
 *     `workspace`.
 *   - Layouts are dense row-major:
 *       activations q,k [B,T,H,dk], v,o [B,T,H,dv] in the io dtype;
 *       alpha [B,T,H,dk] fp32; omega [B,T,H,dk] (diag) or [B,T,H] (iso) fp32;
 *       r [B,T,H] fp32; state S [B,H,dk,dv] fp32 (row i = key channel);
 *       variances p [B,H,dk] (diag) or b [B,H] (iso) fp32.
 *   - io dtype: KDN_F32 or KDN_BF16 for q, k, v and o.  Gates, state and
 *     variances are always fp32.  bf16 runs its chunk contractions on bf16
 *     matrix cores with fp32 accumulation (split-operand products for
 *     Diagonal unless KDN_MATH_BF16 is given, below); fp32 runs them in
 *     fp32.
 *   - Supported sizes: dk in {64, 128} for bf16 and dk = 64 for fp32;
 *     dv a multiple of 64 (bf16) or 32 (fp32), at most 256; B, H >= 1;
 *     T >= 0; B*H*T and every tensor below 2^31 elements.
 *   - Pointers to q, k, v, alpha, omega, o, S0/S_T/S and p0/p_T must be
 *     16-byte aligned.
 *   - Preconditions (documented, not checked per element): r > 0,
 *     0 <= alpha <= 1, omega >= 0, p0/b0 > 0, mu >= 0, all finite.  Outside
 *     them results are unspecified (NaN propagates; nothing faults).
 *   - Strong decay in the chunked forwards (every call here but kdn_step):
 *     the chunk products pair the cumulative decay G_t from a 16-token
 *     chunk's start with its reciprocal.  Where a channel's chunk decays by
 *     more than 2^100 the kernels measure G from a power-of-two reference
 *     inside the chunk (exact up to rounding) down to a chunk product of
 *     2^-224 (about 4e-68).  Below that, fp32 cannot span the chunk: every
 *     alpha of that channel and chunk under 2^-14 (zero included) is taken
 *     as 2^-14 in the memory decay (the variance recurrence keeps the true
 *     alpha), which leaves at most 2^-14 of the previous state row per such
 *     token where the method would leave alpha of it.
 *   - Validation is synchronous: on any invalid argument the call returns a
 *     negative status and launches nothing.  Launch failures return
 *     KDN_ERR_HIP.  Kernel faults surface at the caller's stream
 *     synchronisation.  Results are asynchronous on `stream`.
 *   - Results are deterministic run to run (no floating-point atomics).
 *   - Inputs are never modified, except S and var_state in kdn_step.
 *   - kdn_last_error_message() returns a thread-local description of the
 *     last failure on the calling thread.
 */
#ifndef KDN_H
#define KDN_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDN_OK = 0,
    KDN_ERR_INVALID_ARG = -1,
    KDN_ERR_UNSUPPORTED = -2,
    KDN_ERR_WORKSPACE = -3,
    KDN_ERR_HIP = -4
} kdn_status;

typedef enum { KDN_F32 = 0, KDN_BF16 = 1 } kdn_dtype;
typedef enum { KDN_DIAG = 0, KDN_ISO = 1 } kdn_variant;

/* Contraction precision of the bf16 forward, OR-ed into io_dtype of
 * kdn_diag_fwd, kdn_iso_fwd, kdn_fwd_ex, kdn_fwd_preact and
 * kdn_fwd_workspace_size (no other call accepts it; nor KDN_OUT_F32 below).
 *
 * By default the Diagonal bf16 forward runs every chunk contraction as three
 * bf16 matrix-core products of split operands, x = hi + lo with hi = bf16(x)
 * and lo = bf16(x - hi), summed in fp32 (hi.hi + lo.hi + hi.lo): about 16
 * significant bits per operand, near fp32 results (~1e-5 relative L2 against
 * an fp64 reference).  This is the higher-precision Diagonal of the KDN
 * reading notes (results part §6: the mixer throughput figure ran Diagonal in
 * FP32 / TF32x3 within a BF16 configuration; conclusions part §2: Diagonal
 * pays for an extra scan and higher-precision compute).  The Isotropic bf16
 * forward runs single bf16 products, as the notes ran it.
 *
 * KDN_MATH_BF16 makes the Diagonal bf16 forward run single bf16 products as
 * well: faster, ~4e-3 relative L2 on o.  With fp32 io it is
 * KDN_ERR_INVALID_ARG. */
enum { KDN_MATH_BF16 = 0x100 };

/* Output dtype flag, OR-ed into io_dtype of the same forward calls: with bf16
 * q, k, v, the Diagonal forward's split-product contractions write o in fp32
 * ([B,T,H,dv] float, 16-byte aligned) instead of rounding it to bf16, so o
 * keeps the contractions' precision.  KDN_ERR_UNSUPPORTED with Isotropic or
 * with KDN_MATH_BF16; KDN_ERR_INVALID_ARG with fp32 io (o is fp32 there
 * already). */
enum { KDN_OUT_F32 = 0x200 };

/* Bytes of device workspace with which kdn_diag_fwd / kdn_iso_fwd (and
 * kdn_fwd_ex) run this shape fastest.  The workspace is optional: a call given
 * less (or NULL) runs the serial walk, with the same results up to rounding.
 * Nonzero only for bf16 io with dk == dv when the serial walk would fill at
 * most a quarter of the chip (B*H*dv/64 workgroups against 256 compute
 * units, MI355X's count, taken as fixed so that the size is a pure function
 * of the shape, whatever the device) and T splits into 4 or 8
 * segments of at least 1024 tokens, each a multiple of 64: the state
 * recurrence is affine in the state over any span of tokens (method part §2
 * and §6 of the KDN reading notes), so the segments run as independent walks
 * whose linear and affine parts a short per-head combine chains, and the
 * segment-entry variances come from the gain scan (method part §6).  The size
 * is then the gain scan's carries, two segment-variance planes and four
 * [B*S,H,dk,dv] fp32 state planes.  Returns 0 for invalid shapes too; the
 * forward call reports those. */
size_t kdn_fwd_workspace_size(int variant, int B, int T, int H, int dk, int dv,
                              int io_dtype);

/*
 * Diagonal KDN forward over T tokens (KDN reading notes, method part §4-§6;
 * Appendix D chunking).
 *   q, k   [B,T,H,dk] io dtype       v, o  [B,T,H,dv] io dtype
 *   alpha  [B,T,H,dk] fp32 decay      omega [B,T,H,dk] fp32 process noise
 *   r      [B,T,H]    fp32 observation noise
 *   S0     [B,H,dk,dv] fp32 initial state, or NULL for zeros
 *   p0     [B,H,dk]    fp32 initial variances, or NULL for ones
 *   mu     information scale (the pages' default is dk)
 *   S_T    [B,H,dk,dv] fp32 final state (required)
 *   p_T    [B,H,dk]    fp32 final variances (required)
 *   workspace / workspace_bytes: optional device scratch, 16-byte aligned;
 *     with kdn_fwd_workspace_size(...) bytes or more, shapes with few heads
 *     and long sequences run split over the sequence (NULL: serial walk).
 *     When it is used it must not overlap any other argument
 *     (KDN_ERR_INVALID_ARG).
 *   stream: a hipStream_t (NULL = the null stream)
 * S_T may alias S0 exactly (each workgroup reads its own columns of the
 * state before it overwrites them).  p_T may alias p0 exactly only when
 * dv <= 64 for bf16 io (dv <= 32 for fp32), i.e. one workgroup per head: with
 * more, every value-tile workgroup reads the initial variances and nothing
 * orders that read before the first tile's final write, so the call returns
 * KDN_ERR_INVALID_ARG (use separate p0 / p_T buffers).  A partial overlap of
 * either pair, or o aliasing q, k or v, is rejected with KDN_ERR_INVALID_ARG.
 */
kdn_status kdn_diag_fwd(int B, int T, int H, int dk, int dv, int io_dtype, float mu,
                        const void* q, const void* k, const void* v,
                        const float* alpha, const float* omega, const float* r,
                        const float* S0, const float* p0,
                        void* o, float* S_T, float* p_T,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Isotropic KDN forward (KDN reading notes, method part §7, Eq. (40);
 * Appendix C).  Same layouts as kdn_diag_fwd except
 *   omega  [B,T,H] fp32 (one process-noise scalar per head and token)
 *   b0     [B,H] fp32 initial variance, or NULL for ones
 *   b_T    [B,H] fp32 final variance (required)
 */
kdn_status kdn_iso_fwd(int B, int T, int H, int dk, int dv, int io_dtype, float mu,
                       const void* q, const void* k, const void* v,
                       const float* alpha, const float* omega, const float* r,
                       const float* S0, const float* b0,
                       void* o, float* S_T, float* b_T,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * One decode step, one token per sequence (KDN reading notes, method part
 * §8: token-by-token inference runs the same recurrence as the scan).
 *   variant   KDN_DIAG or KDN_ISO
 *   q, k [B,H,dk], v, o [B,H,dv] io dtype; alpha [B,H,dk] fp32;
 *   omega [B,H,dk] (diag) or [B,H] (iso) fp32; r [B,H] fp32
 *   S         [B,H,dk,dv] fp32, read and overwritten in place
 *   var_state p [B,H,dk] (diag) or b [B,H] (iso) fp32, in place
 * Equivalent to the forward call with T = 1, S0 = S_T = S and
 * p0 = p_T = var_state.
 */
kdn_status kdn_step(int variant, int B, int H, int dk, int dv, int io_dtype, float mu,
                    const void* q, const void* k, const void* v,
                    const float* alpha, const float* omega, const float* r,
                    float* S, float* var_state, void* o, void* stream);

/*
 * Extended forward (either variant) with the trained per-head parameters of
 * the end-to-end network (KDN reading notes, method part §8: a learned scalar
 * initial covariance c_{0,h} I and information scale mu per head) and the
 * effective write strength diagnostic (method part §2:
 * beta_eff_t = k_t^T kappa_t = z_t / (r_t + z_t); its distribution is the
 * results part's §4, Fig. 2).  Arguments as in kdn_diag_fwd / kdn_iso_fwd
 * (variant KDN_DIAG or KDN_ISO; var0 / var_T are p0 / p_T or b0 / b_T), plus
 *   mu_h      [H] fp32 device, nullable: information scale of head h (used
 *             instead of mu; entries must be finite and >= 0, not checked)
 *   c0_h      [H] fp32 device, nullable: initial variance of head h, every
 *             channel (Diagonal) or the head's scalar (Isotropic); only
 *             when var0 is NULL -- giving both is KDN_ERR_INVALID_ARG
 *   beta_eff  [B,T,H] fp32 device, nullable: written with beta_eff of every
 *             token; must not alias r, o, S_T or var_T
 * All three are 4-byte aligned.  With all three NULL the call equals
 * kdn_diag_fwd / kdn_iso_fwd.  In the bf16 forward z_t is the diagonal of the
 * chunk's bf16 key product, so beta_eff carries the same bf16 rounding as
 * the gain it describes.
 */
kdn_status kdn_fwd_ex(int variant, int B, int T, int H, int dk, int dv, int io_dtype, float mu,
                      const float* mu_h, const void* q, const void* k, const void* v,
                      const float* alpha, const float* omega, const float* r, const float* S0,
                      const float* var0, const float* c0_h, void* o, float* S_T, float* var_T,
                      float* beta_eff, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Extended decode step: kdn_step with a per-head information scale mu_h [H]
 * (nullable, as in kdn_fwd_ex) and the token's effective write strength
 * beta_eff [B,H] fp32 (nullable).  Same passages as kdn_fwd_ex.
 */
kdn_status kdn_step_ex(int variant, int B, int H, int dk, int dv, int io_dtype, float mu,
                       const float* mu_h, const void* q, const void* k, const void* v,
                       const float* alpha, const float* omega, const float* r, float* S,
                       float* var_state, void* o, float* beta_eff, void* stream);

/*
 * Exact dense-covariance Kalman memory for small d_k (KDN reading notes,
 * method part §2, Eq. (12)-(17)), with the Diagonal KDN's gates as the
 * transition D_t = diag(alpha_t) and process noise Omega_t = diag(omega_t):
 * the filter whose mean-field projection is Diagonal KDN (method part §4).
 * An ablation and cross-check tool (a serial Riccati step per token), not a
 * throughput path; the information scale mu does not apply to it.
 *   q, k   [B,T,H,dk] io dtype       v, o  [B,T,H,dv] io dtype
 *   alpha, omega [B,T,H,dk] fp32     r     [B,T,H] fp32
 *   S0 [B,H,dk,dv] fp32 (NULL: zeros),  P0 [B,H,dk,dk] fp32 (NULL: identity)
 *   S_T, P_T  final state and covariance (required; may alias S0 / P0
 *             exactly, a partial overlap is KDN_ERR_INVALID_ARG)
 *   beta_eff  [B,T,H] fp32, nullable: z / (r + z), z = k^T P^ k
 * dk in {16, 32, 64}, dv in {16, 32, 64, 128}; fp32 arithmetic throughout.
 */
kdn_status kdn_dense_fwd(int B, int T, int H, int dk, int dv, int io_dtype, const void* q,
                         const void* k, const void* v, const float* alpha, const float* omega,
                         const float* r, const float* S0, const float* P0, void* o, float* S_T,
                         float* P_T, float* beta_eff, void* stream);

/*
 * Forward from the gates' pre-activations (KDN reading notes, method part
 * §8: the end-to-end network produces alpha = sigmoid(a), omega =
 * softplus(w) and r = r_min + softplus(rho) from its projections; the notes
 * use r_min = 0.01).  Arguments as kdn_fwd_ex, with the gates replaced by
 *   a_pre  [B,T,H,dk] io dtype (bf16 or fp32, as q/k/v), 16-byte aligned
 *   w_pre  [B,T,H,dk] (Diagonal) or [B,T,H] (Isotropic), io dtype, 16-byte aligned
 *   r_pre  [B,T,H] io dtype, 16-byte aligned
 *   r_min  > 0 and finite (keeps r > 0)
 * With bf16 io (and fp32 o not requested) the forward reads a_pre (and the
 * Diagonal w_pre) itself and forms alpha (and omega) on chip, with the
 * arithmetic of kdn_gates_from_preact; only r (and the Isotropic per-token
 * omega) pass through the workspace.  With fp32 io an elementwise pre-pass
 * writes all three gates into the workspace and the forward of kdn_fwd_ex
 * runs on them.  Either way the result equals, bit for bit, kdn_fwd_ex on
 * the gates kdn_gates_from_preact returns.  The workspace
 * (kdn_fwd_preact_workspace_size bytes, 16-byte aligned, disjoint from every
 * argument) is sized for the fp32 gates.  Validation happens before anything
 * is launched.  Every finite pre-activation is
 * accepted: a very negative a gives a small or zero alpha (sigmoid saturates
 * to 0 below about -88), which the strong-decay rule above covers.
 */
size_t kdn_fwd_preact_workspace_size(int variant, int B, int T, int H, int dk);
kdn_status kdn_fwd_preact(int variant, int B, int T, int H, int dk, int dv, int io_dtype,
                          float mu, const float* mu_h, const void* q, const void* k,
                          const void* v, const void* a_pre, const void* w_pre, const void* r_pre,
                          float r_min, const float* S0, const float* var0, const float* c0_h,
                          void* o, float* S_T, float* var_T, float* beta_eff, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * The gates alone from their pre-activations (KDN reading notes, method part
 * §8), as the forward from pre-activations forms them:
 *   alpha = sigmoid(a_pre)           [B,T,H,dk]
 *   omega = softplus(w_pre)          [B,T,H,dk] (Diagonal) or [B,T,H] (Isotropic)
 *   r     = r_min + softplus(r_pre)  [B,T,H]
 * Pre-activations in io_dtype (KDN_F32 or KDN_BF16, no flags), outputs fp32;
 * every pointer device memory, 16-byte aligned, non-null when T > 0, and no
 * output overlaps any input or other output.  r_min > 0 and finite.  The
 * sigmoid and softplus use the hardware exp2 / log2 (~1 ulp each; softplus
 * through log1p as log(u) e / (u - 1), u = 1 + e); the same operations form
 * the gates inside the bf16 forward, so its results equal kdn_fwd_ex's on
 * these gates bit for bit.  Asynchronous on `stream`.
 */
kdn_status kdn_gates_from_preact(int variant, int B, int T, int H, int dk, int io_dtype,
                                 const void* a_pre, const void* w_pre, const void* r_pre,
                                 float r_min, float* alpha, float* omega, float* r,
                                 void* stream);

/*
 * Backward pass of Diagonal / Isotropic KDN (the mixer is trained through the
 * scanned recurrence, KDN reading notes, method part §8; the notes print no
 * gradient formulas, so this is the reverse-mode derivative of the
 * recurrences of method part §2, §4-§5 and §7, including the information-
 * scaled variance update).  It returns the gradients of a loss L given
 *   d_o     [B,T,H,dv] io dtype: dL/do
 *   dS_T    [B,H,dk,dv] fp32, nullable (zero): dL/dS_T
 *   dvar_T  shape of var0, fp32, nullable (zero): dL/dp_T or dL/db_T
 * for the forward defined by the same arguments as kdn_fwd_ex (variant,
 * sizes, io_dtype, mu, mu_h, q, k, v, alpha, omega, r, S0, var0, c0_h).
 * Outputs (device, written in full; none may overlap any other buffer):
 *   dq, dk [B,T,H,dk] and dv [B,T,H,dv] in the io dtype
 *   dalpha [B,T,H,dk], domega (the shape of omega), dr [B,T,H] fp32
 *   dS0 [B,H,dk,dv], dvar0 (shape of var0), dmu [B,H] fp32, each nullable:
 *     the gradients by the initial state, the initial variance (also when it
 *     came from c0_h or the default 1; dL/dc0_h sums it over b and, for
 *     Diagonal, channels) and by the information scale each (b,h) used
 *     (dL/dmu_h sums it over b)
 * dk in {64, 128}, dv a multiple of 16 up to 256; fp32 arithmetic whatever
 * the io type.  q, k, v, d_o and alpha are 16-byte aligned, the other fp32
 * arrays 4-byte aligned, dq / dk / dv aligned to their element size.  The
 * forward is recomputed inside: the gain, then the state at every 16th token
 * (Diagonal with bf16 io and dv a multiple of 64: by the forward walk with
 * split-bf16 products, ~1e-5 relative; otherwise in fp32 products).
 * With dv a multiple of 64 the memory part runs in 16-token chunks on the
 * matrix cores (fp32 products); otherwise token by token from stored
 * innovations.  The workspace (kdn_bwd_workspace_size bytes, 16-byte aligned)
 * holds those and per-column-block partial sums.  Diagonal shapes with
 * dk = dv whose B*H*(dv/64) workgroups fill at most half of the chip and
 * whose T splits into 2, 4 or 8 segments of at least 1024 tokens (each a
 * multiple of 64) run split over the sequence with bf16 io: the state map
 * over a span is affine (method part §2, §6), so the reverse pass carries
 * the state adjoint into a segment from its right as M^T dS + (the
 * segment's own part), and the segments run side by side (their entry
 * states from the forward walk with split-bf16 products).  For those shapes
 * kdn_bwd_workspace_size includes the split's planes; a smaller workspace of
 * at least the rest runs the same call without the split.  Deterministic (no
 * atomics).  Asynchronous on `stream`; validation as for the forward.
 */
size_t kdn_bwd_workspace_size(int variant, int B, int T, int H, int dk, int dv);
kdn_status kdn_bwd(int variant, int B, int T, int H, int dk, int dv, int io_dtype, float mu,
                   const float* mu_h, const void* q, const void* k, const void* v,
                   const float* alpha, const float* omega, const float* r, const float* S0,
                   const float* var0, const float* c0_h, const void* d_o, const float* dS_T,
                   const float* dvar_T, void* dq, void* dk_out, void* dv_out, float* dalpha,
                   float* domega, float* dr, float* dS0, float* dvar0, float* dmu,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward of kdn_fwd_preact: the gradients by the gates' pre-activations
 * (KDN reading notes, method part §8; d sigmoid(a)/da = alpha (1 - alpha),
 * d softplus(x)/dx = sigmoid(x)).  Arguments as kdn_bwd with the gates
 * replaced by a_pre, w_pre, r_pre and r_min as in kdn_fwd_preact, and their
 * gradients da_pre [B,T,H,dk], dw_pre (shape of w_pre), dr_pre [B,T,H] in
 * fp32 in place of dalpha, domega, dr.  The prologue writes the gates into the
 * front of the workspace (kdn_bwd_preact_workspace_size bytes, 16-byte
 * aligned), kdn_bwd runs on them with the rest of it, then the chain rule is
 * applied in place.  No output and no part of the workspace may overlap the
 * pre-activations.
 */
size_t kdn_bwd_preact_workspace_size(int variant, int B, int T, int H, int dk, int dv);
kdn_status kdn_bwd_preact(int variant, int B, int T, int H, int dk, int dv, int io_dtype,
                          float mu, const float* mu_h, const void* q, const void* k,
                          const void* v, const void* a_pre, const void* w_pre, const void* r_pre,
                          float r_min, const float* S0, const float* var0, const float* c0_h,
                          const void* d_o, const float* dS_T, const float* dvar_T, void* dq,
                          void* dk_out, void* dv_out, float* da_pre, float* dw_pre, float* dr_pre,
                          float* dS0, float* dvar0, float* dmu, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * Gain scan alone (the variance recurrence and Kalman gain without the
 * memory), exposed for the chunk-parallel regime's tests and diagnostics.
 * Inputs as in the forward calls (q, v not needed).  Writes
 *   kappa [B,T,H,dk] fp32 gain (nullable),
 *   var_T p_T [B,H,dk] (diag) or b_T [B,H] (iso) fp32 (required).
 * The scan composes the per-channel 2x2 Moebius maps
 *   M_t = [[alpha^2, omega], [u alpha^2, 1 + u omega]]
 * (KDN reading notes, method part §6, Eq. (32)-(39)) within 64-token chunks
 * (one lane per channel for Diagonal, a wavefront scan over the tokens for
 * Isotropic), then applies the chunk summaries to the variance in chunk order
 * to get every chunk's entry variance, then replays each chunk from it.
 * Needs kdn_gain_workspace_size(...) bytes of workspace.
 */
size_t kdn_gain_workspace_size(int variant, int B, int T, int H, int dk);
kdn_status kdn_gain_scan(int variant, int B, int T, int H, int dk, int io_dtype, float mu,
                         const void* k, const float* alpha, const float* omega,
                         const float* r, const float* var0,
                         float* kappa, float* var_T,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * The gain scan above without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments, results and validation
 * as kdn_gain_scan; its scratch (the chunk summaries and carries) is a static
 * device array of kdn_gain_scan_static_max_bytes() bytes (32 MiB) that every
 * GPU the library runs on holds from the library's load until the process
 * ends.  A shape whose kdn_gain_workspace_size exceeds that returns
 * KDN_ERR_WORKSPACE and launches nothing.  The call allocates nothing.
 * Every call on one GPU shares that GPU's scratch, which keeps the last call's
 * contents (nothing in it needs clearing: each call writes what it reads), so
 * calls that overlap on one GPU (concurrent streams, or threads without
 * ordering) race: order them on one stream.
 */
size_t kdn_gain_scan_static_max_bytes(void);
kdn_status kdn_gain_scan_static(int variant, int B, int T, int H, int dk, int io_dtype, float mu,
                                const void* k, const float* alpha, const float* omega,
                                const float* r, const float* var0, float* kappa, float* var_T,
                                void* stream);

/*
 * ---------------------------------------------------------------------------
 * The operators around the mixer in its layer: layer norm, the short causal
 * convolution that feeds q, k and v, and a gated recurrence per channel (the
 * memory recurrence S <- D S + ... without keys).  Conventions as above, with
 * these differences:
 *   - io dtype KDN_F32 or KDN_BF16 (no flags but KDN_CLEAR_TAIL, below);
 *     parameters (weight, bias), statistics and recurrent states are fp32; all
 *     arithmetic is fp32 and a value is rounded once, when it is stored.
 *   - Any channel count D from 1 to 2^20; rows, or B T, up to 2^30; B below
 *     2^24.  Pointers need only their element's alignment
 *     (workspaces: 16 bytes); 16-byte alignment and D a multiple of 8 run
 *     fastest.
 *   - Inputs marked "rows of D, `stride` apart" may be slices of wider rows
 *     (one third of a fused projection, say): row i starts at element
 *     i * stride, D <= stride <= 2^30 (2^22 in kdn_rec_fwd and kdn_rec_bwd).
 *     Everything else is dense.
 *   - No output may overlap any other buffer, unless a call says so.
 *   - Packed sequences: with `cu_seqlens` (device, int32 [N+1], N >= 1) B must
 *     be 1, and sequence n is the tokens cu_seqlens[n] .. cu_seqlens[n+1] - 1
 *     of the row.  Offsets start at 0, never decrease and end at or before T;
 *     a sequence may be empty.  Tokens from cu_seqlens[N] on belong to no
 *     sequence: nothing of an output is written there (zeros with
 *     KDN_CLEAR_TAIL), and they add to no gradient.  Without cu_seqlens (NULL, N ignored) each of the B rows is one
 *     sequence and N below means B.  Offsets are not checked; bad ones give
 *     unspecified values, but no access outside the tensors.
 *   - Infinities and NaN of one sequence never reach another one; in the
 *     recurrence's states and adjoints they go on to the end of their own.
 *   - Deterministic, capturable into a HIP graph; two calls that may run at
 *     the same time need a workspace each.
 */

/*
 * OR-ed into the io_dtype of the forward and backward calls that take packed
 * sequences (kdn_conv, kdn_rec, kdn_linattn): the rows of y, of h and
 * checkpoints, of o and of the gradients by token behind the last packed sequence are set to
 * zero instead of left as they were.
 */
enum { KDN_CLEAR_TAIL = 0x400 };

/*
 * Layer norm over the last axis: rows of D,
 *   mean = sum(x) / D, rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
 *   y = (x - mean) rstd weight + bias
 *   x      rows of D, x_stride apart, io dtype     y [rows, D] io dtype
 *   weight, bias [D] fp32, each nullable (ones, zeros)
 *   mean, rstd   [rows] fp32, written; each nullable
 *   eps    finite, >= 0
 * The variance is taken around the mean, in a second pass over the row.
 */
kdn_status kdn_layer_norm_fwd(int rows, int D, int io_dtype, float eps, const void* x,
                              long long x_stride, const float* weight, const float* bias,
                              void* y, float* mean, float* rstd, void* stream);

/*
 * Backward of kdn_layer_norm_fwd.  With g = dy weight and xh = (x - mean) rstd:
 *   dx = rstd (g - mean(g) - xh mean(g xh)),
 *   dweight = sum over rows of dy xh, dbias = sum over rows of dy
 *   dy [rows, D] io dtype; x as in the forward; mean, rstd [rows] from it
 *   dx [rows, D] io dtype; dweight, dbias [D] fp32, each nullable
 * The workspace (kdn_layer_norm_bwd_workspace_size bytes) holds partial sums
 * of dweight and dbias; it is not needed when both are NULL.
 */
size_t kdn_layer_norm_bwd_workspace_size(int rows, int D);
kdn_status kdn_layer_norm_bwd(int rows, int D, int io_dtype, const void* dy, const void* x,
                              long long x_stride, const float* mean, const float* rstd,
                              const float* weight, void* dx, float* dweight, float* dbias,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Activation of the convolution's output. */
typedef enum { KDN_ACT_NONE = 0, KDN_ACT_SILU = 1 } kdn_activation;

/*
 * Short causal convolution, one filter of W taps (2 <= W <= 4) per channel:
 *   z_t = bias + sum_{j < W} weight[W-1-j] x_{t-j},   y = z, or z sigmoid(z)
 * where the W - 1 inputs before a sequence's first token are its state0 (oldest
 * first; zeros when NULL).
 *   x [B,T,D] rows x_stride apart, y [B,T,D] io dtype
 *   weight [W,D] fp32 (the last row multiplies the current token),
 *   bias [D] fp32, nullable
 *   state0, state_T [N,W-1,D] io dtype, nullable: the last W - 1 inputs before
 *   the sequence and at its end (with state0 moved up for a sequence that is
 *   shorter).  They must not overlap.
 */
kdn_status kdn_conv_fwd(int B, int T, int D, int W, int io_dtype, int activation, const void* x,
                        long long x_stride, const float* weight, const float* bias,
                        const void* state0, const int* cu_seqlens, int N, void* y, void* state_T,
                        void* stream);

/*
 * Backward of kdn_conv_fwd (z is formed again from x).  dy [B,T,D] and
 * dstate_T [N,W-1,D] (nullable: zeros) in the io dtype are the gradients by y
 * and state_T; dx [B,T,D] (rows of a dense tensor), dstate0 [N,W-1,D] (nullable) io dtype,
 * dweight [W,D] and dbias [D] (nullable) fp32 are written in full, but for dx
 * of tokens behind the last sequence.
 */
size_t kdn_conv_bwd_workspace_size(int B, int T, int D, int W);
kdn_status kdn_conv_bwd(int B, int T, int D, int W, int io_dtype, int activation, const void* dy,
                        const void* x, long long x_stride, const float* weight, const float* bias,
                        const void* state0, const int* cu_seqlens, int N, const void* dstate_T,
                        void* dx, float* dweight, float* dbias, void* dstate0, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * One token of kdn_conv_fwd for each of B sequences: x (rows of D, x_stride
 * apart) and y [B,D]; state [B,W-1,D] is read and moved on in place.
 */
kdn_status kdn_conv_step(int B, int D, int W, int io_dtype, int activation, const void* x,
                         long long x_stride, const float* weight, const float* bias, void* state,
                         void* y, void* stream);

/* How the recurrence gets its decay: alpha itself, or its pre-activation. */
typedef enum { KDN_GATE_ALPHA = 0, KDN_GATE_PREACT = 1 } kdn_gate;

/* Tokens between the states that the recurrence's forward keeps for its
 * backward. */
enum { KDN_REC_CHECKPOINT = 64 };

/*
 * Gated recurrence per channel:
 *   h_t = alpha_t h_{t-1} + u_t,   u_t = x_t, or (1 - alpha_t) x_t with `blend`
 *   x     [B,T,D] rows x_stride apart, io dtype
 *   a     [B,T,D] rows a_stride apart: alpha in fp32 (KDN_GATE_ALPHA, 0 <=
 *         alpha <= 1), or a_pre in the io dtype with alpha = sigmoid(a_pre)
 *         (KDN_GATE_PREACT; 1 - alpha is then formed without cancellation)
 *   h0    [N,D] fp32 state before each sequence, nullable (zeros)
 *   h     [B,T,D] io dtype;  h_T [N,D] fp32, nullable: the state after each
 *         sequence (h0 for an empty one)
 *   checkpoints  [B, ceil(T / KDN_REC_CHECKPOINT), D] fp32, nullable: the state
 *         before every 64th token of the row, for kdn_rec_bwd
 *   workspace    kdn_rec_fwd_workspace_size bytes (0 for short rows)
 */
size_t kdn_rec_fwd_workspace_size(int B, int T, int D);
kdn_status kdn_rec_fwd(int B, int T, int D, int io_dtype, int gate, int blend, const void* x,
                       long long x_stride, const void* a, long long a_stride, const float* h0,
                       const int* cu_seqlens, int N, void* h, float* h_T, float* checkpoints,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward of kdn_rec_fwd, for dh [B,T,D] (io dtype) = dL/dh and dh_T [N,D]
 * (fp32, nullable: zeros) = dL/dh_T.  The states are formed again in fp32 from
 * the forward's checkpoints.  With lam_t = dh_t + alpha_{t+1} lam_{t+1} (dh_T in
 * place of the second term at a sequence's end):
 *   dx = lam, or (1 - alpha) lam with `blend`           [B,T,D] io dtype
 *   da = lam h_{t-1}, or lam (h_{t-1} - x_t), by alpha  [B,T,D] fp32; times
 *        alpha (1 - alpha) by a_pre                     [B,T,D] io dtype
 *   dh0 = alpha_1 lam_1 (dh_T for an empty sequence)    [N,D] fp32, nullable
 */
size_t kdn_rec_bwd_workspace_size(int B, int T, int D);
kdn_status kdn_rec_bwd(int B, int T, int D, int io_dtype, int gate, int blend, const void* dh,
                       const void* x, long long x_stride, const void* a, long long a_stride,
                       const float* checkpoints, const float* h0, const int* cu_seqlens, int N,
                       const float* dh_T, void* dx, void* da, float* dh0, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * One token of kdn_rec_fwd for each of B sequences: x, a (rows of D, x_stride
 * and a_stride apart), h [B,D]; state [B,D] fp32 is read and overwritten.
 */
kdn_status kdn_rec_step(int B, int D, int io_dtype, int gate, int blend, const void* x,
                        long long x_stride, const void* a, long long a_stride, float* state,
                        void* h, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Linear attention with a decay for each head: the memory recurrence without
 * a gain and without the delta rule.  Conventions as for the operators above.
 * Per token and head h, with g = decay[h] and the q and k of head h / (H / Hk):
 *   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
 *   q, k  [B,T,Hk,dk], v [B,T,H,dv] io dtype; H a multiple of Hk (a group of
 *         adjacent heads shares one q and k); dk, dv from 1 to 256.  Token t of
 *         a row's head starts `stride` elements behind token t - 1 (rows follow
 *         one another T tokens apart) and `head_stride` behind the head before:
 *         dim <= head_stride, (heads - 1) head_stride + dim <= stride <= 2^22
 *   decay [H] fp32, 0 <= g <= 1 (constants: they have no gradient here)
 *   scale finite
 *   S0    [N,H,dk,dv] fp32 state before each sequence, nullable (zeros)
 *   o     [B,T,H,dv] io dtype;  S_T [N,H,dk,dv] fp32, nullable: the state after
 *         each sequence (S0 for an empty one)
 *   workspace  kdn_linattn_fwd_workspace_size bytes (0 unless few heads have
 *         many tokens: the states handed between pieces of a sequence)
 * bf16: products of bf16 operands, summed in fp32; operands that are not inputs
 * (the decayed q k^T, the state where o is formed from it, the decayed v that
 * states are summed from) are held to 16 bits, as two bf16 parts, the last to 24
 * where the state is an output and the token still has an eighth of its weight in
 * it: o is off by its own rounding.  fp32: products of fp32 operands.
 * What is not finite stays in its sequence and head and reaches no earlier
 * token; an infinity may become a NaN later in the sequence.
 */
size_t kdn_linattn_fwd_workspace_size(int B, int T, int H, int dk, int dv);
kdn_status kdn_linattn_fwd(int B, int T, int H, int Hk, int dk, int dv, int io_dtype, float scale,
                           const void* q, long long q_stride, long long q_head_stride,
                           const void* k, long long k_stride, long long k_head_stride,
                           const void* v, long long v_stride, long long v_head_stride,
                           const float* decay, const float* S0, const int* cu_seqlens, int N,
                           void* o, float* S_T, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * Backward of kdn_linattn_fwd, for d_o [B,T,H,dv] (io dtype) = dL/do and dS_T
 * [N,H,dk,dv] (fp32, nullable: zeros) = dL/dS_T.  With
 * R_t = scale q_t d_o_t^T + g R_{t+1} (dS_T in place of the second term at a
 * sequence's end):
 *   dq_t = scale S_t d_o_t, dk_t = R_t v_t, summed over a group's heads
 *                                                   [B,T,Hk,dk] io dtype
 *   dv_t = R_t^T k_t                                [B,T,H,dv]  io dtype
 *   dS0  = g R_1 (dS_T for an empty sequence)       [N,H,dk,dv] fp32, nullable
 * S_t is formed again from S0, k and v.
 */
size_t kdn_linattn_bwd_workspace_size(int B, int T, int H, int Hk, int dk, int dv);
kdn_status kdn_linattn_bwd(int B, int T, int H, int Hk, int dk, int dv, int io_dtype, float scale,
                           const void* d_o, const void* q, long long q_stride,
                           long long q_head_stride, const void* k, long long k_stride,
                           long long k_head_stride, const void* v, long long v_stride,
                           long long v_head_stride, const float* decay, const float* S0,
                           const int* cu_seqlens, int N, const float* dS_T, void* dq, void* dk_out,
                           void* dv_out, float* dS0, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * One token of kdn_linattn_fwd for each of B sequences: q, k (rows of [Hk,dk]),
 * v (rows of [H,dv]), strides as above; o [B,H,dv]; state [B,H,dk,dv] fp32 is
 * updated in place.
 */
kdn_status kdn_linattn_step(int B, int H, int Hk, int dk, int dv, int io_dtype, float scale,
                            const void* q, long long q_stride, long long q_head_stride,
                            const void* k, long long k_stride, long long k_head_stride,
                            const void* v, long long v_stride, long long v_head_stride,
                            const float* decay, float* state, void* o, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Group norm with an activation, channels last: x [N,S,C], N samples of S
 * positions, G groups of C / G adjacent channels.  Over the positions and a
 * group's channels of a sample,
 *   mean = sum(x) / n, rstd = 1 / sqrt(sum((x - mean)^2) / n + eps),  n = S C / G
 *   z = (x - mean) rstd weight + bias,   y = z, or z sigmoid(z) (KDN_ACT_SILU)
 * S = 1 with a head's outputs as a group normalises each head of a token.
 *   x      rows of C, x_stride apart (N S of them), io dtype;  y [N,S,C] io dtype
 *   weight, bias [C] fp32, each nullable (ones, zeros)
 *   mean, rstd   [N,G] fp32, written (zeros where S = 0); each nullable
 *   eps    finite, >= 0;  N G below 2^24
 *   workspace    kdn_group_norm_fwd_workspace_size bytes (0 unless a group is
 *          too large for one workgroup, or not whole vectors in a large call)
 */
size_t kdn_group_norm_fwd_workspace_size(int N, int S, int C, int G);
kdn_status kdn_group_norm_fwd(int N, int S, int C, int G, int io_dtype, int activation, float eps,
                              const void* x, long long x_stride, const float* weight,
                              const float* bias, void* y, float* mean, float* rstd, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Backward of kdn_group_norm_fwd with its mean and rstd, weight and bias (which
 * the activation's slope needs).  With g = dy, or dy times the slope at z, and
 * xh = (x - mean) rstd:
 *   dx = rstd (g w - mean(g w) - xh mean(g w xh)), means over the group
 *   dweight = sum of g xh, dbias = sum of g, over samples and positions
 *   dy, dx [N,S,C] io dtype; dweight, dbias [C] fp32, each nullable
 */
size_t kdn_group_norm_bwd_workspace_size(int N, int S, int C, int G);
kdn_status kdn_group_norm_bwd(int N, int S, int C, int G, int io_dtype, int activation,
                              const void* dy, const void* x, long long x_stride, const float* mean,
                              const float* rstd, const float* weight, const float* bias, void* dx,
                              float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * Dropout from a counter-based generator, with the residual stream added:
 *   y = (kept ? x / (1 - p') : 0) + residual
 * Element i of [rows,D] is kept where its 16 random bits are at least p' 2^16,
 * p' being p (0 <= p <= 1) rounded to a multiple of 2^-16, ties to even.  The
 * bits are word (i % 8) / 2, half i % 2 (0: the low one) of Philox4x32-10
 * (Salmon, Moraes, Dror, Shaw 2011) for the counter {i / 8 (64 bits), offset
 * (64 bits)} under the key `seed`, low words first: they depend on nothing but
 * seed, offset and i.  Calls that are to be independent take offsets (or
 * seeds) of their own.
 *   seed_offset  nullable; device, int64 {seed, offset}, read by the kernel in
 *        place of the two arguments: a captured graph that is replayed takes
 *        what stands there then
 *   x    rows of D, x_stride apart, io dtype; residual [rows,D] io dtype,
 *        nullable; y [rows,D] io dtype
 * What is dropped may be infinite or NaN: it leaves no trace.
 */
kdn_status kdn_dropout_fwd(int rows, int D, int io_dtype, double p, unsigned long long seed,
                           unsigned long long offset, const long long* seed_offset, const void* x,
                           long long x_stride, const void* residual, void* y, void* stream);

/*
 * Backward of kdn_dropout_fwd by x, for the same p, seed and offset: dx = kept ?
 * dy / (1 - p') : 0.  (The residual's gradient is dy.)  dy, dx [rows,D].
 */
kdn_status kdn_dropout_bwd(int rows, int D, int io_dtype, double p, unsigned long long seed,
                           unsigned long long offset, const long long* seed_offset, const void* dy,
                           void* dx, void* stream);

const char* kdn_status_string(int status);
const char* kdn_last_error_message(void);

/* Library version, e.g. "kdn-mi355x 0.1.0 gfx950". */
const char* kdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDN_H */
