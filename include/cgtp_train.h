/*
 * cgtp_train.h -- C ABI of the operators that surround a convolution when an
 * equivariant network is trained: the gated residual norm of a block and the
 * optimizer step.  Same library, status codes, element types and stream rules
 * as cgtp.h.  The paper pages have no counterpart: "An Efficient Sparse Kernel
 * Generator ...", "Sobek ..." and "LunaTP ..." take both from the user's model.
 */
#ifndef CGTP_TRAIN_H
#define CGTP_TRAIN_H

#include "cgtp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cgtp_resnorm_s* cgtp_resnorm;

/* Gate a(q): none (a = 1, q is not read), a = q, sigmoid(q), q sigmoid(q). */
typedef enum { CGTP_ACT_NONE = 0, CGTP_ACT_IDENTITY = 1, CGTP_ACT_SIGMOID = 2, CGTP_ACT_SILU = 3 } cgtp_act;

/*
 * Gated residual norm.  Rows are irreps features in the layout of cgtp.h; block b
 * has mul channels of 2l+1 components, c = (b, u) numbers the channels (C in
 * all).  With rms_b(x) = (mean over the block's elements of x^2 + eps)^(-1/2),
 * which rotations leave unchanged,
 *
 *   out = alpha h + scale_c a(q_c) post_c rms_b(z) z
 *   y   = pre_c rms_b(out) out
 *
 * One launch joins the end of a block (norm of its result z, gate, residual
 * scale, residual) to the norm in front of the next one.  y is computed from
 * `out` as it is stored.
 *
 *  flags : CGTP_RESNORM_POST (rms of z; without it that factor is 1),
 *      CGTP_RESNORM_PRE (y is wanted), CGTP_RESNORM_STORAGE (below).
 *  dtype : CGTP_F32, CGTP_F64: every tensor in that type.  CGTP_BF16: what the
 *      next product reads (y, gz, gq) in bfloat16 and the rest (h, out, z, q,
 *      gout, gy, gh) in FP32, as CGTP_BF16 plans of cgtp.h have it; with
 *      CGTP_RESNORM_STORAGE every row tensor in bfloat16.  Parameters (post,
 *      scale, pre) and their gradients are FP32 (FP64 for CGTP_F64), arithmetic
 *      and sums too.
 *  alpha : factor of the residual.  eps >= 0, rounded to the type of the arithmetic;
 *      with eps = 0 a block of zeros has no norm (NaN).  Squares are summed in FP32 (FP64):
 *      elements above 1.8e19 overflow them, elements below 1e-19 lose digits in them.
 * The plan owns its tables and the partial sums of the parameter gradients: backwards
 * of the same plan must not overlap on the GPU.
 */
#define CGTP_RESNORM_POST 1
#define CGTP_RESNORM_PRE 2
#define CGTP_RESNORM_STORAGE 4
cgtp_status cgtp_resnorm_create(cgtp_resnorm* plan, const char* irreps, int dtype, int flags, int act, double alpha,
                                double eps);
void cgtp_resnorm_destroy(cgtp_resnorm plan);
/* Row length dim, channels C and number of blocks.  Any pointer may be NULL. */
cgtp_status cgtp_resnorm_info(cgtp_resnorm plan, int64_t* dim, int64_t* channels, int* blocks);
/* Device memory of the plan, as cgtp_plan_device_bytes. */
cgtp_status cgtp_resnorm_device_bytes(cgtp_resnorm plan, int64_t* bytes);

/*
 * cgtp_resnorm_forward
 *  h [N,dim], z [N,dim], q [N,C] -> out [N,dim], y [N,dim]; post, scale, pre [C].
 *  ld_* : distance between rows in elements (0: rows are contiguous), so that
 *      gates and features may be column ranges of one product's output.  Row
 *      tensors need the alignment of their element only; 16-byte aligned rows
 *      are faster.
 *  h may be NULL (no residual); z may be NULL (then out must be NULL, q, post
 *  and scale are not read, the stream is h itself, without alpha, and y is its
 *  norm); post, scale and pre may be NULL (factor 1).  q is read unless act is
 *  CGTP_ACT_NONE or z is NULL.  y must be NULL without CGTP_RESNORM_PRE, and given
 *  with it.
 *  Outputs may not overlap inputs.  N = 0 is allowed and launches nothing; N < 2^30.
 */
cgtp_status cgtp_resnorm_forward(cgtp_resnorm plan, int64_t N, const void* h, int64_t ld_h, const void* z,
                                 int64_t ld_z, const void* q, int64_t ld_q, const void* post, const void* scale,
                                 const void* pre, void* out, int64_t ld_out, void* y, int64_t ld_y, void* stream);

/*
 * cgtp_resnorm_backward -- adjoint for gout [N,dim] (NULL: zero) and gy [N,dim]
 *  (given exactly with CGTP_RESNORM_PRE).  x is the forward's `out`, or h when z is NULL;
 *  it is read for the norm of y only and may be NULL without CGTP_RESNORM_PRE.
 *  gh [N,dim] (NULL: not wanted; alpha enters it only where z is given), gz [N,dim]
 *  and gq [N,C] (given exactly when z is, and q is read); gpost, gscale, gpre [C] (NULL: not wanted; a sum over the N
 *  rows in a fixed order, zero for N = 0).  A NULL factor's gradient may be asked for.
 */
cgtp_status cgtp_resnorm_backward(cgtp_resnorm plan, int64_t N, const void* gout, int64_t ld_gout, const void* gy,
                                  int64_t ld_gy, const void* x, int64_t ld_x, const void* z, int64_t ld_z,
                                  const void* q, int64_t ld_q, const void* post, const void* scale, const void* pre,
                                  void* gh, int64_t ld_gh, void* gz, int64_t ld_gz, void* gq, int64_t ld_gq,
                                  void* gpost, void* gscale, void* gpre, void* stream);

/*
 * AdamW over many tensors in one launch (two above 1024 tensors, and so on).
 * With g' = coefficient * g (1 without clip) and step t >= 1,
 *
 *   m <- beta1 m + (1 - beta1) g'        v <- beta2 v + (1 - beta2) g'^2
 *   p <- p (1 - lr wd_i) - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * where wd_i = weight_decay * decay_scale[i] of tensor i.
 *
 * The states of all tensors lie in one buffer each for m and v: tensor i starts
 * at a multiple of 128 elements, after the tensors before it, so the buffers
 * have state_numel = sum of numel rounded up to 128.  Zeros are the initial
 * states (all four buffers).
 *  CGTP_STATE_FULL : m and v in the type of the parameters.
 *  CGTP_STATE_8BIT : one byte an element and one exponent byte for each 128
 *      elements (m_exp, v_exp [state_numel / 128]), CGTP_F32 parameters.  A
 *      block's exponent is a power of two, so the codes' grid stays where it is
 *      from step to step.  m: sign, 4-bit exponent, 3-bit mantissa; v: 5-bit
 *      exponent, 3-bit mantissa; below the smallest exponent the codes are
 *      linear to zero.  The update uses the unrounded m and v; what is stored is
 *      rounded stochastically (changes far below one code step, such as 0.1% of
 *      v, still move it on average), with 16 bits that depend on seed, t and the
 *      element's place alone.  The mean of what is stored lies up to 2^-17 of a
 *      code step nearer to zero: v settles up to 0.1% low for beta2 = 0.999, 10%
 *      for 0.99999.  A positive v is never stored as zero.  A block that holds an
 *      infinity, a NaN or a number above 3.19e38 is stored as NaNs.
 */
typedef struct cgtp_adamw_s* cgtp_adamw;
typedef enum { CGTP_STATE_FULL = 0, CGTP_STATE_8BIT = 1 } cgtp_state;

/*
 *  numel [n_tensors] : HOST array, elements of each tensor (0 is allowed).
 *  decay_scale [n_tensors] : HOST array or NULL (1 for every tensor).
 *  The optimizer owns its tables and the gradient norm's partial sums: norms of
 *  the same optimizer must not overlap on the GPU.
 *  param_dtype : CGTP_F32 or CGTP_F64.  grad_dtype : that type, or CGTP_BF16 with
 *      CGTP_F32 parameters.
 */
cgtp_status cgtp_adamw_create(cgtp_adamw* opt, int n_tensors, const int64_t* numel, const float* decay_scale,
                              int param_dtype, int grad_dtype, int state);
void cgtp_adamw_destroy(cgtp_adamw opt);
/* Elements of the m and v buffers.  The pointer may be NULL. */
cgtp_status cgtp_adamw_info(cgtp_adamw opt, int64_t* state_numel);
cgtp_status cgtp_adamw_device_bytes(cgtp_adamw opt, int64_t* bytes);

/*
 * cgtp_adamw_step -- one step in place.
 *  params, grads : HOST arrays of n_tensors DEVICE pointers, read during the
 *      call only.  A NULL gradient leaves its tensor and states as they are.
 *      Tensors need the alignment of their element; 16-byte aligned ones are
 *      faster.
 *  copies : NULL, or a HOST array of DEVICE pointers (any may be NULL) to
 *      bfloat16 tensors that receive the new parameters rounded once (CGTP_F32).
 *  m, v, m_exp, v_exp : DEVICE states, 16-byte aligned (m_exp, v_exp NULL for
 *      CGTP_STATE_FULL).
 *  clip : NULL, or what cgtp_grad_norm wrote.  Where its coefficient is not a
 *      finite number the step changes nothing.
 *  lr, step, seed and the other numbers are host values, taken at the call.  In a
 *      captured graph they are those of the capture: every replay repeats that
 *      step's bias correction and rounding bits (an 8-bit v that is always rounded
 *      with the same bits may stop moving).  A training loop captures its passes
 *      and calls the step outside the graph, or captures the step anew.
 */
cgtp_status cgtp_adamw_step(cgtp_adamw opt, void* const* params, const void* const* grads, void* const* copies,
                            void* m, void* v, void* m_exp, void* v_exp, double lr, double beta1, double beta2,
                            double eps, double weight_decay, int64_t step, uint64_t seed, const void* clip,
                            void* stream);

/*
 * cgtp_grad_norm -- out[0] = norm of all gradients together, out[1] = the
 * coefficient min(1, max_norm / norm) (NaN where the norm is not finite), in the
 * type of the parameters; max_norm > 0 (infinity: the norm alone).  NULL
 * gradients count as zero.  Summed in a fixed order.
 */
cgtp_status cgtp_grad_norm(cgtp_adamw opt, const void* const* grads, double max_norm, void* out, void* stream);

/* The values the 8-bit states stand for, as FP32 m_out, v_out [state_numel]. */
cgtp_status cgtp_adamw_state_values(cgtp_adamw opt, const void* m, const void* v, const void* m_exp,
                                    const void* v_exp, float* m_out, float* v_out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CGTP_TRAIN_H */
