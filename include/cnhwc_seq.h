/*
 * cnhwc_seq.h -- C ABI of the sequence operators of the channels-last library
 * for AMD MI355X (gfx950): layer norm and root-mean-square norm over channels,
 * the short causal (depthwise) convolution, the selective state space scan,
 * rotary positions and linear attention with a decay for each head, each forward
 * and backward; the convolution, the scan and linear attention also for single tokens.
 *
 * Together with the pointwise conv1d of cnhwc.h they make up sequence blocks:
 * norm, projection, causal convolution, scan with its gate, projection; or norm,
 * projection, rotary positions of q and k, linear attention, projection.
 *
 * Layouts.  Sequences are [N,L,C] with the channels innermost (stride 1).
 * Input tensors carry the element strides of N and L in the descriptor, so a
 * tensor may be a slice of a wider projection's rows; strides are >= 0 and
 * bounded so that no offset passes 2^62.  Outputs, gradients, states and
 * parameters are dense.  dtype is the element type of the activations (F32,
 * F16, BF16); every sum, statistic and state is held in fp32 and each output is
 * rounded once, round-to-nearest-even.
 *
 * lengths (may be NULL: every position is valid): N int32 on the device, the
 * number of valid leading positions of each sequence, clamped to [0, L].
 * Positions past it are never read; outputs and gradients there are 0, the
 * states stay what they were after the last valid position.  No output depends
 * on what a tensor holds past the lengths.
 *
 * Ownership, threading, streams and errors are those of cnhwc.h: the caller
 * owns every buffer, calls queue kernels on the given stream and neither
 * allocate nor synchronise, every argument is checked before anything is
 * queued, and results depend on the arguments alone, with the same bits on
 * every call (no atomics).  Tensor pointers are aligned to their element, the
 * workspace and fp32 tensors to 16 bytes.  Outputs overlap nothing, except
 * where they are named as updated in place (a step's state_out on its state).
 */
#ifndef CNHWC_SEQ_H_
#define CNHWC_SEQ_H_

#include <stdint.h>

#include "cnhwc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ layer norm
 * y = (x - mean) * rstd * w + b over the C channels of each of the N*L rows,
 * rstd = 1 / sqrt(var + eps), var the mean square of x - mean. */
typedef struct {
  int32_t dtype;        /* cnhwc_dtype_t of x, y, dy, dx */
  int32_t w_dtype;      /* of w, b, dw, db: dtype or CNHWC_F32 */
  int64_t n, l, c;      /* each in [1, 2^31) */
  int64_t x_stride[2];  /* elements: sequence, position */
  int64_t dy_stride[2]; /* backward only */
  float eps;            /* >= 0 */
  int32_t reserved;     /* 0 */
} cnhwc_layer_norm_desc_t;

/* w, b: [C], both may be NULL (w NULL: 1, b NULL: 0; b needs w).
 * mean, rstd: fp32 [N*L], both or neither; the backward pass takes them. */
cnhwc_status_t cnhwc_layer_norm_fwd(const cnhwc_layer_norm_desc_t* desc, const void* x, const void* w,
                                    const void* b, void* y, float* mean, float* rstd, void* hip_stream);

/* Bytes of workspace of the backward pass (0 without parameter gradients). */
cnhwc_status_t cnhwc_layer_norm_bwd_workspace(const cnhwc_layer_norm_desc_t* desc, int32_t param_grads,
                                              uint64_t* bytes);

/* dx [N,L,C], and dw, db [C] (both, with w, or neither). */
cnhwc_status_t cnhwc_layer_norm_bwd(const cnhwc_layer_norm_desc_t* desc, const void* dy, const void* x,
                                    const float* mean, const float* rstd, const void* w, void* dx,
                                    void* dw, void* db, void* workspace, uint64_t workspace_bytes,
                                    void* hip_stream);

/* ------------------------------------------------------------ causal convolution
 * X = K-1 rows of state (zeros if NULL) followed by the valid rows of x:
 *   pre[t,c] = bias[c] + sum_k w[c,k] X[t+k,c],  y = act(pre)
 * so position t sees itself and the K-1 before it.  state_out = the last K-1
 * rows of X.  w [C,K], bias [C] (may be NULL) and the states [N,K-1,C] have
 * the activations' dtype. */
typedef enum { CNHWC_ACT_NONE = 0, CNHWC_ACT_SILU = 1 } cnhwc_activation_t;

#define CNHWC_CAUSAL_CONV_MAX_K 8

typedef struct {
  int32_t dtype;
  int32_t activation;   /* cnhwc_activation_t */
  int64_t n, l, c;      /* each in [1, 2^31) */
  int32_t k;            /* taps, in [1, CNHWC_CAUSAL_CONV_MAX_K]; more is UNSUPPORTED */
  int32_t reserved;     /* 0 */
  int64_t x_stride[2];
  int64_t dy_stride[2]; /* backward only */
} cnhwc_causal_conv_desc_t;

/* state, lengths and state_out may be NULL. */
cnhwc_status_t cnhwc_causal_conv_fwd(const cnhwc_causal_conv_desc_t* desc, const void* x, const void* w,
                                     const void* bias, const void* state, const int32_t* lengths,
                                     void* y, void* state_out, void* hip_stream);

cnhwc_status_t cnhwc_causal_conv_bwd_workspace(const cnhwc_causal_conv_desc_t* desc, uint64_t* bytes);

/* dx [N,L,C], dw [C,K], dbias [C] (with bias, else NULL), dstate [N,K-1,C] (may
 * be NULL), from dy and dstate_out (the gradient of state_out; NULL: 0). */
cnhwc_status_t cnhwc_causal_conv_bwd(const cnhwc_causal_conv_desc_t* desc, const void* dy,
                                     const void* dstate_out, const void* x, const void* w,
                                     const void* bias, const void* state, const int32_t* lengths,
                                     void* dx, void* dw, void* dbias, void* dstate, void* workspace,
                                     uint64_t workspace_bytes, void* hip_stream);

/* One position (l == 1, x [N,C] at x_stride[0]).  state_out may be state
 * itself (updated in place); any other overlap of the two is an error. */
cnhwc_status_t cnhwc_causal_conv_step(const cnhwc_causal_conv_desc_t* desc, const void* x,
                                      const void* state, const void* w, const void* bias, void* y,
                                      void* state_out, void* hip_stream);

/* ------------------------------------------------------------ selective scan
 *   D[t,d] = softplus(delta[t,d] + delta_bias[d])     (softplus == 0: the sum)
 *   h[t,d,s] = exp(D[t,d] a[d,s]) h[t-1,d,s] + D[t,d] u[t,d] b[t,s]
 *   y[t,d] = (sum_s c[t,s] h[t,d,s] + skip[d] u[t,d]) * silu(gate[t,d])
 * b and c are shared by all channels.  The state h is fp32 [N,D,S].  The decays of
 * up to a chunk of positions are joined in one exponential of the sum of D a, which
 * does not overflow where D a <= 0; states that grow by e^88 and more do not fit
 * fp32, and may come out as NaN. */
#define CNHWC_SCAN_MAX_STATE 64

typedef struct {
  int32_t dtype;          /* of u, delta, b, c, gate, y, dy and their gradients */
  int32_t softplus;       /* 0 or 1 */
  int64_t n, l, d;        /* each in [1, 2^31) */
  int32_t s;              /* in [1, CNHWC_SCAN_MAX_STATE]; more is UNSUPPORTED */
  int32_t reserved;       /* 0 */
  int64_t u_stride[2], delta_stride[2], b_stride[2], c_stride[2], gate_stride[2];
  int64_t dy_stride[2];   /* backward only */
} cnhwc_scan_desc_t;

typedef struct {
  const void* u;            /* [N,L,D] */
  const void* delta;        /* [N,L,D] */
  const float* a;           /* [D,S] */
  const void* b;            /* [N,L,S] */
  const void* c;            /* [N,L,S] */
  const float* skip;        /* [D] or NULL (0) */
  const void* gate;         /* [N,L,D] or NULL (no gate factor) */
  const float* delta_bias;  /* [D] or NULL (0) */
  const float* state;       /* [N,D,S] or NULL (0) */
  const int32_t* lengths;   /* [N] or NULL */
} cnhwc_scan_inputs_t;

typedef struct {
  void* u;            /* [N,L,D] */
  void* delta;        /* [N,L,D] */
  float* a;           /* [D,S] */
  void* b;            /* [N,L,S] */
  void* c;            /* [N,L,S] */
  float* skip;        /* [D], with inputs.skip, else NULL */
  void* gate;         /* [N,L,D], with inputs.gate, else NULL */
  float* delta_bias;  /* [D], with inputs.delta_bias, else NULL */
  float* state;       /* [N,D,S] or NULL */
} cnhwc_scan_grads_t;

cnhwc_status_t cnhwc_scan_fwd_workspace(const cnhwc_scan_desc_t* desc, uint64_t* bytes);

/* y [N,L,D]; state_out [N,D,S] may be NULL. */
cnhwc_status_t cnhwc_scan_fwd(const cnhwc_scan_desc_t* desc, const cnhwc_scan_inputs_t* in, void* y,
                              float* state_out, void* workspace, uint64_t workspace_bytes,
                              void* hip_stream);

cnhwc_status_t cnhwc_scan_bwd_workspace(const cnhwc_scan_desc_t* desc, uint64_t* bytes);

/* Gradients of every input from dy [N,L,D] and dstate_out (the gradient of the
 * final state; NULL: 0).  Nothing has to be kept from the forward pass. */
cnhwc_status_t cnhwc_scan_bwd(const cnhwc_scan_desc_t* desc, const cnhwc_scan_inputs_t* in,
                              const void* dy, const float* dstate_out,
                              const cnhwc_scan_grads_t* grads, void* workspace,
                              uint64_t workspace_bytes, void* hip_stream);

/* One position (l == 1; in->state is required, in->lengths must be NULL).
 * state_out may be in->state itself (updated in place). */
cnhwc_status_t cnhwc_scan_step(const cnhwc_scan_desc_t* desc, const cnhwc_scan_inputs_t* in, void* y,
                               float* state_out, void* hip_stream);

/* ------------------------------------------------------------ root-mean-square norm
 * z = x + residual (x alone without one), rstd = 1 / sqrt(mean z^2 + eps) over the C
 * channels of each of the N*L rows, y = z rstd w.  sum receives z in the
 * activations' dtype; y comes from z before that rounding.  The mean is fp32: a row
 * with elements beyond about 1e19 has rstd 0, and so y 0.
 *
 * The 8-bit form stores q in e4m3 (OCP: 448 the largest value) and scale, fp32, so
 * that y = q * scale: scale = max |y| / 448 over the row [N*L], or over each group of
 * `group` channels [N*L, C / group], and at least 2^-100.  NaN stays NaN and counts
 * for no maximum; where |y| is infinite the whole row or group is NaN. */
typedef struct {
  int32_t dtype;              /* cnhwc_dtype_t of x, residual, sum, y, dy, dsum, dx */
  int32_t w_dtype;            /* of w, dw: dtype or CNHWC_F32 */
  int64_t n, l, c;            /* each in [1, 2^31) */
  int64_t x_stride[2];        /* elements: sequence, position */
  int64_t residual_stride[2]; /* of residual; in the backward pass of dsum */
  int64_t dy_stride[2];       /* backward only */
  float eps;                  /* >= 0 */
  int32_t group;              /* 8-bit form: channels to a scale, 32, 64 or 128, dividing C; 0: the row.
                                 0 elsewhere */
} cnhwc_rms_norm_desc_t;

/* residual, w [C], sum and rstd (fp32 [N*L]) may be NULL; sum needs residual, and
 * may be residual itself where that is dense (updated in place). */
cnhwc_status_t cnhwc_rms_norm_fwd(const cnhwc_rms_norm_desc_t* desc, const void* x, const void* residual,
                                  const void* w, void* y, void* sum, float* rstd, void* hip_stream);

/* q: one byte an element. */
cnhwc_status_t cnhwc_rms_norm_fwd_q8(const cnhwc_rms_norm_desc_t* desc, const void* x, const void* residual,
                                     const void* w, void* q, float* scale, void* sum, float* rstd,
                                     void* hip_stream);

/* Bytes of workspace of the backward pass (0 without the parameter's gradient). */
cnhwc_status_t cnhwc_rms_norm_bwd_workspace(const cnhwc_rms_norm_desc_t* desc, int32_t param_grads,
                                            uint64_t* bytes);

/* dx [N,L,C], the gradient of z and so of x and of residual, and dw [C] (with w, or
 * NULL), from dy and dsum (what reaches z past the norm; NULL: 0); x is z. */
cnhwc_status_t cnhwc_rms_norm_bwd(const cnhwc_rms_norm_desc_t* desc, const void* dy, const void* dsum,
                                  const void* x, const float* rstd, const void* w, void* dx, void* dw,
                                  void* workspace, uint64_t workspace_bytes, void* hip_stream);

/* ------------------------------------------------------------ rotary positions
 * The first R channels of each head of x [N,L,H,D] turn in R/2 pairs, by the angle
 * position * freqs[i] and times scale; the channels from R on are copied.  The
 * pair i: channels i and i + R/2, or 2i and 2i + 1 (interleaved).  The position is
 * offset + positions[n,t], or offset + t without positions.  inverse turns back
 * (still times scale): the gradient. */
typedef struct {
  int32_t dtype;              /* of x and out */
  int32_t interleaved;        /* 0 or 1 */
  int64_t n, l, h;            /* each in [1, 2^31) */
  int32_t d, r;               /* d >= 1; r even, in [0, d] */
  int64_t x_stride[3], out_stride[3]; /* elements: sequence, position, head */
  int64_t position_stride[2];
  int64_t offset;             /* within 2^40 of 0 */
  float scale;
  int32_t inverse;            /* 0 or 1 */
  int64_t reserved;           /* 0 */
} cnhwc_rotary_desc_t;

/* freqs: fp64 [R/2], radians a position; positions: int32 or NULL.  out has
 * strides of its own and may be x itself, with the same ones. */
cnhwc_status_t cnhwc_rotary(const cnhwc_rotary_desc_t* desc, const void* x, const double* freqs,
                            const int32_t* positions, void* out, void* hip_stream);

/* ------------------------------------------------------------ linear attention
 *   S[t] = exp(log_decay[h]) S[t-1] + k[t]^T v[t],   y[t] = scale q[t] S[t]
 * for each head; the state S is fp32 [N,H,DK,DV].  Decays are meant (log_decay <= 0,
 * minus infinity included).  Growth is taken where exp(log_decay) and every state fit
 * fp32 (a state of 0 stays 0 however long), for values and products of q and k up to 1e19;
 * it runs in smaller steps, slower, from exp(1.3) a position on (exp(0.6) in log_decay's
 * gradient), in f16 from exp(0.25).  An
 * infinity or NaN in v reaches, as NaN, the y of its channel from its position on.
 * Heads may be shared through strides of 0; gradients are those of each head.  N * H
 * above 2^20 and L above 2^30 are UNSUPPORTED.
 *
 * Arithmetic: the states, their decays and every sum are fp32.  With 16-bit activations an
 * operand of a matrix product is rounded to their type once (the products of q and
 * k under their decays, the state that 32 positions start from) on the way to y and the
 * gradients of q, k and v; on the way to a state and to log_decay's gradient it is taken
 * in terms: three of bf16, fp32's digits; two of f16 on the way to a state.  f16 has a
 * narrow range: what is rounded once is off by 2^-11 of itself or 2^-39 of the largest that it
 * stands beside (a position's products, 16 columns of a state), what is in two terms by 2^-22
 * of itself or 2^-39 of the largest of its column in 32 positions (2^-50 where log_decay * 32
 * is beyond 5.5 either way). */
#define CNHWC_LINEAR_ATTENTION_MAX_DIM 256

typedef struct {
  int32_t dtype;          /* of q, k, v, y, dy and their gradients */
  int32_t reserved;       /* 0 */
  int64_t n, l, h;        /* each in [1, 2^31) */
  int32_t dk, dv;         /* in [1, CNHWC_LINEAR_ATTENTION_MAX_DIM]; more is UNSUPPORTED */
  int64_t q_stride[3], k_stride[3], v_stride[3];  /* elements: sequence, position, head */
  int64_t dy_stride[3];   /* backward only */
  float scale;
  int32_t reserved2;      /* 0 */
} cnhwc_linear_attention_desc_t;

typedef struct {
  const void* q;            /* [N,L,H,DK] */
  const void* k;            /* [N,L,H,DK] */
  const void* v;            /* [N,L,H,DV] */
  const float* log_decay;   /* [H] */
  const float* state;       /* [N,H,DK,DV] or NULL (0) */
  const int32_t* lengths;   /* [N] or NULL */
} cnhwc_linear_attention_inputs_t;

typedef struct {
  void* q;                  /* [N,L,H,DK] */
  void* k;                  /* [N,L,H,DK] */
  void* v;                  /* [N,L,H,DV] */
  float* log_decay;         /* [H] or NULL (not wanted) */
  float* state;             /* [N,H,DK,DV] or NULL */
} cnhwc_linear_attention_grads_t;

cnhwc_status_t cnhwc_linear_attention_fwd_workspace(const cnhwc_linear_attention_desc_t* desc, uint64_t* bytes);

/* y [N,L,H,DV]; state_out [N,H,DK,DV] may be NULL. */
cnhwc_status_t cnhwc_linear_attention_fwd(const cnhwc_linear_attention_desc_t* desc,
                                          const cnhwc_linear_attention_inputs_t* in, void* y, float* state_out,
                                          void* workspace, uint64_t workspace_bytes, void* hip_stream);

cnhwc_status_t cnhwc_linear_attention_bwd_workspace(const cnhwc_linear_attention_desc_t* desc,
                                                    int32_t decay_grad, uint64_t* bytes);

/* Gradients from dy [N,L,H,DV] and dstate_out (the gradient of the final state;
 * NULL: 0).  Nothing has to be kept from the forward pass. */
cnhwc_status_t cnhwc_linear_attention_bwd(const cnhwc_linear_attention_desc_t* desc,
                                          const cnhwc_linear_attention_inputs_t* in, const void* dy,
                                          const float* dstate_out, const cnhwc_linear_attention_grads_t* grads,
                                          void* workspace, uint64_t workspace_bytes, void* hip_stream);

/* One position (l == 1; in->state is required, in->lengths must be NULL).
 * state_out may be in->state itself (updated in place). */
cnhwc_status_t cnhwc_linear_attention_step(const cnhwc_linear_attention_desc_t* desc,
                                           const cnhwc_linear_attention_inputs_t* in, void* y,
                                           float* state_out, void* hip_stream);

#ifdef __cplusplus
}
#endif
#endif /* CNHWC_SEQ_H_ */
