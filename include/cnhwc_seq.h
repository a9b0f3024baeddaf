/*
 * cnhwc_seq.h -- C ABI of the sequence operators of the channels-last library
 * for AMD MI355X (gfx950): layer norm over channels, the short causal
 * (depthwise) convolution, and the selective state space scan, each forward
 * and backward, and the last two also for single tokens.
 *
 * Together with the pointwise conv1d of cnhwc.h they make up a sequence block:
 * norm, projection, causal convolution, scan with its gate, projection.
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
 * where a step's state_out is its state.
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

#ifdef __cplusplus
}
#endif
#endif /* CNHWC_SEQ_H_ */
