/*
 * pararnn_block.h -- C ABI of libpararnn_block.so: what a recurrent language model's block and its training step are made
 * of beside the operators of pararnn_lm.h, on MI355X (gfx950): a short causal convolution, the selective state space scan,
 * a gated feed-forward product, each with its gradients, and an AdamW step over many tensors.
 *
 * Conventions are those of pararnn_lm.h: device pointers, status codes, asynchronous on `stream`, arguments checked before
 * anything is launched, nothing thrown, no allocation, no synchronisation, capturable in a HIP graph, a 256-byte aligned
 * workspace of the queried size whose contents need not be initialised; planes strided with a dense last dimension (strides in
 * elements, nonnegative); `dtype` (pararnn_dtype) is the storage type of the big planes, arithmetic and everything else is
 * float32; sizes of any value; pointers need the alignment of their element type only; outputs must not overlap inputs unless an
 * entry says so; every result is a fixed sequence of operations on its inputs.
 */
#ifndef PARARNN_BLOCK_H
#define PARARNN_BLOCK_H

#include "pararnn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PARARNN_BLOCK_ABI_VERSION 1

/* ------------------------------------------------------------------------------------------------
 * Short causal convolution along time, each channel by itself, K taps (1 <= K <= PARARNN_BLOCK_MAX_TAPS, else
 * UNSUPPORTED):
 *     p_t = bias + sum_k w[k] x_{t-K+1+k},     y_t = p_t sig(p_t)   (y_t = p_t without silu)
 * The K - 1 steps before a sequence's first are its state; the last K - 1 of state and sequence together are the state that
 * leaves it.  UNSUPPORTED also: 2^31 or more elements in one row of time chunks by channel tiles (a launch's limit).
 * ---------------------------------------------------------------------------------------------- */
#define PARARNN_BLOCK_MAX_TAPS 8

typedef struct {
  int32_t dtype;             /* of x, y and, in the gradient, dy, d_x                                   */
  int32_t silu;              /* 0 or 1                                                                  */
  int64_t B, T, D;           /* each >= 0                                                               */
  int64_t K;
  const void* x;             /* [B][T][D]                                                               */
  int64_t sx[2];             /* its strides over b and t                                                */
  const float* weight;       /* [D][K]                                                                  */
  const float* bias;         /* [D] or NULL                                                             */
  const float* state;        /* [B][n][K-1][D] steps before each sequence, oldest first, dense, n = 1 without
                                cu_seqlens, else n_seqs; NULL = zeros                                   */
  const int32_t* cu_seqlens; /* as in pararnn_lm_scan                                                   */
  int64_t n_seqs;
} pararnn_block_conv;

/* one size for both calls; 0 for invalid sizes */
size_t pararnn_block_conv_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t K);

/*   y     [B][T][D] of dtype, strides sy
 *   last  [B][n][K-1][D] float32: the state leaving each sequence, or NULL; it may be the array `state` itself */
pararnn_status pararnn_block_causal_conv(const pararnn_block_conv* prob, void* y, const int64_t sy[2], float* last,
                                         void* stream);

/* Gradients for dy [B][T][D] of dtype and d_last [B][n][K-1][D] (NULL = zeros):
 *   d_x [B][T][D] of dtype;  d_weight [D][K], d_bias [D], d_state [B][n][K-1][D] float32, each may be NULL    */
typedef struct {
  const void* dy;
  const float* d_last;
  void* d_x;
  int64_t sdy[2], sdx[2];
  float *d_weight, *d_bias, *d_state;
} pararnn_block_conv_grad;
pararnn_status pararnn_block_causal_conv_vjp(const pararnn_block_conv* prob, const pararnn_block_conv_grad* grad, void* ws,
                                             size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Selective state space scan.  For every batch row b, channel d, state n and step t, with g the channel's group:
 *     dt = softplus(delta_t[d] + dt_bias[d]),    h_t[d,n] = exp(dt A[d,n]) h_{t-1}[d,n] + dt x_t[d] B_t[g,n]
 *     y_t[d] = (sum_n C_t[g,n] h_t[d,n] + skip[d] x_t[d]) z_t[d] sig(z_t[d])
 * The D channels form G groups of D / G consecutive ones, which share B and C.  N <= PARARNN_BLOCK_MAX_STATES (else
 * UNSUPPORTED); so are a T of 2^31 - 16 or more, strides over t of PARARNN_BLOCK_SSM_MAX_STEP or more (T > 1), and a launch of 2^32
 * threads.  A's sign is not checked: positive rates grow.  A rate of -infinity is a state that forgets at every step; its gradients with
 * respect to delta and dt_bias are NaN (0 times infinity), all others are finite.
 * ---------------------------------------------------------------------------------------------- */
#define PARARNN_BLOCK_MAX_STATES 32
#define PARARNN_BLOCK_SSM_MAX_STEP (1 << 24)
/* steps of one chunk (the state entering each is what the gradient rebuilds h from) */
#define PARARNN_BLOCK_SSM_CHUNK 16

typedef struct {
  int32_t dtype;             /* of x, delta, z, B, C, y and, in the gradient, dy and their gradients    */
  int64_t B, T, D, N, G;     /* B, T, D >= 0; N, G >= 1; G divides D                                    */
  const void *x, *delta, *z; /* [B][T][D]; z may be NULL (no gate)                                      */
  int64_t sx[2], sdelta[2], sz[2];
  const void *b, *c;         /* [B][T][G][N]                                                            */
  int64_t sb[3], sc[3];      /* their strides over b, t and g                                           */
  const float* A;            /* [D][N]                                                                  */
  const float* skip;         /* [D] or NULL (0)                                                         */
  const float* dt_bias;      /* [D] or NULL (0)                                                         */
  const float* h0;           /* [B][n][D][N] state entering each sequence, dense, n = 1 without cu_seqlens, else
                                n_seqs; NULL = zeros                                                    */
  const int32_t* cu_seqlens; /* as in pararnn_lm_scan                                                   */
  int64_t n_seqs;
} pararnn_block_ssm;

/* chunks of a row of T steps: a middle size of `carry` */
int64_t pararnn_block_ssm_chunks(int64_t T);
/* for the forward call and for the gradient; 0 for invalid sizes */
size_t pararnn_block_ssm_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, int gradient);

/*   y       [B][T][D] of dtype, strides sy
 *   h_last  [B][n][D][N] float32: the state leaving each sequence (h0 where it is empty), or NULL; it may be h0 itself
 *   carry   [B][chunks][N][D] float32: the state entering each chunk (not of its steps' sequences where one begins at the
 *           chunk's first step), which the gradient needs, or NULL                                       */
pararnn_status pararnn_block_selective_scan(const pararnn_block_ssm* prob, void* y, const int64_t sy[2], float* h_last,
                                            float* carry, void* ws, size_t ws_bytes, void* stream);

/* Gradients for dy [B][T][D] of dtype and d_last [B][n][D][N] float32 (NULL = zeros), from the carry of the same problem:
 *   d_x, d_delta, d_z [B][T][D], d_b, d_c [B][T][G][N] of dtype (d_z: with z only, else NULL)
 *   d_A [D][N], d_skip [D], d_dt_bias [D], d_h0 [B][n][D][N] float32, each may be NULL                   */
typedef struct {
  const float* carry;
  const void* dy;
  const float* d_last;
  void *d_x, *d_delta, *d_z, *d_b, *d_c;
  int64_t sdy[2], sdx[2], sddelta[2], sdz[2], sdb[3], sdc[3];
  float *d_A, *d_skip, *d_dt_bias, *d_h0;
} pararnn_block_ssm_grad;
pararnn_status pararnn_block_selective_scan_vjp(const pararnn_block_ssm* prob, const pararnn_block_ssm_grad* grad, void* ws,
                                                size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Gated feed-forward product of R rows:  g = x w_gate^T,  u = x w_up^T,  h = act(g) u, with act(g) = g sig(g) or
 * g Phi(g) in its tanh form.  x [R][D], w_gate, w_up [F][D], h [R][F] of dtype, with row strides.
 *   pre  [R][2F] float32, dense: g and u of each row side by side, for the gradient; or NULL
 * Bfloat16 products are exact and summed in float32.  Float32 products have float32's accuracy; an infinity among float32 values
 * makes the results it enters infinite or NaN, which of the two depends on the sizes (up to 64 rows the forward pass multiplies in
 * float32, otherwise a value is split into bfloat16).
 * UNSUPPORTED: R, D or F of 2^31 - 512 or more.
 * ---------------------------------------------------------------------------------------------- */
typedef enum { PARARNN_BLOCK_SILU = 0, PARARNN_BLOCK_GELU = 1 } pararnn_block_act;
size_t pararnn_block_gated_linear_workspace_bytes(int dtype, int64_t R, int64_t D, int64_t F, int gradient);
pararnn_status pararnn_block_gated_linear(int dtype, int act, int64_t R, int64_t D, int64_t F, const void* x, int64_t x_stride,
                                          const void* w_gate, int64_t gate_stride, const void* w_up, int64_t up_stride,
                                          void* h, int64_t h_stride, float* pre, void* ws, size_t ws_bytes, void* stream);
/* Gradients for dh [R][F] of dtype, from the forward's pre:  dg = dh u act'(g),  du = dh act(g) (with bfloat16 planes held as a
 * sum of two bfloat16, off by at most 2^-16 of each value: the products' operands),
 *     d_x = dg w_gate + du w_up,  d_w_gate = dg^T x,  d_w_up = du^T x, in dtype; d_x [R][D] with a row stride or NULL,
 *     d_w_gate, d_w_up [F][D] with row strides, both or none NULL                                        */
pararnn_status pararnn_block_gated_linear_vjp(int dtype, int act, int64_t R, int64_t D, int64_t F, const void* x,
                                              int64_t x_stride, const void* w_gate, int64_t gate_stride, const void* w_up,
                                              int64_t up_stride, const float* pre, const void* dh, int64_t dh_stride, void* d_x,
                                              int64_t d_x_stride, void* d_w_gate, int64_t d_gate_stride, void* d_w_up,
                                              int64_t d_up_stride, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * One AdamW step over `count` tensors.  With g' = grad_scale g:
 *     m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2,
 *     p = p (1 - lr weight_decay) - lr (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 * Tensor j has numel[j] elements; its moments begin at element offset[j] of the state, a multiple of
 * PARARNN_BLOCK_ADAMW_BLOCK; elements of a tensor's last block past its end are neither read nor written (32 bits) or written as
 * zero (8 bits).
 * bits = 32: m, v float32.  bits = 8: a byte each, with a float32 scale s for each block of PARARNN_BLOCK_ADAMW_BLOCK elements
 * of m and of v, the smallest power of two of at least 2^-80 with max |value| <= 1.875 s.  A code's lowest three bits are f, the
 * bits above it e (m: four and a sign above them, bias 15; v: five, bias 31): the magnitude is s (1 + f/8) 2^(e-bias), for e = 0
 * s f/8 2^(1-bias).  A new moment is rounded up or down at random, with probabilities that keep its mean to 2^-16 of a step (to
 * nearest, slow averages would stand still): up where its place between two codes and a multiple of 2^-16 below one, 16 bits of a hash of
 * the seed, the step and the element's place in the state, add up to one or more (m) or to more than one (v).  A block
 * with a NaN, an infinity or a magnitude above 1.875 2^127 has s = NaN, and its values are NaN from then on.
 * The step and, if wanted, lr and grad_scale may be read from device memory, so that a captured graph follows them.
 * The same tensor must not be given twice, nor overlapping ones.
 * ---------------------------------------------------------------------------------------------- */
#define PARARNN_BLOCK_ADAMW_BLOCK 256
typedef struct {
  void* param;               /* float32 or bfloat16, updated in place                                   */
  const void* grad;
  int64_t numel, offset;
  int32_t param_dtype, grad_dtype;
} pararnn_block_adamw_tensor;
typedef struct {
  int32_t bits;              /* 8 or 32                                                                 */
  double beta1, beta2, eps, weight_decay;   /* betas in [0, 1), eps >= 0, all finite                    */
  double lr, grad_scale;     /* used where the pointers below are NULL                                  */
  int64_t step;              /* >= 1; used where step_ptr is NULL                                       */
  const float *lr_ptr, *grad_scale_ptr;
  const int64_t* step_ptr;   /* device memory                                                           */
  uint64_t seed;             /* 8 bits                                                                  */
  void *m, *v;
  float *m_scale, *v_scale;  /* 8 bits: [state elements / PARARNN_BLOCK_ADAMW_BLOCK]                    */
} pararnn_block_adamw_args;
/* `tensors` is host memory, read before the call returns */
pararnn_status pararnn_block_adamw(const pararnn_block_adamw_args* args, const pararnn_block_adamw_tensor* tensors, int64_t count,
                                   void* stream);
/* The values of n elements of 8-bit moments (n a multiple of PARARNN_BLOCK_ADAMW_BLOCK), in bfloat16, which holds them exactly */
pararnn_status pararnn_block_adamw_moments(int64_t n, const void* m, const void* v, const float* m_scale, const float* v_scale,
                                           void* m_out, void* v_out, void* stream);

/* PARARNN_BLOCK_ABI_VERSION of the built library */
int pararnn_block_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* PARARNN_BLOCK_H */
