/*
 * pararnn_lm.h -- C ABI of libpararnn_lm.so: the operators that a recurrent language model runs around the
 * solves of pararnn.h, on MI355X (gfx950): a gated linear recurrence, layer normalisation and the log
 * probabilities of given tokens, each with its gradients.
 *
 * Conventions are those of pararnn.h (device pointers, status codes, asynchronous on `stream`, arguments
 * checked before anything is launched, nothing thrown, no allocation, no synchronisation, capturable in a HIP
 * graph, a 256-byte aligned workspace of the queried size whose contents need not be initialised), with
 * these differences:
 *  - Planes may be strided: the last dimension is dense, the strides of the others are arguments, counted in
 *    elements (nonnegative; they may exceed 32 bits).  Outputs must not overlap inputs unless an entry
 *    says so.
 *  - `dtype` (pararnn_dtype) is the storage type of the big planes, float32 or bfloat16.  Arithmetic, states,
 *    statistics, parameters and their gradients are float32; an output in bfloat16 is rounded once, to the
 *    nearest even.
 *  - Sizes of any value are accepted (odd ones included); pointers need the alignment of their element type
 *    only.
 *  - Every result is a fixed sequence of operations on its inputs: it is the same bits in every run.
 */
#ifndef PARARNN_LM_H
#define PARARNN_LM_H

#include "pararnn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PARARNN_LM_ABI_VERSION 1

/* ------------------------------------------------------------------------------------------------
 * Gated linear recurrence.  For every batch row b, channel d and step t:
 *     a_t = exp(-c softplus(lam) sig(r_t)),     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(i_t) x_t
 * (sig(r) opens the decay, sig(i) the input; the square root keeps the state's variance).  It is solved by a
 * parallel scan along time, whatever T is; T <= 16 runs without one, in a single launch (one generated token is
 * T = 1).  UNSUPPORTED: 2^24 or more tiles of 64 channels by PARARNN_LM_SCAN_CHUNK steps.
 * ---------------------------------------------------------------------------------------------- */
/* steps of one chunk of the scan (the state entering each is what the gradient rebuilds h from) */
#define PARARNN_LM_SCAN_CHUNK 64

typedef struct {
  int32_t dtype;             /* of x, r, i, h and, in the gradient, dh, d_x, d_r, d_i                   */
  float c;                   /* decay scale, finite and positive                                        */
  int64_t B, T, D;           /* each >= 0; an empty problem writes h_last = h0 (or zeros)               */
  const void *x, *r, *i;     /* [B][T][D] values and the two gates' pre-activations                     */
  int64_t sx[2], sr[2], si[2]; /* their strides over b and t                                            */
  const float* lam;          /* [D]                                                                     */
  const float* h0;           /* [B][n][D] state entering each sequence, dense, n = 1 without cu_seqlens, else
                                n_seqs; NULL = zeros                                                    */
  const int32_t* cu_seqlens; /* NULL: one sequence per row.  Else n_seqs + 1 nondecreasing offsets (device):
                                sequence j is steps cu[j] .. cu[j+1]-1 of every row, cu[0] is read as 0 and
                                cu[n_seqs] as T.  Nothing flows from one sequence to the next, NaN and
                                infinities included.  A sequence may be empty.  The offsets are not checked
                                (they are device memory); wrong ones give wrong numbers, no access outside
                                the arrays.                                                             */
  int64_t n_seqs;            /* >= 1 with cu_seqlens, ignored without                                   */
} pararnn_lm_scan;

/* chunks of a row of T steps: the middle size of `carry` */
int64_t pararnn_lm_scan_chunks(int64_t T);
/* one size for both calls; 0 for invalid sizes */
size_t pararnn_lm_scan_workspace_bytes(int64_t B, int64_t T, int64_t D);

/*   h       [B][T][D] of dtype, strides sh
 *   h_last  [B][n][D] float32: the state leaving each sequence (h0 where it is empty), or NULL; it may be
 *           the array h0 itself (a decoder's state updated in place)
 *   carry   [B][chunks][D] float32: the state entering each chunk, which the gradient needs, or NULL      */
pararnn_status pararnn_lm_gated_scan(const pararnn_lm_scan* prob, void* h, const int64_t sh[2], float* h_last,
                                     float* carry, void* ws, size_t ws_bytes, void* stream);

/* Gradients.  With l_t = dh_t + a_{t+1} l_{t+1} (plus d_last at a sequence's last step), u = sig(i) x,
 * m = sqrt(1 - a^2), k = -c softplus(lam), e_t = l_t (a_t h_{t-1} - u_t a_t^2 / m_t) (0 for the quotient where m_t = 0):
 *     d_r = e k sig(r) (1 - sig(r)),  d_i = l m u (1 - sig(i)),  d_x = l m sig(i),
 *     d_lam = -c sig(lam) sum_{b,t} e sig(r),  d_h0 = a_t l_t at a sequence's first step (d_last where it is empty).
 *   carry   as pararnn_lm_gated_scan wrote it for the same problem
 *   dh      [B][T][D] of dtype, strides sdh;  d_last [B][n][D] float32 or NULL (zeros)
 *   d_x, d_r, d_i  [B][T][D] of dtype, strides sdx, sdr, sdi (three slices of one array, for instance)
 *   d_lam   [D] float32 or NULL;  d_h0 [B][n][D] float32 or NULL                                       */
typedef struct {
  const float* carry;
  const void* dh;
  const float* d_last;
  void *d_x, *d_r, *d_i;
  int64_t sdh[2], sdx[2], sdr[2], sdi[2];
  float *d_lam, *d_h0;
} pararnn_lm_scan_grad;
pararnn_status pararnn_lm_gated_scan_vjp(const pararnn_lm_scan* prob, const pararnn_lm_scan_grad* grad, void* ws,
                                         size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Layer normalisation of N rows of D channels (D <= PARARNN_LM_NORM_MAX_D, else UNSUPPORTED; so
 * is N above 2^28 - 16, 2^26 - 4 where D > 256, 2^24 - 1 where D > 1024, 2^22 - 1 where D > 4096):
 *     s = x + residual (rounded to dtype; s = x without one),  mean and variance of each row of s,
 *     y = (s - mean) / sqrt(var + eps) * weight + bias
 *   x, residual (or NULL), y, sum  [N][D] of dtype with row strides; weight [D], bias [D] or NULL float32
 *   sum     the rounded s; required with a residual, must be NULL without; it may be x or residual itself
 *   stats   [N][2] float32 (mean, 1 / sqrt(var + eps)) for the gradient, or NULL; not written where D = 0
 * ---------------------------------------------------------------------------------------------- */
#define PARARNN_LM_NORM_MAX_D 16384
pararnn_status pararnn_lm_layer_norm(int dtype, int64_t N, int64_t D, const void* x, int64_t x_stride,
                                     const void* residual, int64_t residual_stride, const float* weight,
                                     const float* bias, float eps, void* y, int64_t y_stride, void* sum,
                                     int64_t sum_stride, float* stats, void* stream);

/* Gradients.  n = (s - mean) rstd, g = dy weight:
 *     d_x = rstd (g - mean(g) - n mean(g n)) + d_sum,  d_weight = sum_rows dy n,  d_bias = sum_rows dy
 *   s       the normalised input (the forward's sum, or x without a residual);  stats as the forward wrote them
 *   d_sum   [N][D] gradient that reaches s from elsewhere (the residual path), or NULL
 *   d_x     [N][D] of dtype (it is the gradient of x and of the residual alike); it may be dy or d_sum itself
 *   d_weight, d_bias  [D] float32, each or both may be NULL                                             */
size_t pararnn_lm_layer_norm_vjp_workspace_bytes(int64_t N, int64_t D);
pararnn_status pararnn_lm_layer_norm_vjp(int dtype, int64_t N, int64_t D, const void* dy, int64_t dy_stride,
                                         const void* s, int64_t s_stride, const float* weight, const float* stats,
                                         const void* d_sum, int64_t d_sum_stride, void* d_x, int64_t d_x_stride,
                                         float* d_weight, float* d_bias, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Log probabilities of given tokens: for each of N rows of V logits z (V < 2^31), p = softmax(z):
 *     lse = ln sum_j e^{z_j},  logp = z_target - lse,  entropy = -sum_j p_j ln p_j (0 for p_j = 0)
 * and the `top` largest logits in descending order, ties by ascending index (0 <= top <= min(V, PARARNN_LM_MAX_TOP)).
 *   targets [N] int32 or int64 (target_bytes 4 or 8).  A negative one means that no token is scored: logp = 0.
 *           One at or above V gives logp = NaN.
 *   lse, logp, entropy [N] float32: lse and entropy may be NULL; logp is given with targets and NULL without;
 *   top_logp [N][top] float32, top_ids [N][top] int64 (NULL when top = 0)
 *   ws      of the queried size and aligned like any other; nothing is kept there at present
 * UNSUPPORTED: N of 2^26 or more, 2^24 where V > 4096, 2^22 where V > 32768.
 * Logits of -infinity are tokens ruled out.  A row with nothing left has lse = -infinity, logp = -infinity,
 * entropy = 0 and a gradient of zeros.  A NaN or +infinity makes its row's numbers NaN; a NaN ranks as -infinity.
 * ---------------------------------------------------------------------------------------------- */
#define PARARNN_LM_MAX_TOP 32
size_t pararnn_lm_token_logprobs_workspace_bytes(int64_t N, int64_t V, int top);
pararnn_status pararnn_lm_token_logprobs(int dtype, int64_t N, int64_t V, const void* logits, int64_t stride,
                                         const void* targets, int target_bytes, float* lse, float* logp,
                                         float* entropy, int top, float* top_logp, int64_t* top_ids, void* ws,
                                         size_t ws_bytes, void* stream);

/* Gradient of sum_n g_logp logp + g_entropy entropy (logp of a negative target has none; the top alternatives
 * are reports and have none):
 *     d_z_j = g_logp (1[j = target] - p_j) - g_entropy p_j (ln p_j + entropy)
 *   lse, entropy as the forward wrote them (entropy may be NULL when g_entropy is).  p does not carry the rounding of lse:
 *           rows with |lse| > 32 are read once more, and their normaliser is summed about lse.  An lse that differs from
 *           the row's by more than rounding (that of a longer row, of which these logits are a part) is used as it is
 *   g_logp [N] float32 (NULL with targets NULL), g_entropy [N] float32 or NULL
 *   d_logits [N][V] of dtype, row stride d_stride; it may be logits itself (same stride)                */
pararnn_status pararnn_lm_token_logprobs_vjp(int dtype, int64_t N, int64_t V, const void* logits, int64_t stride,
                                             const void* targets, int target_bytes, const float* lse,
                                             const float* entropy, const float* g_logp, const float* g_entropy,
                                             void* d_logits, int64_t d_stride, void* stream);

/* PARARNN_LM_ABI_VERSION of the built library */
int pararnn_lm_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* PARARNN_LM_H */
