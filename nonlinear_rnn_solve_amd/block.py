"""What a recurrent language model's block and its training step are made of beside the operators of ``lm``: a short causal
convolution, the selective state space scan, a gated feed-forward product, each with its gradients, and an AdamW step over
many tensors.

The kernels are libpararnn_block.so (C ABI in include/pararnn_block.h); a compiled binding checks the arguments, allocates
the results with torch and passes the current HIP stream.  As in ``lm``, there is no fallback, wrong tensors raise
ValueError, statuses of the C ABI PararnnError; big planes are float32 or bfloat16, dense in their last dimension and strided
as they like in the others; float32 arguments (states, parameters) are contiguous and of the stated shape, dimensions of one
entry aside, or flat; results are detached from autograd (examples/selective_lm.py wraps the operators in autograd functions) and a
tensor given to be written counts as modified in place; it shares no memory with an input or another output unless its operator
says so (ValueError where both are dense and overlap or begin at the same place; interleaved views are not told apart).  Nothing here synchronises, so calls can be captured in a HIP graph.
"""
from __future__ import annotations

import importlib
import os
import sysconfig

from .api import PararnnError  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpararnn_block.so")
BINDING_PATH = os.path.join(_HERE, "_block_binding" + sysconfig.get_config_var("EXT_SUFFIX"))   # of this interpreter
ABI_VERSION = 1           # PARARNN_BLOCK_ABI_VERSION
MAX_TAPS = 8              # PARARNN_BLOCK_MAX_TAPS
MAX_STATES = 32           # PARARNN_BLOCK_MAX_STATES
SSM_CHUNK = 16            # PARARNN_BLOCK_SSM_CHUNK
ADAMW_BLOCK = 256         # PARARNN_BLOCK_ADAMW_BLOCK

_binding = None


def load_library():
    """Load libpararnn_block.so and its binding (built by ``python -m nonlinear_rnn_solve_amd.build``); raises if absent."""
    global _binding
    if _binding is None:
        for path in (LIB_PATH, BINDING_PATH):
            if not os.path.exists(path):
                raise RuntimeError("%s not built: run `python -m nonlinear_rnn_solve_amd.build` "
                                   "(there is no CPU fallback)" % os.path.basename(path))
        b = importlib.import_module("._block_binding", __package__)
        if not b.abi_version() == b.ABI_VERSION == ABI_VERSION:
            raise RuntimeError("%s ABI mismatch" % os.path.basename(LIB_PATH))
        _binding = b
    return _binding


# ---------------------------------------------------------------- short causal convolution
def causal_conv(x, weight, bias=None, state=None, cu_seqlens=None, silu=True, out=None, last=None):
    """Causal convolution along T of each channel by itself, K taps:

        p_t = bias + sum_k weight[:, k] x_{t-K+1+k},  y_t = p_t sigmoid(p_t)   (y_t = p_t without silu)

    x: [B, T, D]; weight [D, K] float32, K <= MAX_TAPS; bias [D] float32 or None.  state: float32 [B, K-1, D], the steps
    before the rows, oldest first; zeros without it.  cu_seqlens: int32 [n_seqs + 1] offsets of sequences packed along T
    (every row); state is then [B, n_seqs, K-1, D], and a sequence may be empty.
    Returns (y, last): y [B, T, D] in x's type; last, in state's shape, the last K-1 steps of state and sequence together.
    out, last: tensors to write into; last may be state itself (a decoder's state updated in place).
    """
    return (_binding or load_library()).causal_conv(x, weight, bias, state, cu_seqlens, silu, out, last)


def causal_conv_vjp(x, weight, dy, bias=None, state=None, d_last=None, cu_seqlens=None, silu=True, out=None, want_params=True,
                    want_state=True):
    """Gradients of causal_conv for dy = dL/dy (x's shape and type) and d_last = dL/dlast (float32; zeros without it).

    Returns dict: d_x [B, T, D] in x's type; d_weight [D, K], d_bias [D] float32 (want_params); d_state float32 (want_state).
    out: a tensor for d_x.
    """
    return (_binding or load_library()).causal_conv_vjp(x, weight, dy, bias, state, d_last, cu_seqlens, silu, out, want_params,
                                                        want_state)


# ---------------------------------------------------------------- selective state space scan
def selective_scan(x, dt, A, b, c, skip=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, want_carry=False, out=None,
                   h_last=None):
    """Selective state space scan along T.  For channel d of group g and state n:

        s_t = softplus(dt_t + dt_bias),  h_t[n] = exp(s_t A[n]) h_{t-1}[n] + s_t x_t b_t[g, n]
        y_t = (sum_n c_t[g, n] h_t[n] + skip x_t) z_t sigmoid(z_t)

    x, dt, z: [B, T, D] (z None: no gate); A [D, N] float32, N <= MAX_STATES; b, c: [B, T, N] or, for G groups of D / G
    consecutive channels each, [B, T, G, N], in x's type; skip, dt_bias [D] float32 or None.
    h0: float32 states entering the rows, [B, D, N]; zeros without it.  cu_seqlens as in causal_conv; h0 is then
    [B, n_seqs, D, N].  Returns (y, h_last, carry): y [B, T, D] in x's type; h_last, the float32 states leaving the
    sequences, in h0's shape; carry, what selective_scan_vjp needs (float32 [B, chunks, N, D], or None without want_carry).
    out, h_last: tensors to write into; h_last may be h0 itself (a decoder's state updated in place).
    Steps of any plane are less than 2^24 elements apart (PararnnError otherwise).
    """
    return (_binding or load_library()).selective_scan(x, dt, A, b, c, skip, z, dt_bias, h0, cu_seqlens, want_carry, out, h_last)


def selective_scan_vjp(x, dt, A, b, c, carry, dy, skip=None, z=None, dt_bias=None, h0=None, d_last=None, cu_seqlens=None, out=None,
                       want_params=True, want_h0=True):
    """Gradients of selective_scan for dy = dL/dy (x's shape and type) and d_last = dL/dh_last (float32, h0's shape; zeros
    without it), from the carry that selective_scan returned for the same inputs.

    Returns dict: d_x, d_dt, d_z (with z) [B, T, D], d_b, d_c in b's shape, in x's type; d_A [D, N], d_skip, d_dt_bias [D]
    float32 (want_params); d_h0 float32 (want_h0).
    out: five tensors or None (d_x, d_dt, d_z, d_b, d_c) to write into, strided as they like.
    A channel with a rate A of -inf has a d_dt and d_dt_bias of NaN; the other gradients are finite.
    """
    return (_binding or load_library()).selective_scan_vjp(x, dt, A, b, c, carry, dy, skip, z, dt_bias, h0, d_last, cu_seqlens, out,
                                                           want_params, want_h0)


# ---------------------------------------------------------------- gated feed-forward product
def gated_linear(x, w_gate, w_up, activation="silu", want_pre=False, out=None):
    """A gated feed-forward block's two projections, its activation and their product, in one kernel:

        h = act(x w_gate^T) * (x w_up^T)

    x: [..., D], rows of any one stride; w_gate, w_up: [F, D] in x's type (two halves of one tensor, for instance);
    activation: "silu" or "gelu" (its tanh form).  Products are summed in float32 (an infinity among float32 values makes the
    results it enters infinite or NaN, by the sizes).
    Returns (h, pre): h [..., F] in x's type; pre, float32 [rows, 2 F], what gated_linear_vjp needs, or None without
    want_pre.  out: a tensor for h.
    """
    return (_binding or load_library()).gated_linear(x, w_gate, w_up, activation, want_pre, out)


def gated_linear_vjp(x, w_gate, w_up, pre, dh, activation="silu", want_x=True, want_params=True, out=None, w_out=None):
    """Gradients of gated_linear for dh = dL/dh ([..., F], x's type), from the pre that it returned.

    The gradients of the two projections' results are not rounded to x's type before they are multiplied: in bfloat16 each is
    held as a sum of two bfloat16, within 2^-16 of it.
    Returns dict, all in x's type: d_x in x's shape (want_x); d_w_gate, d_w_up [F, D] (want_params).
    out: a tensor for d_x; w_out: two tensors or None for d_w_gate and d_w_up, rows of any stride.
    """
    return (_binding or load_library()).gated_linear_vjp(x, w_gate, w_up, pre, dh, activation, want_x, want_params, out, w_out)


# ---------------------------------------------------------------- AdamW
def adamw_state_size(params):
    """Elements of the moments of a list of tensors: each tensor's begin at a multiple of ADAMW_BLOCK, in order."""
    return (_binding or load_library()).adamw_state_size(params)


def adamw_step(params, grads, m, v, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, grad_scale=1.0, m_scale=None,
               v_scale=None, seed=0):
    """One AdamW step over a list of tensors, in place.  With g' = grad_scale g:

        m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
        p = p (1 - lr weight_decay) - lr (m / (1 - b1^step)) / (sqrt(v / (1 - b2^step)) + eps)

    params, grads: contiguous tensors, float32 or bfloat16 each (a bfloat16 parameter is rounded to nearest); no two
    parameters may overlap.  m, v: the moments of all tensors, adamw_state_size(params) elements (zeros at the start),
    float32 or, in 8 bits, uint8; then m_scale, v_scale are float32, one value for each ADAMW_BLOCK elements, and a moment
    is rounded up or down at random so that its mean is kept, by a hash of seed, step and the element's place.
    step: 1 for the first; step (int64), lr and grad_scale (float32) may each be a GPU tensor of one element, which a captured
    graph reads at each replay.
    """
    (_binding or load_library()).adamw_step(params, grads, m, v, step, lr, betas, eps, weight_decay, grad_scale, m_scale, v_scale,
                                            seed)


def adamw_moments(m, v, m_scale, v_scale):
    """(m, v) of 8-bit moments as the values that their codes stand for, in bfloat16, which holds them exactly."""
    return (_binding or load_library()).adamw_moments(m, v, m_scale, v_scale)
