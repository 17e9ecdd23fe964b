"""Operators that a recurrent language model runs around this package's solves: a gated linear recurrence, layer
normalisation and the log probabilities of given tokens, each with its gradients.

The kernels are libpararnn_lm.so (C ABI in include/pararnn_lm.h); a compiled binding checks the arguments, allocates the
results with torch and passes the current HIP stream.  There is no fallback -- if a library or a GPU is missing, calls
raise.  Wrong tensors raise ValueError, statuses of the C ABI PararnnError.  Float32 arguments (states, statistics,
per-token numbers, parameters) are contiguous and of the stated shape, dimensions of one entry aside, or flat.  Results are
detached from autograd (examples/gated_lm.py wraps the operators in autograd functions); a tensor given to be written
counts as modified in place.  Nothing here synchronises, so calls can be captured in a HIP graph (torch.cuda.graph; a
captured call's workspace belongs to the graph).
"""
from __future__ import annotations

import importlib
import os
import sysconfig
from typing import NamedTuple

import torch

from .api import PararnnError  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpararnn_lm.so")
BINDING_PATH = os.path.join(_HERE, "_lm_binding" + sysconfig.get_config_var("EXT_SUFFIX"))   # of this interpreter
ABI_VERSION = 1           # PARARNN_LM_ABI_VERSION
SCAN_CHUNK = 64           # PARARNN_LM_SCAN_CHUNK
NORM_MAX_D = 16384        # PARARNN_LM_NORM_MAX_D
MAX_TOP = 32              # PARARNN_LM_MAX_TOP

_binding = None


def load_library():
    """Load libpararnn_lm.so and its binding (built by ``python -m nonlinear_rnn_solve_amd.build``); raises if absent."""
    global _binding
    if _binding is None:
        for path in (LIB_PATH, BINDING_PATH):
            if not os.path.exists(path):
                raise RuntimeError("%s not built: run `python -m nonlinear_rnn_solve_amd.build` "
                                   "(there is no CPU fallback)" % os.path.basename(path))
        b = importlib.import_module("._lm_binding", __package__)
        if not b.abi_version() == b.ABI_VERSION == ABI_VERSION:
            raise RuntimeError("%s ABI mismatch" % os.path.basename(LIB_PATH))
        _binding = b
    return _binding


# ---------------------------------------------------------------- gated linear recurrence
def gated_scan(x, r, i, lam, h0=None, c=8.0, cu_seqlens=None, want_carry=False, out=None, h_last=None):
    """Gated linear recurrence along T, by a parallel scan:

        a_t = exp(-c softplus(lam) sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t

    x, r, i: [B, T, D] float32 or bfloat16, dense along D (three slices of one projection, for instance); lam [D]
    float32.  h0: float32 state entering the rows, [B, D] (or [B, 1, D]); zeros without it.
    cu_seqlens: int32 [n_seqs + 1] offsets of sequences packed along T (every row); h0 is then [B, n_seqs, D],
    nothing flows from one sequence to the next, and a sequence may be empty.
    Returns (h, h_last, carry): h [B, T, D] in x's type; h_last, the float32 states leaving the sequences, in h0's
    shape; carry, what gated_scan_vjp needs (float32 [B, chunks, D], or None without want_carry).
    out, h_last: tensors to write into; h_last may be h0 itself (a decoder's state updated in place).
    """
    return (_binding or load_library()).gated_scan(x, r, i, lam, h0, c, cu_seqlens, want_carry, out, h_last)


def gated_scan_vjp(x, r, i, lam, carry, dh, h0=None, d_last=None, c=8.0, cu_seqlens=None, out=None, want_lam=True,
                   want_h0=True):
    """Gradients of gated_scan for dh = dL/dh ([B, T, D], x's type) and d_last = dL/dh_last (float32, h0's shape;
    zeros without it), from the carry that gated_scan returned for the same inputs.

    Returns dict: d_x, d_r, d_i [B, T, D] in x's type; d_lam [D] float32 (want_lam); d_h0 float32 (want_h0).
    out: three tensors (d_x, d_r, d_i) to write into, strided as they like (slices of one projection's gradient).
    """
    return (_binding or load_library()).gated_scan_vjp(x, r, i, lam, carry, dh, h0, d_last, c, cu_seqlens, out, want_lam,
                                                       want_h0)


# ---------------------------------------------------------------- layer normalisation
def layer_norm(x, weight, bias=None, residual=None, eps=1e-5, want_stats=False, out=None, sum_out=None):
    """Layer normalisation over the last dimension of s = x + residual (rounded to x's type; s = x without one):

        y = (s - mean) / sqrt(var + eps) * weight + bias

    x, residual: [..., D] float32 or bfloat16, D <= NORM_MAX_D, rows of any one stride; weight [D] float32, bias [D]
    float32 or None.  Returns (y, s, stats): y and s in x's shape and type (s is x itself without a residual); stats,
    the float32 [N, 2] that layer_norm_vjp needs, or None without want_stats.
    out, sum_out: tensors for y and s; sum_out may be residual or x itself (the residual stream updated in place).
    """
    return (_binding or load_library()).layer_norm(x, weight, bias, residual, eps, want_stats, out, sum_out)


def layer_norm_vjp(dy, s, weight, stats, d_sum=None, out=None, want_params=True):
    """Gradients of layer_norm for dy = dL/dy, from the s and stats that it returned.

    d_sum: what reaches s from elsewhere (the residual path), added to d_x, or None.  Returns dict: d_x in s's shape
    and type (the gradient of x and of the residual alike); with want_params d_weight, d_bias [D] float32.
    out: a tensor for d_x; it may be dy or d_sum itself.
    """
    return (_binding or load_library()).layer_norm_vjp(dy, s, weight, stats, d_sum, out, want_params)


# ---------------------------------------------------------------- log probabilities of tokens
class TokenLogprobs(NamedTuple):
    logp: torch.Tensor | None       # [...] float32, None without targets
    entropy: torch.Tensor           # [...] float32
    lse: torch.Tensor               # [...] float32, log of the sum of exponentials
    top_logp: torch.Tensor | None   # [..., top] float32, None for top = 0
    top_ids: torch.Tensor | None    # [..., top] int64


def token_logprobs(logits, targets=None, top=0):
    """Log probabilities of `targets` under softmax(logits), the distributions' entropies and the `top` (<= MAX_TOP)
    most probable tokens of each row, in descending order, ties by ascending index.

    logits: [..., V] float32 or bfloat16, rows of any one stride (-inf rules a token out; a row with nothing left has
    logp -inf, entropy 0); targets: [...] int64 or int32, a negative one scores nothing (logp 0), one at or above V
    gives NaN; None: no logp.  Returns TokenLogprobs.
    """
    return TokenLogprobs._make((_binding or load_library()).token_logprobs(logits, targets, top))


def token_logprobs_vjp(logits, targets, lse, entropy, g_logp, g_entropy=None, out=None):
    """Gradient with respect to logits of sum(g_logp * logp + g_entropy * entropy), from the lse and entropy that
    token_logprobs returned; g_logp, g_entropy float32 in lse's shape (g_entropy may be None).  The top alternatives
    are reports and have no gradient.  An offset that a row's logits have in common costs no accuracy, but time (rows with
    |lse| > 32 are read twice).  Returns [..., V] in logits' type; out: a tensor for it, logits itself allowed.
    """
    return (_binding or load_library()).token_logprobs_vjp(logits, targets, lse, entropy, g_logp, g_entropy, out)
