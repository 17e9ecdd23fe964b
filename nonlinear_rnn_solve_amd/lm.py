"""Operators that a recurrent language model runs around this package's solves: a gated linear recurrence, layer
normalisation and the log probabilities of given tokens, each with its gradients.

A thin binding over libpararnn_lm.so (C ABI in include/pararnn_lm.h): argument checks and marshalling only.  torch
provides device memory and the current HIP stream; there is no fallback -- if the library or a GPU is missing, calls
raise.  Nothing here synchronises, so calls can be captured in a HIP graph (on a stream that has run the same call
before, so that its workspace is there).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import NamedTuple

import torch

from .api import PararnnError

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpararnn_lm.so")
ABI_VERSION = 1
SCAN_CHUNK = 64           # PARARNN_LM_SCAN_CHUNK
NORM_MAX_D = 16384        # PARARNN_LM_NORM_MAX_D
MAX_TOP = 32              # PARARNN_LM_MAX_TOP

# pararnn_lm_scan and pararnn_lm_scan_grad as the C compiler lays them out
_SCAN = struct.Struct("@if3q3P6qPPPq")
_SCAN_GRAD = struct.Struct("@6P8qPP")
_PAIR = struct.Struct("@2q")

_lib = None


def load_library():
    """Load libpararnn_lm.so (built by ``python -m nonlinear_rnn_solve_amd.build``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("%s not built: run `python -m nonlinear_rnn_solve_amd.build` "
                           "(there is no CPU fallback)" % os.path.basename(LIB_PATH))
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    for name, res, args in (
            ("abi_version", i32, []),
            ("scan_chunks", i64, [i64]),
            ("scan_workspace_bytes", sz, [i64, i64, i64]),
            ("gated_scan", i32, [vp, vp, vp, vp, vp, vp, sz, vp]),
            ("gated_scan_vjp", i32, [vp, vp, vp, sz, vp]),
            ("layer_norm", i32, [i32, i64, i64, vp, i64, vp, i64, vp, vp, f32, vp, i64, vp, i64, vp, vp]),
            ("layer_norm_vjp_workspace_bytes", sz, [i64, i64]),
            ("layer_norm_vjp", i32, [i32, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, vp, sz, vp]),
            ("token_logprobs_workspace_bytes", sz, [i64, i64, i32]),
            ("token_logprobs", i32, [i32, i64, i64, vp, i64, vp, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]),
            ("token_logprobs_vjp", i32, [i32, i64, i64, vp, i64, vp, i32, vp, vp, vp, vp, vp, i64, vp])):
        fn = getattr(lib, "pararnn_lm_" + name)
        fn.restype, fn.argtypes = res, args
    if lib.pararnn_lm_abi_version() != ABI_VERSION:
        raise RuntimeError("%s ABI mismatch" % os.path.basename(LIB_PATH))
    _lib = lib
    return lib


# ---------------------------------------------------------------- checks and marshalling
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_ws_cache: dict = {}
# the raw handle of the current stream and the current device, without building a Stream object for each call
_raw_stream = torch._C._cuda_getCurrentRawStream
_get_device = torch._C._cuda_getDevice


def _workspace(nbytes, index, stream):
    """A cached device workspace per (device, stream), grown on demand: calls on different streams may overlap,
    calls on one stream follow each other."""
    buf = _ws_cache.get((index, stream))
    if buf is None or buf.numel() < nbytes:
        buf = _ws_cache[index, stream] = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=index)
    return buf


def _call(name, device, fn, *args, ws=None):
    """Run the C entry with `device` current; `ws`: the bytes of workspace it takes, before the stream."""
    index = device.index
    if index != _get_device():
        with torch.cuda.device(index):
            return _call(name, device, fn, *args, ws=ws)
    stream = _raw_stream(index)
    if ws is None:
        rc = fn(*args, stream)
    else:
        buf = _workspace(ws, index, stream)
        rc = fn(*args, buf.data_ptr(), buf.numel(), stream)
    if rc != 0:
        raise PararnnError(rc, name)


def _plane(t, name, dtype, shape, device):
    """A tensor of the big planes: its last dimension dense, the others strided as they are."""
    if t.dtype is dtype and t.shape == shape and t.device == device and (t.stride(-1) == 1 or t.shape[-1] <= 1):
        return t
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor (no CPU path exists)" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("all tensors must be on %s (got %s)" % (device, t.device))
    raise ValueError("%s must be dense in its last dimension" % name)


def _dense(t, name, dtype, numel, device):
    """An optional contiguous tensor of `numel` values; its address or None."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == numel and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor (no CPU path exists)" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("all tensors must be on %s (got %s)" % (device, t.device))
    raise ValueError("%s must be contiguous and hold %d values, got %s" % (name, numel, tuple(t.shape)))


def _storage(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a GPU tensor (no CPU path exists)" % name)
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if t.dim() < 1:
        raise ValueError("%s must have at least one dimension" % name)
    return dt


def _rows(t, name):
    """[..., D] as rows of D: their number and stride, without a copy."""
    if t.dim() == 2:
        return t.shape[0], t.stride(0)
    if t.is_contiguous():
        D = t.shape[-1]
        return (t.numel() // D if D else t.shape[:-1].numel()), D
    try:
        v = t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError("%s: its leading dimensions must merge into rows of one stride" % name) from None
    return v.shape[0], v.stride(0)


def _like(t, name, given, shape, device):
    """An output in t's type and shape: `given`, checked, or a new dense tensor."""
    return torch.empty(shape, dtype=t.dtype, device=device) if given is None else _plane(given, name, t.dtype, shape, device)


@functools.lru_cache(maxsize=4096)
def _ws_bytes(entry, *sizes):
    """The C library's answer to a workspace query, which depends on the sizes alone."""
    return getattr(load_library(), "pararnn_lm_%s_workspace_bytes" % entry)(*sizes)


# ---------------------------------------------------------------- gated linear recurrence
def _scan_problem(x, r, i, lam, h0, c, cu_seqlens):
    dt = _storage(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D], got %s" % (tuple(x.shape),))
    dev, shape, dtype = x.device, x.shape, x.dtype
    B, T, D = shape
    _plane(x, "x", dtype, shape, dev)
    _plane(r, "r", dtype, shape, dev)
    _plane(i, "i", dtype, shape, dev)
    n, cu = 1, 0
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a 1-D tensor of n_seqs + 1 offsets")
        n = cu_seqlens.numel() - 1
        cu = _dense(cu_seqlens, "cu_seqlens", torch.int32, n + 1, dev)
    states = (B, n, D)
    if h0 is not None and h0.shape != states and not (cu_seqlens is None and h0.shape == (B, D)):
        raise ValueError("h0 must be %s, got %s" % (states, tuple(h0.shape)))
    xs, rs, si = x.stride(), r.stride(), i.stride()
    prob = _SCAN.pack(dt, c, B, T, D, x.data_ptr(), r.data_ptr(), i.data_ptr(), xs[0], xs[1], rs[0], rs[1], si[0], si[1],
                      _dense(lam, "lam", torch.float32, D, dev) or 0, _dense(h0, "h0", torch.float32, B * n * D, dev) or 0,
                      cu, n)
    return prob, states if cu_seqlens is not None else (B, D)


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
    lib = _lib or load_library()
    prob, states = _scan_problem(x, r, i, lam, h0, c, cu_seqlens)
    B, T, D = shape = x.shape
    dev = x.device
    out = _like(x, "out", out, shape, dev)
    if h_last is None:
        h_last = torch.empty(states if h0 is None else h0.shape, dtype=torch.float32, device=dev)
        last = h_last.data_ptr()
    else:
        last = _dense(h_last, "h_last", torch.float32, torch.Size(states).numel(), dev)
    carry = torch.empty((B, -(-T // SCAN_CHUNK), D), dtype=torch.float32, device=dev) if want_carry else None
    os = out.stride()
    _call("pararnn_lm_gated_scan", dev, lib.pararnn_lm_gated_scan, prob, out.data_ptr(), _PAIR.pack(os[0], os[1]), last,
          carry.data_ptr() if want_carry else None, ws=_ws_bytes("scan", B, T, D))
    return out, h_last, carry


def gated_scan_vjp(x, r, i, lam, carry, dh, h0=None, d_last=None, c=8.0, cu_seqlens=None, out=None, want_lam=True,
                   want_h0=True):
    """Gradients of gated_scan for dh = dL/dh ([B, T, D], x's type) and d_last = dL/dh_last (float32, h0's shape;
    zeros without it), from the carry that gated_scan returned for the same inputs.

    Returns dict: d_x, d_r, d_i [B, T, D] in x's type; d_lam [D] float32 (want_lam); d_h0 float32 (want_h0).
    out: three tensors (d_x, d_r, d_i) to write into, strided as they like (slices of one projection's gradient).
    """
    lib = _lib or load_library()
    prob, states = _scan_problem(x, r, i, lam, h0, c, cu_seqlens)
    B, T, D = x.shape
    dev = x.device
    n = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _plane(dh, "dh", x.dtype, x.shape, dev)
    if carry is None:
        raise ValueError("carry is missing: call gated_scan with want_carry=True")
    pc = _dense(carry, "carry", torch.float32, B * -(-T // SCAN_CHUNK) * D, dev)
    pl = _dense(d_last, "d_last", torch.float32, B * n * D, dev)
    if out is None:
        out = [torch.empty((B, T, D), dtype=x.dtype, device=dev) for _ in range(3)]
    dx, dr, di = (_plane(t, "out[%d]" % k, x.dtype, x.shape, dev) for k, t in enumerate(out))
    d_lam = torch.empty(D, dtype=torch.float32, device=dev) if want_lam else None
    like = h0 if h0 is not None else d_last
    d_h0 = torch.empty(states if like is None else like.shape, dtype=torch.float32, device=dev) if want_h0 else None
    strides = [s for t in (dh, dx, dr, di) for s in t.stride()[:2]]
    grad = _SCAN_GRAD.pack(pc or 0, dh.data_ptr(), pl or 0, dx.data_ptr(), dr.data_ptr(), di.data_ptr(), *strides,
                           d_lam.data_ptr() if want_lam else 0, d_h0.data_ptr() if want_h0 else 0)
    _call("pararnn_lm_gated_scan_vjp", dev, lib.pararnn_lm_gated_scan_vjp, prob, grad,
          ws=_ws_bytes("scan", B, T, D))
    res = {"d_x": dx, "d_r": dr, "d_i": di}
    if want_lam:
        res["d_lam"] = d_lam
    if want_h0:
        res["d_h0"] = d_h0
    return res


# ---------------------------------------------------------------- layer normalisation
def layer_norm(x, weight, bias=None, residual=None, eps=1e-5, want_stats=False, out=None, sum_out=None):
    """Layer normalisation over the last dimension of s = x + residual (rounded to x's type; s = x without one):

        y = (s - mean) / sqrt(var + eps) * weight + bias

    x, residual: [..., D] float32 or bfloat16, D <= NORM_MAX_D, rows of any one stride; weight [D] float32, bias [D]
    float32 or None.  Returns (y, s, stats): y and s in x's shape and type (s is x itself without a residual); stats,
    the float32 [N, 2] that layer_norm_vjp needs, or None without want_stats.
    out, sum_out: tensors for y and s; sum_out may be residual or x itself (the residual stream updated in place).
    """
    lib = _lib or load_library()
    dt = _storage(x, "x")
    dev, shape, dtype = x.device, x.shape, x.dtype
    D = shape[-1]
    N, xs = _rows(_plane(x, "x", dtype, shape, dev), "x")
    y = _like(x, "out", out, shape, dev)
    s, rp, rs, sp, ss = x, None, 0, None, 0
    if residual is not None:
        rs = _rows(_plane(residual, "residual", dtype, shape, dev), "residual")[1]
        s = _like(x, "sum_out", sum_out, shape, dev)
        ss = _rows(s, "sum_out")[1]
        rp, sp = residual.data_ptr(), s.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    stats = torch.empty((N, 2), dtype=torch.float32, device=dev) if want_stats else None
    _call("pararnn_lm_layer_norm", dev, lib.pararnn_lm_layer_norm, dt, N, D, x.data_ptr(), xs, rp, rs,
          _dense(weight, "weight", torch.float32, D, dev), _dense(bias, "bias", torch.float32, D, dev), eps,
          y.data_ptr(), _rows(y, "out")[1], sp, ss, stats.data_ptr() if want_stats else None)
    return y, s, stats


def layer_norm_vjp(dy, s, weight, stats, d_sum=None, out=None, want_params=True):
    """Gradients of layer_norm for dy = dL/dy, from the s and stats that it returned.

    d_sum: what reaches s from elsewhere (the residual path), added to d_x, or None.  Returns dict: d_x in s's shape
    and type (the gradient of x and of the residual alike); with want_params d_weight, d_bias [D] float32.
    out: a tensor for d_x; it may be dy or d_sum itself.
    """
    lib = _lib or load_library()
    dt = _storage(s, "s")
    dev, shape, D = s.device, s.shape, s.shape[-1]
    N, ss = _rows(_plane(s, "s", s.dtype, shape, dev), "s")
    gs = _rows(_plane(dy, "dy", s.dtype, shape, dev), "dy")[1]
    if stats is None:
        raise ValueError("stats are missing: call layer_norm with want_stats=True")
    pp, ps = None, 0
    if d_sum is not None:
        ps = _rows(_plane(d_sum, "d_sum", s.dtype, shape, dev), "d_sum")[1]
        pp = d_sum.data_ptr()
    dx = _like(s, "out", out, shape, dev)
    dw = torch.empty((2, D), dtype=torch.float32, device=dev) if want_params else None
    pw = dw.data_ptr() if want_params else None
    _call("pararnn_lm_layer_norm_vjp", dev, lib.pararnn_lm_layer_norm_vjp, dt, N, D, dy.data_ptr(), gs, s.data_ptr(), ss,
          _dense(weight, "weight", torch.float32, D, dev), _dense(stats, "stats", torch.float32, 2 * N, dev), pp, ps,
          dx.data_ptr(), _rows(dx, "out")[1], pw, pw + 4 * D if want_params else None,
          ws=_ws_bytes("layer_norm_vjp", N, D))
    res = {"d_x": dx}
    if want_params:
        res["d_weight"], res["d_bias"] = dw[0], dw[1]
    return res


# ---------------------------------------------------------------- log probabilities of tokens
class TokenLogprobs(NamedTuple):
    logp: torch.Tensor | None       # [...] float32, None without targets
    entropy: torch.Tensor           # [...] float32
    lse: torch.Tensor               # [...] float32, log of the sum of exponentials
    top_logp: torch.Tensor | None   # [..., top] float32, None for top = 0
    top_ids: torch.Tensor | None    # [..., top] int64


def _targets(targets, lead, dev):
    """(address, bytes of a target), (None, 0) without targets"""
    if targets is None:
        return None, 0
    size = 8 if targets.dtype is torch.int64 else 4
    if size == 4 and targets.dtype is not torch.int32:
        raise ValueError("targets must be int64 or int32, got %s" % targets.dtype)
    if targets.shape != lead:
        raise ValueError("targets must be %s, got %s" % (tuple(lead), tuple(targets.shape)))
    return _dense(targets, "targets", targets.dtype, targets.numel(), dev), size


def token_logprobs(logits, targets=None, top=0):
    """Log probabilities of `targets` under softmax(logits), the distributions' entropies and the `top` (<= MAX_TOP)
    most probable tokens of each row, in descending order, ties by ascending index.

    logits: [..., V] float32 or bfloat16, rows of any one stride (-inf rules a token out; a row with nothing left has
    logp -inf, entropy 0); targets: [...] int64 or int32, a negative one scores nothing (logp 0), one at or above V
    gives NaN; None: no logp.  Returns TokenLogprobs.
    """
    lib = _lib or load_library()
    dt = _storage(logits, "logits")
    dev, shape = logits.device, logits.shape
    lead, V = shape[:-1], shape[-1]
    N, zs = _rows(_plane(logits, "logits", logits.dtype, shape, dev), "logits")
    tp, tb = _targets(targets, lead, dev)
    if not 0 <= top <= min(V, MAX_TOP):
        raise ValueError("top must be in 0 .. min(V, %d) = %d, got %d" % (MAX_TOP, min(V, MAX_TOP), top))
    lse, entropy, logp = torch.empty((3,) + lead, dtype=torch.float32, device=dev).unbind(0)
    top_logp = top_ids = pl = pi = None
    if top:
        top_logp = torch.empty(lead + (top,), dtype=torch.float32, device=dev)
        top_ids = torch.empty(lead + (top,), dtype=torch.int64, device=dev)
        pl, pi = top_logp.data_ptr(), top_ids.data_ptr()
    _call("pararnn_lm_token_logprobs", dev, lib.pararnn_lm_token_logprobs, dt, N, V, logits.data_ptr(), zs, tp, tb,
          lse.data_ptr(), logp.data_ptr() if tb else None, entropy.data_ptr(), top, pl, pi,
          ws=_ws_bytes("token_logprobs", N, V, top))
    return TokenLogprobs(logp if tb else None, entropy, lse, top_logp, top_ids)


def token_logprobs_vjp(logits, targets, lse, entropy, g_logp, g_entropy=None, out=None):
    """Gradient with respect to logits of sum(g_logp * logp + g_entropy * entropy), from the lse and entropy that
    token_logprobs returned; g_logp, g_entropy float32 in lse's shape (g_entropy may be None).  The top alternatives
    are reports and have no gradient.  Returns [..., V] in logits' type; out: a tensor for it, logits itself allowed.
    """
    lib = _lib or load_library()
    dt = _storage(logits, "logits")
    dev, shape = logits.device, logits.shape
    V = shape[-1]
    N, zs = _rows(_plane(logits, "logits", logits.dtype, shape, dev), "logits")
    tp, tb = _targets(targets, shape[:-1], dev)
    if tb and g_logp is None:
        raise ValueError("g_logp is missing")
    if g_entropy is not None and entropy is None:
        raise ValueError("entropy is missing")
    dz = _like(logits, "out", out, shape, dev)
    _call("pararnn_lm_token_logprobs_vjp", dev, lib.pararnn_lm_token_logprobs_vjp, dt, N, V, logits.data_ptr(), zs, tp, tb,
          _dense(lse, "lse", torch.float32, N, dev), _dense(entropy, "entropy", torch.float32, N, dev),
          _dense(g_logp, "g_logp", torch.float32, N, dev) if tb else None,
          _dense(g_entropy, "g_entropy", torch.float32, N, dev), dz.data_ptr(), _rows(dz, "out")[1])
    return dz
