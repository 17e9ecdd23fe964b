"""Plain 64-bit forms of the block operators (CPU, one step after the other), written from the formulas in
include/pararnn_block.h, for the tests.  All but the optimizer's support torch's autograd."""
import math

import torch

from lm_plain import U32, f64, sequences


def silu(p):
    return p / (1 + torch.exp(-p))


def gelu(g):
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def conv(x, weight, bias=None, state=None, cu=None, act=True):
    """(y [B, T, D], last [B, n, K-1, D])."""
    B, T, D = x.shape
    K = weight.shape[1]
    ys, lasts = [], []
    n = len(sequences(cu, T))
    for j, (t0, t1) in enumerate(sequences(cu, T)):
        head = torch.zeros(B, K - 1, D, dtype=torch.float64) if state is None else state.reshape(B, n, K - 1, D)[:, j]
        ext = torch.cat([head, x[:, t0:t1]], 1)
        for t in range(t1 - t0):
            ys.append((ext[:, t:t + K] * weight.t()).sum(1))
        lasts.append(ext[:, t1 - t0:])
    y = torch.stack(ys, 1) if ys else torch.zeros(B, 0, D, dtype=torch.float64)
    if bias is not None:
        y = y + bias
    return (silu(y) if act else y), torch.stack(lasts, 1)


def ssm(x, dt, A, b, c, skip=None, z=None, dt_bias=None, h0=None, cu=None):
    """(y [B, T, D], h_last [B, n, D, N])."""
    B, T, D = x.shape
    N = A.shape[1]
    b, c = (t.reshape(B, T, -1, N) for t in (b, c))
    b, c = (t.repeat_interleave(D // t.shape[2], 2) for t in (b, c))
    s = torch.nn.functional.softplus(dt if dt_bias is None else dt + dt_bias, threshold=700.0)
    ys, last = [], []
    n = len(sequences(cu, T))
    for j, (t0, t1) in enumerate(sequences(cu, T)):
        h = torch.zeros(B, D, N, dtype=torch.float64) if h0 is None else h0.reshape(B, n, D, N)[:, j]
        for t in range(t0, t1):
            h = torch.exp(s[:, t, :, None] * A) * h + (s[:, t] * x[:, t])[..., None] * b[:, t]
            ys.append((c[:, t] * h).sum(-1))
        last.append(h)
    y = torch.stack(ys, 1) if ys else torch.zeros(B, 0, D, dtype=torch.float64)
    if skip is not None:
        y = y + skip * x
    return (y if z is None else y * silu(z)), torch.stack(last, 1)


def gated(x, w_gate, w_up, activation="silu"):
    return {"silu": silu, "gelu": gelu}[activation](x @ w_gate.t()) * (x @ w_up.t())


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after a step."""
    g = g * grad_scale
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    u = (m / (1 - betas[0] ** step)) / (torch.sqrt(v / (1 - betas[1] ** step)) + eps)
    return p * (1 - lr * weight_decay) - lr * u, m, v


def values(bias):
    """What the codes 0 .. 255 stand for at a scale of 1 (bias 15: with a sign; 31: without)."""
    out = []
    for code in range(256):
        q = code & 127 if bias == 15 else code
        e, f = q >> 3, q & 7
        x = (1 + f / 8) * 2.0 ** (e - bias) if e else f / 8 * 2.0 ** (1 - bias)
        out.append(-x if bias == 15 and code > 127 else x)
    return torch.tensor(out, dtype=torch.float64)


def grads(outs, wants, leaves):
    """Gradients of sum(out * want) with respect to the leaves (None stays None, unused ones are zeros)."""
    loss = sum((o * w).sum() for o, w in zip(outs, wants) if w is not None) + 0 * sum(t.sum() for t in leaves if t is not None)
    some = [t for t in leaves if t is not None]
    got = iter(torch.autograd.grad(loss, some))
    return [None if t is None else next(got) for t in leaves]


def leaf(t):
    return None if t is None else f64(t).requires_grad_()


def biggest(t):
    return float(t.detach().abs().max()) if t.numel() else 0.0


__all__ = ["U32", "f64"]
