"""Plain 64-bit forms of the language-model operators (CPU, one step after the other), written from the formulas in
include/pararnn_lm.h, for the tests.  All of them support torch's autograd."""
import torch

U32 = 2.0 ** -24      # unit roundoff of float32
U16 = 2.0 ** -8       # unit roundoff of bfloat16 (8 significant bits, to nearest)


def f64(t):
    return None if t is None else t.detach().cpu().double()


def sequences(cu, T):
    """[(t0, t1)] of a row's sequences: the first begins at 0, the last ends at T."""
    if cu is None:
        return [(0, T)]
    cu = [int(v) for v in cu]
    return list(zip([0] + cu[1:-1], cu[1:-1] + [T]))


def scan(x, r, i, lam, h0=None, c=8.0, cu=None):
    """(h [B, T, D], h_last [B, n, D]) of the gated linear recurrence."""
    B, T, D = x.shape
    rate = c * torch.nn.functional.softplus(lam, threshold=700.0)
    log_a = -rate * torch.sigmoid(r)
    a, m = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    v = m * torch.sigmoid(i) * x
    hs, last = [], []
    for j, (t0, t1) in enumerate(sequences(cu, T)):
        h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.reshape(B, -1, D)[:, j]
        for t in range(t0, t1):
            h = a[:, t] * h + v[:, t]
            hs.append(h)
        last.append(h)
    return (torch.stack(hs, 1) if hs else torch.zeros(B, 0, D, dtype=torch.float64)), torch.stack(last, 1)


def scan_decays(r, lam, c=8.0):
    """(smallest 1 - a) of a problem, from which the memory length follows"""
    q = -torch.expm1(-c * torch.nn.functional.softplus(lam, threshold=700.0) * torch.sigmoid(r))
    return float(q.min()) if q.numel() else 1.0


def norm(x, weight, bias=None, residual=None, eps=1e-5, dtype=torch.float64):
    """(y, s): s = x + residual rounded to `dtype`."""
    s = x if residual is None else (x + residual).to(dtype).double()
    mean = s.mean(-1, keepdim=True)
    y = (s - mean) / torch.sqrt(((s - mean) ** 2).mean(-1, keepdim=True) + eps) * weight
    return (y if bias is None else y + bias), s


def logp(z, targets):
    """(logp, entropy, lse) of rows with at least one token left; targets < 0 score 0."""
    lse = torch.logsumexp(z, -1)
    l = z - lse[..., None]
    p = torch.exp(l)
    ent = -(p * torch.where(p > 0, l, torch.zeros_like(l))).sum(-1)
    at = targets.clamp(min=0)
    return torch.where(targets >= 0, l.gather(-1, at[..., None])[..., 0], torch.zeros_like(lse)), ent, lse


def top(z, k):
    """ids of the k largest of each row, ties by ascending index; NaN ranks as -infinity"""
    return torch.sort(torch.nan_to_num(z, nan=float("-inf"), posinf=float("inf"), neginf=float("-inf")), dim=-1,
                      descending=True, stable=True).indices[..., :k]


def close(got, want, tol, what=""):
    """Every element within tol (a number or a tensor) of want, finite and non-finite alike."""
    g, w = f64(got), f64(want)
    assert g.shape == w.shape, (what, tuple(g.shape), tuple(w.shape))
    if not g.numel():
        return
    same = (g == w) | (torch.isnan(g) & torch.isnan(w))
    err = torch.where(same, torch.zeros_like(g), (g - w).abs())
    err = torch.where(torch.isnan(err), torch.full_like(err, float("inf")), err)
    over = err - tol
    k = int(over.argmax())
    assert float(over.reshape(-1)[k]) <= 0, "%s: off by %.3e at %d (got %r, want %r)" % (
        what, float(err.reshape(-1)[k]), k, float(g.reshape(-1)[k]), float(w.reshape(-1)[k]))


def rounded(want, tol, dtype):
    """Tolerance of an output stored in `dtype` whose float32 value is within tol: its own rounding added."""
    return tol if dtype == torch.float32 else tol + U16 * (want.detach().abs() + tol)
