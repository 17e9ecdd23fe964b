"""Cases of the language-model operators, for timing them and for comparing them with their plain forms.

Three operators, each of which a recurrent language model runs around the solves of this package:
  scan   the gated linear recurrence h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(i_t) x_t,
         a_t = exp(-c softplus(lam) sig(r_t)), and its gradients
  norm   layer normalisation with an optional residual sum, and its gradients
  logp   log probabilities of given tokens with the entropy and the top alternatives, and the gradient

A case's "pass" is "forward" (scoring, prompts, single tokens) or "train" (forward and gradients).
"""
import math

import torch

own = False   # False: the plain forms below; True: the package's operators

C = 8.0       # the recurrence's decay scale
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def _scan(name, mode, dtype, B, T, D, seqs=0):
    return {"name": name, "op": "scan", "pass": mode, "dtype": dtype, "B": B, "T": T, "D": D, "seqs": seqs}


def _norm(name, mode, dtype, N, D, residual):
    return {"name": name, "op": "norm", "pass": mode, "dtype": dtype, "N": N, "D": D, "residual": residual}


def _logp(name, mode, dtype, N, V, top, banned=0.0):
    return {"name": name, "op": "logp", "pass": mode, "dtype": dtype, "N": N, "V": V, "top": top, "banned": banned}


def listed():
    return [
        # one generated token for a batch of 32 streams: latency
        _scan("scan-token", "forward", "bf16", 32, 1, 1024),
        # prompts of seven users packed into one row, an odd number of channels, states kept for decoding
        _scan("scan-prompts", "forward", "f32", 1, 5003, 1025, seqs=7),
        # a training step at the shape of the package's wide bf16 workload
        _scan("scan-train-wide", "train", "bf16", 2, 4096, 4096),
        # a training step at the shape of the package's long-context workload
        _scan("scan-train-long", "train", "bf16", 1, 131072, 1024),
        # a training step in float32, packed documents in every row
        _scan("scan-train-f32", "train", "f32", 8, 2048, 1000, seqs=5),
        # one generated token for a batch of 32 streams, with the block's residual sum
        _norm("norm-token", "forward", "bf16", 32, 1024, True),
        # a training step of a wide block with its residual sum
        _norm("norm-train-wide", "train", "bf16", 8192, 4096, True),
        # a training step in float32 at an odd width, no residual
        _norm("norm-train-odd", "train", "f32", 5001, 2047, False),
        # sampling step of 32 streams with a tenth of the vocabulary banned, 20 alternatives each
        _logp("logp-token", "forward", "bf16", 32, 50001, 20, banned=0.1),
        # scoring a long document over a large vocabulary, 5 alternatives a token
        _logp("logp-score", "forward", "bf16", 4096, 131072, 5),
        # policy-gradient training: log probabilities and entropy with their gradient
        _logp("logp-train", "train", "f32", 4096, 32000, 0),
        # byte-level training: many short rows
        _logp("logp-train-bytes", "train", "bf16", 65536, 256, 0),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, mode = rng.choice(("scan", "norm", "logp")), rng.choice(("forward", "train"))
    dtype = rng.choice(("bf16", "f32"))
    if op == "scan":
        D = _spread(rng, 16, 4096)
        T = _spread(rng, 1, 131072) if rng.random() < 0.8 else 1
        B = _spread(rng, 1, max(1, min(64, (1 << 26) // (T * D))))
        T = min(T, max(1, (1 << 26) // (B * D)))
        seqs = rng.randrange(2, 10) if rng.random() < 0.3 else 0
        c = _scan("", mode, dtype, B, T, D, seqs)
    elif op == "norm":
        D = _spread(rng, 16, 8192)
        N = _spread(rng, 1, min(65536, (1 << 25) // D))
        c = _norm("", mode, dtype, N, D, rng.random() < 0.5)
    else:
        V = _spread(rng, 200, 131072)
        N = _spread(rng, 1, min(65536, (1 << 27) // V))
        c = _logp("", mode, dtype, N, V, 0 if mode == "train" else rng.choice((0, 1, 5, 20)), rng.choice((0.0, 0.1)))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "scan":
        B, T, D, n = case["B"], case["T"], case["D"], max(1, case["seqs"])
        # gates and values as one projection writes them: three slices of each step's row
        proj = normal(B, T, 3 * D, dtype=dt)
        s["x"], s["r"], s["i"] = proj[..., :D], proj[..., D:2 * D], proj[..., 2 * D:]
        # decays between 0.9 and 0.999 at an open gate
        a = torch.rand(D, generator=g, device="cuda", dtype=torch.float64) * 0.099 + 0.9
        s["lam"] = torch.log(torch.expm1(-torch.log(a) / C)).float()
        s["h0"] = normal(B, n, D, scale=0.5)
        s["cu"] = None
        if case["seqs"]:
            cuts = torch.randint(0, T + 1, (n - 1,), generator=g, device="cuda").sort().values
            s["cu"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
        if case["pass"] == "train":
            s["dh"], s["d_last"] = normal(B, T, D, dtype=dt), normal(B, n, D)
    elif case["op"] == "norm":
        N, D = case["N"], case["D"]
        s["x"] = normal(N, D, dtype=dt, scale=1.5)
        s["res"] = normal(N, D, dtype=dt) if case["residual"] else None
        s["weight"], s["bias"] = 1.0 + normal(D, scale=0.1), normal(D, scale=0.1)
        if case["pass"] == "train":
            s["dy"] = normal(N, D, dtype=dt)
            s["dsum"] = normal(N, D, dtype=dt) if case["residual"] else None
    else:
        N, V = case["N"], case["V"]
        s["logits"] = normal(N, V, dtype=dt, scale=2.5)
        if case["banned"]:
            s["logits"].masked_fill_(torch.rand(N, V, generator=g, device="cuda") < case["banned"], float("-inf"))
        s["targets"] = torch.randint(0, V, (N,), generator=g, device="cuda")
        s["targets"].masked_fill_(torch.rand(N, generator=g, device="cuda") < 0.05, -100)   # prompt tokens: no loss
        if case["pass"] == "train":
            s["g_logp"], s["g_entropy"] = normal(N), normal(N, scale=0.01)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return {"scan": _run_scan, "norm": _run_norm, "logp": _run_logp}[s["case"]["op"]](s)


def _run_scan(s):
    train = s["case"]["pass"] == "train"
    if own:
        from nonlinear_rnn_solve_amd import lm
        h, h_last, carry = lm.gated_scan(s["x"], s["r"], s["i"], s["lam"], h0=s["h0"], c=C, cu_seqlens=s["cu"],
                                         want_carry=train)
        out = {"h": h, "h_last": h_last}
        if train:
            out.update(lm.gated_scan_vjp(s["x"], s["r"], s["i"], s["lam"], carry, s["dh"], h0=s["h0"],
                                         d_last=s["d_last"], c=C, cu_seqlens=s["cu"]))
        return out
    x, r, i, h0 = s["x"].float(), s["r"].float(), s["i"].float(), s["h0"]
    dt, (B, T, D) = s["x"].dtype, x.shape
    start, end, seq, empty = _sequences(s["cu"], T, x.device)
    kappa = -C * (torch.log1p(torch.exp(-s["lam"].abs())) + s["lam"].clamp(min=0))
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    q = torch.expm1(kappa * sr)
    a, w = 1 + q, -q * (2 + q)
    m, u = torch.sqrt(w), si * x
    h_in = h0[:, seq[start]]                                  # the state entering each sequence that has steps
    ar, b = a.clone(), m * u
    b[:, start] += a[:, start] * h_in
    ar[:, start] = 0
    h = _linear_scan(ar, b)
    h_last = h0.clone()
    h_last[:, seq[end]] = h[:, end]
    out = {"h": h.to(dt), "h_last": h_last}
    if train:
        lam = s["dh"].to(torch.float32, copy=True)
        lam[:, end] += s["d_last"][:, seq[end]]
        a_next = torch.cat([ar[:, 1:], ar[:, :1] * 0], 1)
        lam = _linear_scan(a_next.flip(1), lam.flip(1)).flip(1)
        h_prev = torch.cat([h[:, :1], h[:, :-1]], 1)
        h_prev[:, start] = h_in
        dlog = lam * (a * h_prev - torch.where(w > 0, a * a * u / m, 0.0))
        dh0 = s["d_last"] * empty[:, None]
        dh0[:, seq[start]] = a[:, start] * lam[:, start]
        out.update({"d_x": (lam * m * si).to(dt), "d_r": (dlog * kappa * sr * (1 - sr)).to(dt),
                    "d_i": (lam * m * u * (1 - si)).to(dt),
                    "d_lam": -C * torch.sigmoid(s["lam"]) * (dlog * sr).sum((0, 1)), "d_h0": dh0})
    return out


def _sequences(cu, T, device):
    """Steps that begin and that end a sequence, each step's sequence, and which sequences have no step."""
    if cu is None:
        return (torch.zeros(1, dtype=torch.int64, device=device), torch.full((1,), T - 1, device=device),
                torch.zeros(T, dtype=torch.int64, device=device), torch.zeros(1, device=device))
    length = (cu[1:] - cu[:-1]).long()
    some = length > 0
    start, end = cu[:-1].long()[some], cu[1:].long()[some] - 1
    return start, end, torch.repeat_interleave(torch.arange(len(length), device=device), length), (~some).float()


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling."""
    n, T = 1, a.shape[1]
    while n < T:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _run_norm(s):
    train = s["case"]["pass"] == "train"
    if own:
        from nonlinear_rnn_solve_amd import lm
        y, total, stats = lm.layer_norm(s["x"], s["weight"], s["bias"], residual=s["res"], eps=EPS, want_stats=train)
        out = {"y": y}
        if s["res"] is not None:
            out["sum"] = total
        if train:
            out.update(lm.layer_norm_vjp(s["dy"], total, s["weight"], stats, d_sum=s["dsum"]))
        return out
    dt = s["x"].dtype
    total = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(dt)
    x = total.float()
    d = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    xh = d * rstd
    out = {"y": (xh * s["weight"] + s["bias"]).to(dt)}
    if s["res"] is not None:
        out["sum"] = total
    if train:
        dy = s["dy"].float()
        g = dy * s["weight"]
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        out.update({"d_x": dx.to(dt), "d_weight": (dy * xh).sum(0), "d_bias": dy.sum(0)})
    return out


def _run_logp(s):
    train, top = s["case"]["pass"] == "train", s["case"]["top"]
    if own:
        from nonlinear_rnn_solve_amd import lm
        t = lm.token_logprobs(s["logits"], s["targets"], top=top)
        out = {"logp": t.logp, "entropy": t.entropy}
        if top:
            out.update({"top_logp": t.top_logp, "top_ids": t.top_ids})
        if train:
            out["d_logits"] = lm.token_logprobs_vjp(s["logits"], s["targets"], t.lse, t.entropy, s["g_logp"],
                                                    s["g_entropy"])
        return out
    z, given = s["logits"].float(), s["targets"] >= 0
    at = s["targets"].clamp(min=0)[:, None]
    d = z - z.amax(1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    lp, p = d - torch.log(total), e / total
    plp = torch.where(p > 0, p * lp, 0.0)
    entropy = -plp.sum(1)
    out = {"logp": torch.where(given, lp.gather(1, at)[:, 0], 0.0), "entropy": entropy}
    if top:
        bits = (z + 0.0).view(torch.int32)
        bits = bits ^ ((bits >> 31) & 0x7FFFFFFF)             # whole numbers in the order of the values
        index = torch.arange(z.shape[1], device=z.device)
        key = torch.topk((bits.long() << 32) | (0xFFFFFFFF - index), top, dim=1).values   # ties: the lowest index
        out["top_ids"] = 0xFFFFFFFF - (key & 0xFFFFFFFF)
        out["top_logp"] = lp.gather(1, out["top_ids"])
    if train:
        g, ge = torch.where(given, s["g_logp"], 0.0)[:, None], s["g_entropy"][:, None]
        dz = -g * p - ge * (plp + p * entropy[:, None])
        out["d_logits"] = dz.scatter_add_(1, at, g).to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["pass"] == "train"
    if case["op"] == "scan":
        n, states = case["B"] * case["T"] * case["D"], case["B"] * max(1, case["seqs"]) * case["D"]
        # x, r, i in, h out; training: dh in, d_x, d_r, d_i out; states in and out in 32 bits
        return {"bytes": n * e * (8 if train else 4) + states * 4 * (4 if train else 2), "flops": n * (60 if train else 25)}
    if case["op"] == "norm":
        n, r = case["N"] * case["D"], case["residual"]
        # x (and the residual) in, y (and the sum) out; training: dy (and the sum's gradient) in, d_x out
        planes = (4 if r else 2) + ((3 if r else 2) if train else 0)
        return {"bytes": n * e * planes + case["D"] * 4 * (4 if train else 2), "flops": n * (20 if train else 8)}
    n = case["N"] * case["V"]
    return {"bytes": n * e * (2 if train else 1) + case["N"] * (20 + 12 * case["top"]), "flops": n * (12 if train else 6)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return {"scan": _exact_scan, "norm": _exact_norm, "logp": _exact_logp}[case["op"]](case, s, f)


def _exact_scan(case, s, f):
    """The recurrence and its adjoint one step after the other."""
    B, T, D = f["x"].shape
    rate = C * torch.nn.functional.softplus(f["lam"], threshold=700.0)
    open_r, open_i = 1 / (1 + torch.exp(-f["r"])), 1 / (1 + torch.exp(-f["i"]))
    log_a = -rate * open_r
    a, w = torch.exp(log_a), -torch.expm1(2 * log_a)
    v = torch.sqrt(w) * open_i * f["x"]
    cu = [0, T] if s["cu"] is None else s["cu"].tolist()
    h, before, last = torch.empty_like(v), torch.empty_like(v), f["h0"].clone()
    for j, (t0, t1) in enumerate(zip(cu[:-1], cu[1:])):
        state = f["h0"][:, j]
        for t in range(t0, t1):
            state = torch.addcmul(v[:, t], a[:, t], state, out=h[:, t])
        if t1 > t0:
            before[:, t0], before[:, t0 + 1:t1], last[:, j] = f["h0"][:, j], h[:, t0:t1 - 1], state
    out = {"h": h, "h_last": last}
    if case["pass"] == "train":
        lam, d_h0 = torch.empty_like(v), f["d_last"].clone()
        g = f["dh"].clone()
        for j, (t0, t1) in enumerate(zip(cu[:-1], cu[1:])):
            if t1 > t0:
                g[:, t1 - 1] += f["d_last"][:, j]
                lam[:, t1 - 1] = g[:, t1 - 1]
                for t in range(t1 - 2, t0 - 1, -1):
                    torch.addcmul(g[:, t], a[:, t + 1], lam[:, t + 1], out=lam[:, t])
                d_h0[:, j] = a[:, t0] * lam[:, t0]
        d_a = lam * (before - open_i * f["x"] * a / torch.sqrt(w))
        d_open = d_a * a * -rate
        d_rate = -(d_a * a * open_r).sum((0, 1))
        out.update({"d_x": lam * torch.sqrt(w) * open_i, "d_r": d_open * open_r * (1 - open_r),
                    "d_i": lam * v * (1 - open_i), "d_lam": d_rate * C / (1 + torch.exp(-f["lam"])), "d_h0": d_h0})
    return out


def _exact_norm(case, s, f):
    total = f["x"] if s["res"] is None else (f["x"] + f["res"]).to(s["x"].dtype).double()
    D = total.shape[1]
    mean = total.sum(1, keepdim=True) / D
    sd = torch.sqrt(((total - mean) ** 2).sum(1, keepdim=True) / D + EPS)
    n = (total - mean) / sd
    out = {"y": n * f["weight"] + f["bias"]}
    if s["res"] is not None:
        out["sum"] = total
    if case["pass"] == "train":
        k = f["dy"] * f["weight"] / sd
        d_x = k - k.sum(1, keepdim=True) / D - n * ((k * n).sum(1, keepdim=True) / D)
        out.update({"d_x": d_x if s["dsum"] is None else d_x + f["dsum"], "d_weight": (f["dy"] * n).sum(0),
                    "d_bias": f["dy"].sum(0)})
    return out


def _exact_logp(case, s, f):
    z, rows = f["logits"], torch.arange(case["N"], device=s["logits"].device)
    lp = z - torch.logsumexp(z, 1, keepdim=True)
    p = torch.exp(lp)
    finite = torch.nan_to_num(lp, neginf=0.0)
    ent = -(p * finite).sum(1)
    given = s["targets"] >= 0
    at = torch.where(given, s["targets"], 0)
    out = {"logp": torch.where(given, lp[rows, at], 0.0), "entropy": ent}
    if case["top"]:
        ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["top"]]
        out.update({"top_logp": lp.gather(1, ids), "top_ids": ids})
    if case["pass"] == "train":
        d = -(f["g_logp"] * given)[:, None] * p - f["g_entropy"][:, None] * p * (finite + ent[:, None])
        d[rows, at] += f["g_logp"] * given
        out["d_logits"] = d
    return out
