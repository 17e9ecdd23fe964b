"""The gated linear recurrence and its gradients (include/pararnn_lm.h) against the plain 64-bit recurrence.

Tolerances.  A step rounds a, m u and the fma: at most 3 units in the last place of values up to H = max |h|, of either
sign, and the recurrence remembers M = min(T, 1 / min(1 - a)) steps, so independent roundings add to about
3 sqrt(M) u H; 8 sqrt(M) + 16 units are allowed (u = 2^-24; 16 for the gates' own roundings).  The adjoint obeys the same
recurrence and multiplies two such values: twice that, relative to the largest entry of its output.  A sum of terms is
allowed its terms' relative error times the sum of their magnitudes."""
import math

import pytest
import torch

import lm_plain as plain
from lm_plain import U32, close, f64, rounded
from nonlinear_rnn_solve_amd import lm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(B, T, D, dtype, seed, n=0, layout="slices", state=True, grads=True):
    g = torch.Generator().manual_seed(seed)
    proj = torch.randn(B, T, 3 * D, generator=g).to(dtype)
    if layout == "slices":
        x, r, i = proj.cuda().split(D, -1) if D else [proj.cuda()[..., :0]] * 3
    elif layout == "time-major":
        x, r, i = (p.transpose(0, 1).contiguous().cuda().transpose(0, 1) for p in proj.split(D, -1))
    else:
        x, r, i = (p.contiguous().cuda() for p in proj.split(D, -1))
    a = torch.rand(D, generator=g, dtype=torch.float64) * 0.099 + 0.9
    lam = torch.log(torch.expm1(-torch.log(a) / 8)).float().cuda()
    shape = (B, n, D) if n else (B, D)
    h0 = torch.randn(shape, generator=g).cuda() if state else None
    dh = torch.randn(B, T, D, generator=g).to(dtype).cuda() if grads else None
    dl = torch.randn(shape, generator=g).cuda() if grads and state else None
    return x, r, i, lam, h0, dh, dl


def cuda_cu(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def reference(x, r, i, lam, h0, dh, dl, c=8.0, cu=None):
    leaves = [None if t is None else f64(t).requires_grad_() for t in (x, r, i, lam, h0)]
    h, last = plain.scan(*leaves, c=c, cu=cu)
    out = {"h": h.detach(), "h_last": last.detach()}
    if dh is not None:
        loss = (h * f64(dh)).sum() + (0.0 if dl is None else (last * f64(dl).reshape(last.shape)).sum())
        if not (loss.requires_grad):
            loss = loss + 0 * sum(t.sum() for t in leaves if t is not None)
        want = [t for t in leaves if t is not None]
        gs = torch.autograd.grad(loss, want, allow_unused=True)
        gs = [torch.zeros_like(t) if q is None else q for t, q in zip(want, gs)]
        out.update(zip(("d_x", "d_r", "d_i", "d_lam", "d_h0"), gs))
    M = min(max(1, x.shape[1]), 1 / max(plain.scan_decays(f64(r), f64(lam), c), 1e-7))
    return out, (16 + 8 * math.sqrt(M)) * U32


def check(args, c=8.0, cu=None, seqs=None):
    x, r, i, lam, h0, dh, dl = args
    ref, unit = reference(x, r, i, lam, h0, dh, dl, c, cu)
    dt, dcu = x.dtype, cuda_cu(cu)
    h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, c=c, cu_seqlens=dcu, want_carry=True)
    H = max(1.0, float(ref["h"].abs().max()) if ref["h"].numel() else 1.0,
            float(ref["h_last"].abs().max()) if ref["h_last"].numel() else 1.0)
    close(h, ref["h"], rounded(ref["h"], unit * H, dt), "h")
    close(last.reshape(ref["h_last"].shape), ref["h_last"], unit * H, "h_last")
    if dh is None:
        return
    got = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl, c=c, cu_seqlens=dcu)
    for k in ("d_x", "d_r", "d_i"):
        tol = 2 * unit * max(1.0, float(ref[k].abs().max()) if ref[k].numel() else 1.0)
        close(got[k], ref[k], rounded(ref[k], tol, dt), k)
    if h0 is not None:
        close(got["d_h0"], ref["d_h0"], 2 * unit * max(1.0, float(ref["d_h0"].abs().max()) if ref["d_h0"].numel() else 1.0), "d_h0")
    # d_lam = sum of terms: each as exact as d_r, whose terms carry the same factors
    rate = c * torch.nn.functional.softplus(f64(lam), threshold=700.0)
    s = torch.sigmoid(f64(r))
    terms = (ref["d_r"] / (rate * (1 - s)).clamp(min=1e-30)).abs().sum((0, 1)) * c * torch.sigmoid(f64(lam))
    close(got["d_lam"], ref["d_lam"], 4 * unit * (terms + 1e-6), "d_lam")


SHAPES = [(1, 1, 1), (2, 1, 64), (5, 1, 1030), (3, 5, 7), (1, 16, 130), (2, 17, 33), (2, 63, 65), (1, 64, 32), (2, 65, 70), (1, 127, 64), (1, 128, 65), (2, 129, 66),
          (1, 300, 1), (2, 256, 128), (2, 1000, 48), (1, 4099, 20), (3, 640, 200)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_scan_and_gradients(shape, dtype):
    check(make(*shape, dtype, seed=sum(shape)))


@pytest.mark.parametrize("layout", ["slices", "dense", "time-major"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(3, 150, 96), (3, 150, 95), (2, 3, 10)])
def test_layouts(shape, dtype, layout):
    check(make(*shape, dtype, seed=3, layout=layout))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_state(dtype):
    check(make(2, 200, 40, dtype, seed=4, state=False))


PACKED = [(300, [0, 1, 2, 150, 300]), (200, [0, 63, 64, 65, 128, 200]), (300, [0, 0, 128, 128, 129, 256, 300, 300]), (300, [0, 300]), (5, [0, 0, 2, 2, 5]),
          (1, [0, 0, 1, 1]), (512, [0, 127, 128, 255, 256, 257, 512]), (700, [0] + list(range(1, 700, 7)) + [700]),
          (16, [0, 16, 16]), (1500, [0, 1490, 1500]), (1500, [0, 3, 1500])]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,cu", PACKED)
def test_packed_sequences(T, cu, dtype):
    check(make(2, T, 70, dtype, seed=T + len(cu), n=len(cu) - 1), cu=cu)


def test_packed_ends_are_read_as_0_and_T():
    x, r, i, lam, h0, dh, dl = make(1, 200, 32, F32, seed=6, n=3)
    a = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cuda_cu([0, 50, 120, 200]))[0]
    b = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cuda_cu([7, 50, 120, 130]))[0]
    assert torch.equal(a, b)


@pytest.mark.parametrize("T", [10, 400])
def test_packed_without_states(T):
    args = make(2, T, 33, F32, seed=7, n=3)
    check(args[:4] + (None, args[5], None), cu=[0, 4, T // 2, T])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,cut", [(12, 5), (400, 130), (400, 256)])
def test_nothing_leaks_between_sequences(T, cut, bad):
    x, r, i, lam, h0, dh, dl = make(2, T, 40, F32, seed=8, n=3, layout="dense")
    cu = cuda_cu([0, cut, cut + 3, T])
    clean = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
    gclean = lm.gated_scan_vjp(x, r, i, lam, clean[2], dh, h0=h0, d_last=dl, cu_seqlens=cu)
    x2, dh2 = x.clone(), dh.clone()
    x2[:, cut:cut + 3] = bad          # the middle sequence is spoilt, in both directions
    dh2[:, cut:cut + 3] = bad
    h, last, carry = lm.gated_scan(x2, r, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
    g = lm.gated_scan_vjp(x2, r, i, lam, carry, dh2, h0=h0, d_last=dl, cu_seqlens=cu)
    keep = [t for t in range(T) if not cut <= t < cut + 3]
    assert torch.equal(h[:, keep], clean[0][:, keep]) and torch.equal(last[:, [0, 2]], clean[1][:, [0, 2]])
    for k in ("d_x", "d_r", "d_i"):
        assert torch.equal(g[k][:, keep], gclean[k][:, keep]), k
    assert torch.equal(g["d_h0"][:, [0, 2]], gclean["d_h0"][:, [0, 2]])
    assert not torch.isfinite(h[:, cut:cut + 3]).any()


@pytest.mark.parametrize("T,cut", [(12, 5), (400, 130), (400, 256), (3000, 1500)])
def test_a_spoilt_decay_gate_stays_in_its_sequence(T, cut):
    # NaN decays: the products of decays across a boundary are NaN, and must not count there
    x, r, i, lam, h0, dh, dl = make(2, T, 40, F32, seed=23, n=3, layout="dense")
    cu = cuda_cu([0, cut, cut + 3, T])
    clean = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
    gclean = lm.gated_scan_vjp(x, r, i, lam, clean[2], dh, h0=h0, d_last=dl, cu_seqlens=cu)
    r2 = r.clone()
    r2[:, cut:cut + 3] = float("nan")
    h, last, carry = lm.gated_scan(x, r2, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
    g = lm.gated_scan_vjp(x, r2, i, lam, carry, dh, h0=h0, d_last=dl, cu_seqlens=cu)
    keep = [t for t in range(T) if not cut <= t < cut + 3]
    assert torch.equal(h[:, keep], clean[0][:, keep]) and torch.equal(last[:, [0, 2]], clean[1][:, [0, 2]])
    for k in ("d_x", "d_r", "d_i"):
        assert torch.equal(g[k][:, keep], gclean[k][:, keep]), k
    assert torch.equal(g["d_h0"][:, [0, 2]], gclean["d_h0"][:, [0, 2]])
    assert torch.isnan(h[:, cut:cut + 3]).all() and torch.isnan(g["d_lam"]).all()


@pytest.mark.parametrize("lam_value", [3.0, 30.0])
@pytest.mark.parametrize("T,at", [(14, 2), (400, 3), (1500, 200)])
def test_a_spoilt_value_stays_to_the_end_of_its_sequence(T, at, lam_value):
    # strong decays: their products (lam = 3: of some 10 steps, lam = 30: each one) are zero in float32, which is no cut
    x, r, i, _, h0, dh, dl = make(2, T, 40, F32, seed=29, n=3, layout="dense")
    r = r.abs() + 3
    lam = torch.full((40,), lam_value, device="cuda")
    end, nan = T - 5, float("nan")
    cu = cuda_cu([0, 1, end, T])
    x2, dh2 = x.clone(), dh.clone()
    x2[:, at] = nan
    h, last, carry = lm.gated_scan(x2, r, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
    assert torch.isnan(h[:, at:end]).all() and torch.isnan(last[:, 1]).all()
    assert torch.isfinite(h[:, :at]).all() and torch.isfinite(h[:, end:]).all() and torch.isfinite(last[:, [0, 2]]).all()
    h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
    dh2[:, end - 1 - at] = nan
    g = lm.gated_scan_vjp(x, r, i, lam, carry, dh2, h0=h0, d_last=dl, cu_seqlens=cu)
    assert torch.isnan(g["d_x"][:, 1:end - at]).all() and torch.isnan(g["d_h0"][:, 1]).all()
    keep = [0] + list(range(end - at, T))
    assert torch.isfinite(g["d_x"][:, keep]).all() and torch.isfinite(g["d_h0"][:, [0, 2]]).all()


def test_gates_at_their_limits():
    # closed decay gate: a = 1, the state is held; wide open input; saturated values: finite everywhere
    B, T, D = 2, 300, 16
    x, r, i, lam, h0, dh, dl = make(B, T, D, F32, seed=9, layout="dense")
    r[:, ::3], r[:, 1::3], i[:, ::2], i[:, 1::5] = -float("inf"), 80.0, 90.0, -float("inf")
    h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
    want, wlast = plain.scan(*(f64(t) for t in (x, r, i, lam, h0)))
    close(h, want, 1e-4, "h")
    assert torch.equal(h[:, 0], h0)                   # a = 1, m = 0 exactly
    g = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl)
    for k, v in g.items():
        assert torch.isfinite(v).all(), k
    assert (g["d_r"][:, ::3] == 0).all() and (g["d_x"][:, ::3] == 0).all()


@pytest.mark.parametrize("value", [-90.0, -30.0, -9.0, 0.0, 20.0, 100.0])
def test_decay_parameter_range(value):
    x, r, i, _, h0, dh, dl = make(1, 200, 8, F32, seed=10)
    check((x, r, i, torch.full((8,), value, device="cuda"), h0, dh, dl) if value > -80 else
          (x, r, i, torch.full((8,), value, device="cuda"), h0, None, None))


@pytest.mark.parametrize("c", [0.5, 30.0])
def test_decay_scale(c):
    check(make(2, 140, 24, F32, seed=11), c=c)


@pytest.mark.parametrize("shape", [(0, 5, 4), (2, 0, 4), (2, 5, 0)])
def test_empty(shape):
    B, T, D = shape
    x = torch.zeros(shape, device="cuda")
    lam, h0 = torch.zeros(D, device="cuda"), torch.randn(B, D, device="cuda")
    h, last, carry = lm.gated_scan(x, x, x, lam, h0=h0, want_carry=True)
    assert h.shape == shape and (T > 0 or torch.equal(last, h0))
    dl = torch.randn(B, D, device="cuda")
    g = lm.gated_scan_vjp(x, x, x, lam, carry, x, h0=h0, d_last=dl)
    assert (g["d_lam"] == 0).all() and (T > 0 or torch.equal(g["d_h0"], dl))


def test_token_by_token_equals_the_whole():
    # a decoder that keeps its state in place gives the bits of one call over all steps of up to 16
    x, r, i, lam, h0, _, _ = make(4, 16, 100, BF, seed=12)
    want, last, _ = lm.gated_scan(x, r, i, lam, h0=h0)
    state = h0.clone()
    for t in range(16):
        h, s, _ = lm.gated_scan(x[:, t:t + 1], r[:, t:t + 1], i[:, t:t + 1], lam, h0=state, h_last=state)
        assert s.data_ptr() == state.data_ptr() and torch.equal(h, want[:, t:t + 1])
    assert torch.equal(state, last)


@pytest.mark.parametrize("T,cu", [(500, None), (500, [0, 200, 200, 500])])
def test_state_in_place_over_long_inputs(T, cu):
    x, r, i, lam, h0, _, _ = make(2, T, 64, BF, seed=13, n=3 if cu else 0)
    h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cuda_cu(cu), want_carry=True)
    state = h0.clone()
    h2, _, carry2 = lm.gated_scan(x, r, i, lam, h0=state, h_last=state, cu_seqlens=cuda_cu(cu), want_carry=True)
    assert torch.equal(h, h2) and torch.equal(state, last) and torch.equal(carry, carry2)


def test_split_row_equals_whole_row():
    # the state handed from one call to the next, and its gradient handed back
    x, r, i, lam, h0, dh, dl = make(2, 700, 40, F32, seed=14)
    whole, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
    gw = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl)
    a, b = slice(0, 333), slice(333, 700)
    h1, s1, c1 = lm.gated_scan(x[:, a], r[:, a], i[:, a], lam, h0=h0, want_carry=True)
    h2, s2, c2 = lm.gated_scan(x[:, b], r[:, b], i[:, b], lam, h0=s1, want_carry=True)
    g2 = lm.gated_scan_vjp(x[:, b], r[:, b], i[:, b], lam, c2, dh[:, b], h0=s1, d_last=dl)
    g1 = lm.gated_scan_vjp(x[:, a], r[:, a], i[:, a], lam, c1, dh[:, a], h0=h0, d_last=g2["d_h0"])
    unit = (16 + 8 * math.sqrt(700)) * U32
    close(torch.cat([h1, h2], 1), whole, unit * float(whole.abs().max()), "h")
    close(g1["d_h0"], gw["d_h0"], 2 * unit * float(gw["d_h0"].abs().max()), "d_h0")
    close(torch.cat([g1["d_r"], g2["d_r"]], 1), gw["d_r"], 2 * unit * float(gw["d_r"].abs().max()), "d_r")


def test_gradients_against_differences():
    args = make(2, 150, 6, F32, seed=15)
    x, r, i, lam, h0, dh, dl = args
    carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)[2]
    g = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl)
    gen = torch.Generator().manual_seed(1)
    base = [f64(t) for t in (x, r, i, lam, h0)]

    def loss(ts):
        h, last = plain.scan(*ts)
        return float((h * f64(dh)).sum() + (last * f64(dl)[:, None]).sum())

    for k, name in enumerate(("d_x", "d_r", "d_i", "d_lam", "d_h0")):
        v = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        up, down = list(base), list(base)
        up[k], down[k] = base[k] + step * v, base[k] - step * v
        want = (loss(up) - loss(down)) / (2 * step)
        got = float((f64(g[name]) * v).sum())
        # the difference is exact to ~step^2; float32 gradients to their own tolerance on the terms' magnitudes
        assert abs(got - want) <= 1e-5 * float((f64(g[name]) * v).abs().sum()) + 1e-6, (name, got, want)


def test_gradient_slices_of_one_array():
    x, r, i, lam, h0, dh, dl = make(2, 260, 48, BF, seed=16)
    carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)[2]
    want = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl)
    buf = torch.full((2, 260, 3 * 48 + 5), 7.0, dtype=BF, device="cuda")
    out = [buf[..., 48 * k:48 * (k + 1)] for k in range(3)]
    got = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl, out=out)
    for k in ("d_x", "d_r", "d_i", "d_lam", "d_h0"):
        assert torch.equal(got[k], want[k]), k
    assert (buf[..., 144:] == 7).all()


@pytest.mark.parametrize("T", [3, 300])
def test_broadcast_planes(T):
    # one gate for all rows (stride 0 over b): the gradient is that of each row's use of it
    x, r, i, lam, h0, dh, dl = make(3, T, 20, F32, seed=17)
    r = r[:1].expand(3, -1, -1)
    check((x, r, i, lam, h0, dh, dl))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [0, 4])
def test_a_channel_is_the_same_in_any_width(n, dtype):
    # the channels are independent: a problem's first D are those of a wider one, whatever tiles and lanes they fall to
    T, most = 203, 256
    cu = cuda_cu([0, 60, 60, 133, T]) if n else None

    def run(D, layout):
        x, r, i, lam, h0, dh, dl = make(2, T, most, dtype, seed=35, n=n, layout="dense")
        proj = torch.cat([p[..., :D] for p in (x, r, i)], -1)
        x, r, i = proj.chunk(3, -1) if layout == "slices" else (p.contiguous() for p in proj.chunk(3, -1))
        cut = lambda t: t[..., :D].contiguous()  # noqa: E731
        h0, dl, lam, dh = cut(h0), cut(dl), cut(lam), cut(dh)
        h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
        g = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl, cu_seqlens=cu)
        state = h0.clone()
        lm.gated_scan(x, r, i, lam, h0=state, cu_seqlens=cu, h_last=state)
        assert torch.equal(state, last)
        return [h, last, carry, *g.values()]

    want = run(most, "dense")
    for D in (1, 2, 3, 4, 5, 6, 7, 31, 62, 63, 64, 65, 66, 67, 68, 69, 127, 129, 130, 131, 193, 255):
        for layout in ("dense", "slices"):
            for a, b in zip(run(D, layout), want):
                assert torch.equal(a, b[..., :D]), (D, layout)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,cu", [(7, None), (40, None), (108, None), (333, None), (333, [0, 20, 300, 333])])
def test_planes_broadcast_over_time_or_overlapping(T, cu, dtype):
    # stride 0 over t (the gradient of a mean over time, for instance), steps closer than a row
    n = len(cu) - 1 if cu else 0
    x, r, i, lam, h0, dh, dl = make(2, T, 36, dtype, seed=32, n=n, layout="dense")
    same = lambda p: p[:, T // 2:T // 2 + 1].expand(-1, T, -1)  # noqa: E731
    over = lambda p: p.reshape(-1).as_strided((2, T, 36), (16 * T, 8, 1))  # noqa: E731
    check((x, r, i, lam, h0, same(dh), dl), cu=cu)
    check((same(x), same(r), same(i), lam, h0, dh, dl), cu=cu)
    check((over(x), over(r), over(i), lam, h0, over(dh), dl), cu=cu)
    check((x[..., :33], r[..., :33], i[..., :33], lam[:33], h0[..., :33].contiguous(), same(dh)[..., :33],
           dl[..., :33].contiguous()), cu=cu)


def test_offsets_beyond_32_bits():
    # rows over 2^32 elements apart, steps 2^25 apart: most offsets need 64 bits
    T, D = 130, 64
    x, r, i, lam, h0, _, _ = make(2, T, D, BF, seed=18, grads=False)
    want, last, _ = lm.gated_scan(x, r, i, lam, h0=h0)
    row = 200 << 25
    buf = torch.empty(row + T * (1 << 25) + D, dtype=BF, device="cuda")
    far = buf.as_strided((2, T, D), (row, 1 << 25, 1))
    far.copy_(x)
    got, glast, _ = lm.gated_scan(far, r, i, lam, h0=h0)
    assert torch.equal(got, want) and torch.equal(glast, last)
    outbuf = buf.as_strided((2, T, D), (row, 1 << 25, 1), 64)
    lm.gated_scan(x, r, i, lam, h0=h0, out=outbuf)
    assert torch.equal(outbuf, want)


@pytest.mark.parametrize("D", [64, 50])
def test_steps_too_far_apart_for_32_bits_in_a_tile(D):
    # steps over 2^27 bytes apart, every plane and output of both passes in one array
    T, step = 40, (1 << 26) + 8
    x, r, i, lam, h0, dh, dl = make(2, T, D, BF, seed=33, layout="dense")
    buf = torch.empty(2 * T * step, dtype=BF, device="cuda")
    planes = [buf.as_strided((2, T, D), (T * step, step, 1), 64 * k) for k in range(9)]
    guards = buf.as_strided((2, T, 64), (T * step, step, 1), 64 * 9)
    for p, src in zip(planes, (x, r, i, dh)):
        p.copy_(src)
    guards.fill_(7)
    h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
    g = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl)
    far = planes[:3]
    fh, flast, fcarry = lm.gated_scan(*far, lam, h0=h0, want_carry=True, out=planes[4])
    fg = lm.gated_scan_vjp(*far, lam, fcarry, planes[3], h0=h0, d_last=dl, out=planes[5:8])
    assert torch.equal(fh, h) and torch.equal(flast, last) and torch.equal(fcarry, carry)
    assert set(g) == set(fg) and all(torch.equal(fg[k], g[k]) for k in g)
    assert (guards == 7).all()
    lm.gated_scan(*(p[:, :5] for p in far), lam, h0=h0, out=planes[8][:, :5])
    assert torch.equal(planes[8][:, :5], h[:, :5])


def test_a_single_step_of_any_stride():
    # the stride of a dimension of one entry means nothing
    x, r, i, lam, h0, dh, dl = make(2, 1, 33, BF, seed=34, layout="dense")
    want = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
    g = lm.gated_scan_vjp(x, r, i, lam, want[2], dh, h0=h0, d_last=dl)
    for stride in (0, 1, 3, 64, 1 << 40, (1 << 62) + 1):
        view = lambda t: t.as_strided((2, 1, 33), (33, stride, 1))  # noqa: E731
        out = [torch.empty(66, dtype=BF, device="cuda") for _ in range(4)]
        got = lm.gated_scan(view(x), view(r), view(i), lam, h0=h0, want_carry=True, out=view(out[0]))
        gg = lm.gated_scan_vjp(view(x), view(r), view(i), lam, got[2], view(dh), h0=h0, d_last=dl, out=[view(o) for o in out[1:]])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(gg[k], g[k]) for k in g)


def test_same_bits_in_every_run_and_on_another_stream():
    args = make(2, 2000, 130, BF, seed=19)
    x, r, i, lam, h0, dh, dl = args

    def run():
        h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
        return [h, last, *lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl).values()]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    for a, b, c in zip(want, got, run()):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replays():
    x, r, i, lam, h0, dh, dl = make(2, 700, 64, BF, seed=20, layout="dense")
    new = make(2, 700, 64, BF, seed=21, layout="dense")

    def run():
        h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
        return [h, last, *lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl).values()]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = run()
    torch.cuda.synchronize()
    old = x.clone()
    for src in (old, new[0], old, new[0]):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, run()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_a_graph_keeps_its_workspace():
    # a later, larger call on the stream that the graph was captured on, then other tensors where a workspace could have been
    args = make(2, 700, 64, BF, seed=30, layout="dense")
    big = make(2, 40000, 64, BF, seed=31, layout="dense")

    def run(x, r, i, lam, h0, dh, dl):
        h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
        return [h, last, *lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl).values()]

    want, want_big = run(*args), run(*big)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(*args)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = run(*args)
        got_big = run(*big)
        side.synchronize()
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 22) * 3]
    torch.cuda.synchronize()
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all((o == 7).all() for o in others)
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(got_big, want_big))


def test_refusals():
    x, r, i, lam, h0, dh, dl = make(2, 20, 16, F32, seed=22, layout="dense")
    ok = lambda **k: lm.gated_scan(*(k.get(n, v) for n, v in zip("xril", (x, r, i, lam))), h0=k.get("h0"),  # noqa: E731
                                   c=k.get("c", 8.0), cu_seqlens=k.get("cu"), out=k.get("out"), h_last=k.get("h_last"))
    ok()
    for bad in (dict(x=x.cpu()), dict(r=r.bfloat16()), dict(x=x.half(), r=r.half(), i=i.half()), dict(i=i[:, :5]), dict(x=x[0]),
                dict(r=r.transpose(1, 2).contiguous().transpose(1, 2)), dict(l=lam.double()), dict(l=lam[:3]), dict(h0=h0[:1]),
                dict(h0=h0.bfloat16()), dict(cu=torch.tensor([0, 20], device="cuda")), dict(cu=cuda_cu([0])),
                dict(cu=cuda_cu([0, 5, 20]), h0=h0), dict(out=torch.empty_like(x, dtype=BF)), dict(out=x[:1].clone().expand(2, -1, -1)), dict(h_last=h0[:1])):
        with pytest.raises(ValueError):
            ok(**bad)
    for c in (0.0, -1.0, float("nan")):
        with pytest.raises(lm.PararnnError) as e:
            ok(c=c)
        assert e.value.status == -1
    with pytest.raises(ValueError, match="carry"):
        lm.gated_scan_vjp(x, r, i, lam, None, dh)


def parts_of_the_adjoint(x, r, i, lam, h0, dh, dl, c=8.0, cu=None):
    """What the gradients are products of, in 64 bits, with 1 - sig(v) as sig(-v)."""
    x, r, i, lam, dh = (f64(t) for t in (x, r, i, lam, dh))
    B, T, D = x.shape
    rate = c * torch.nn.functional.softplus(lam, threshold=700.0)
    z = -rate * torch.sigmoid(r)
    a, m, u = torch.exp(z), torch.sqrt(-torch.expm1(2 * z)), torch.sigmoid(i) * x
    h0 = torch.zeros(B, len(cu) - 1 if cu else 1, D, dtype=torch.float64) if h0 is None else f64(h0).reshape(B, -1, D)
    dl = torch.zeros_like(h0) if dl is None else f64(dl).reshape(B, -1, D)
    before, l = torch.empty_like(x), torch.empty_like(x)
    for j, (t0, t1) in enumerate(plain.sequences(cu, T)):
        h, mu = h0[:, j], dl[:, j]
        for t in range(t0, t1):
            before[:, t] = h
            h = a[:, t] * h + m[:, t] * u[:, t]
        for t in range(t1 - 1, t0 - 1, -1):
            l[:, t] = dh[:, t] + mu
            mu = a[:, t] * l[:, t]
    return dict(rate=rate, z=z, a=a, m=m, u=u, l=l, before=before, sr=torch.sigmoid(r), cr=torch.sigmoid(-r), si=torch.sigmoid(i),
                ci=torch.sigmoid(-i))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,D", [(1, 64), (1, 3), (90, 70), (90, 2)])
def test_gradients_of_open_and_closed_gates(T, D, dtype):
    # sequences of one step without a state: every gradient is a product, and each element of it has its relative accuracy.
    # Roundings, in u: the sigmoids' exponentials |v| <= 30 and 4, rates and roots 40, products 16 (90 in all)
    g = torch.Generator().manual_seed(T + D)
    r, i = ((torch.rand(1, T, D, generator=g) * 60 - 30).to(dtype).cuda() for _ in range(2))
    r[0, 0, :3], i[0, 0, :3] = torch.tensor([10.0, 18.0, 30.0])[:D], torch.tensor([16.0, 12.0, 30.0])[:D]
    x, dh = (torch.randn(1, T, D, generator=g).to(dtype).cuda() for _ in range(2))
    lam = make(1, 1, D, F32, seed=1)[3]
    cu = list(range(T + 1)) if T > 1 else None
    carry = lm.gated_scan(x, r, i, lam, cu_seqlens=cuda_cu(cu), want_carry=True)[2]
    got = lm.gated_scan_vjp(x, r, i, lam, carry, dh, cu_seqlens=cuda_cu(cu))
    p = parts_of_the_adjoint(x, r, i, lam, None, dh, None, cu=cu)
    e = -p["l"] * p["u"] * p["a"] ** 2 / p["m"]
    for k, want in (("d_x", p["l"] * p["m"] * p["si"]), ("d_i", p["l"] * p["m"] * p["u"] * p["ci"]),
                    ("d_r", -e * p["rate"] * p["sr"] * p["cr"])):
        close(got[k], want, rounded(want, 96 * U32 * want.abs(), dtype), k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [-30.0, -9.0, 0.0, 20.0])
def test_small_gradients_have_their_own_scale(value, dtype):
    # the adjoint is as exact as in the tests above, 2 unit of its largest value (h and l), and each factor of a gradient as
    # exact as its roundings: 32 u and 4 u |log a|; an a below the smallest normal float32, 2^-126, may be 0
    x, r, i, _, h0, dh, dl = make(1, 200, 8, dtype, seed=10)
    lam = torch.full((8,), value, device="cuda")
    unit = reference(x, r, i, lam, h0, dh, dl)[1]
    carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)[2]
    got = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl)
    p = parts_of_the_adjoint(x, r, i, lam, h0, dh, dl)
    L, H = float(p["l"].abs().max()), max(1.0, float(p["before"].abs().max()))
    rel = 2 * unit + 32 * U32 + 4 * U32 * p["z"].abs()
    jump = p["u"] * p["a"] ** 2 / p["m"]
    gate = p["rate"] * p["sr"] * p["cr"]
    for k, want, size in (("d_x", p["l"] * p["m"] * p["si"], L * p["m"] * p["si"]),
                          ("d_i", p["l"] * p["m"] * p["u"] * p["ci"], L * p["m"] * (p["u"] * p["ci"]).abs()),
                          ("d_r", -p["l"] * (p["a"] * p["before"] - jump) * gate, L * (p["a"] * H + jump.abs()) * gate)):
        assert float(want.abs().max()) > 0
        close(got[k], want, rounded(want, rel * size + 2.0 ** -126 * (1 + (L * H * gate if k == "d_r" else 0)), dtype), k)


def test_arguments_of_another_shape_are_refused():
    # as many values in another order would be states of other rows
    x, r, i, lam, h0, dh, dl = make(3, 70, 5, F32, seed=40, layout="dense")
    h, last, carry = lm.gated_scan(x, r, i, lam, h0=h0, want_carry=True)
    want = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=dl)
    turn = lambda t: t.transpose(0, -1).contiguous()  # noqa: E731
    for bad in (lambda: lm.gated_scan(x, r, i, lam, h0=h0, h_last=turn(h0)), lambda: lm.gated_scan_vjp(x, r, i, lam, turn(carry), dh, h0=h0, d_last=dl),
                lambda: lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=turn(dl))):
        with pytest.raises(ValueError, match="must be"):
            bad()
    cu = cuda_cu([0, 30, 70])
    hp = torch.randn(3, 2, 5, device="cuda")
    hc = lm.gated_scan(x, r, i, lam, h0=hp, cu_seqlens=cu, want_carry=True)[2]
    with pytest.raises(ValueError, match="must be"):
        lm.gated_scan_vjp(x, r, i, lam, hc, dh, h0=hp, d_last=hp.transpose(0, 1).contiguous(), cu_seqlens=cu)
    for same in (lambda t: t[:, None], lambda t: t.flatten()):     # the same order of the same values
        got = lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=same(dl))
        assert all(torch.equal(got[k], want[k]) for k in want)
    state = h0[:, None].clone()
    assert torch.equal(lm.gated_scan(x, r, i, lam, h0=h0, h_last=state)[1][:, 0], last)


def test_written_tensors_tell_autograd():
    # what autograd has saved and a call overwrites must not be used by a backward pass
    x, r, i, lam, h0, dh, dl = make(2, 20, 16, F32, seed=41, layout="dense")
    out, state = torch.empty_like(x), h0.clone()
    before = out._version, state._version, x._version
    carry = lm.gated_scan(x, r, i, lam, h0=state, out=out, h_last=state, want_carry=True)[2]
    assert (out._version, state._version, x._version) == (before[0] + 1, before[1] + 1, before[2])
    grads = [torch.empty_like(x) for _ in range(3)]
    before = [t._version for t in grads]
    lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, out=grads)
    assert [t._version for t in grads] == [v + 1 for v in before]
    with pytest.raises(ValueError):        # a refused call writes nothing
        lm.gated_scan_vjp(x, r, i, lam, carry, dh, h0=h0, d_last=lam, out=grads)
    assert [t._version for t in grads] == [v + 1 for v in before]
    leaf = torch.ones_like(x, requires_grad=True)
    y = leaf * 2
    loss = (y * y).sum()
    lm.gated_scan(x, r, i, lam, out=y.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    with torch.inference_mode():       # tensors without a counter
        lm.gated_scan(x, r, i, lam, out=torch.empty_like(x))
    with torch.inference_mode():
        inference = torch.empty_like(x)
    lm.gated_scan(x, r, i, lam, out=inference)
