"""The gated feed-forward product and its gradients (include/pararnn_block.h) against the plain 64-bit form.

Tolerances, u = 2^-24.  A product of K terms is summed in float32 in some order: at most K u sum |a b| (bfloat16 products are exact);
taken as K u A B with the largest |row| sums estimated by K |a| |b| would be far too loose, so the magnitudes |a| |b|^T themselves are
summed.  The activation's slope is at most 1.13, its own error 8 u relative.  In bfloat16 dg and du are rounded once more (2^-8
relative each term), g and u too (2^-8, through slopes and products), before the sums: each term of d_x, d_w is off by at most
4 2^-8 of its magnitude, the magnitudes being those without cancellation."""
import pytest
import torch

import block_plain as plain
from lm_plain import U16, U32, close, f64, rounded
from nonlinear_rnn_solve_amd import block

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(R, D, F, dtype, seed, layout="dense"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w, dh = r(R, D).to(dtype).cuda(), (r(2, F, D) / max(1, D) ** 0.5).to(dtype).cuda(), r(R, F).to(dtype).cuda()
    if layout == "wide":                # rows with a stride of their own, at odd places
        big = torch.zeros(R, D + 5, device="cuda", dtype=dtype)
        big[:, 3:3 + D] = x
        x = big[:, 3:3 + D]
        both = torch.zeros(2 * F, D + 1, device="cuda", dtype=dtype)
        both[:, 1:] = w.reshape(2 * F, D)
        w = both[:, 1:].unflatten(0, (2, F)) if F else w
        hb = torch.zeros(R, F + 3, device="cuda", dtype=dtype)
        hb[:, 1:1 + F] = dh
        dh = hb[:, 1:1 + F]
    return x, w[0], w[1], dh


def check(args, activation="silu"):
    x, wg, wu, dh = args
    dt, (R, D), F = x.dtype, x.shape, wg.shape[0]
    leaves = [plain.leaf(t) for t in (x, wg, wu)]
    h = plain.gated(*leaves, activation)
    got_h, pre = block.gated_linear(x, wg, wu, activation, want_pre=True)
    with torch.no_grad():
        X, G, U, dH = f64(x), f64(wg), f64(wu), f64(dh)
        mg, mu = X.abs() @ G.abs().t(), X.abs() @ U.abs().t()          # magnitudes of the sums
        g, u = X @ G.t(), X @ U.t()
        eg, eu = (D + 2) * U32 * mg, (D + 2) * U32 * mu
        th = 1.13 * eg * u.abs() + g.abs() * eu + eg * eu + 16 * U32 * (g * u).abs()
        close(got_h, h, rounded(h, th, dt), "h")
        close(pre.reshape(R, 2, F)[:, 0], g, rounded(g, eg, dt), "gate")
        close(pre.reshape(R, 2, F)[:, 1], u, rounded(u, eu, dt), "up")
    if R * F * D == 0:
        want = [torch.zeros_like(t) for t in leaves]
    else:
        want = torch.autograd.grad((h * f64(dh)).sum(), leaves)
    got = block.gated_linear_vjp(x, wg, wu, pre, dh, activation)
    with torch.no_grad():
        sg, su = 1.13 * (dH * u).abs(), (dH * g).abs()                   # magnitudes of dg, du
        one = 4 * U16 if dt == BF else 32 * U32
        # what an error of g and u does to dg and du: slopes' slopes are below 1
        og = one * sg + dH.abs() * (eu * 1.13 + u.abs() * eg + ((u.abs() * g.abs() + u.abs()) * U16 if dt == BF else 0))
        ou = one * su + dH.abs() * (1.13 * eg + (1.13 * g.abs() * U16 if dt == BF else 0))
        tx = og @ G.abs() + ou @ U.abs() + 2 * F * U32 * (sg @ G.abs() + su @ U.abs())
        twg = og.t() @ X.abs() + R * U32 * (sg.t() @ X.abs())
        twu = ou.t() @ X.abs() + R * U32 * (su.t() @ X.abs())
    for name, w, t in zip(("d_x", "d_w_gate", "d_w_up"), want, (tx, twg, twu)):
        close(got[name], w, rounded(w, t, dt), name)
        if w.numel() > 8:
            far = float((f64(got[name]) - w).norm()) / max(float(w.norm()), 1e-30)
            assert far <= (1.5e-2 if dt == BF else 1e-5), (name, far)


SHAPES = [(1, 1, 1), (1, 64, 16), (2, 3, 5), (7, 33, 65), (32, 128, 256), (33, 129, 31), (31, 70, 300), (64, 64, 64), (65, 200, 130), (128, 256, 128),
          (130, 65, 257), (200, 1000, 100), (300, 257, 513), (513, 96, 70), (16, 4096, 40), (600, 512, 640)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_product_and_gradients(shape, dtype):
    check(make(*shape, dtype, seed=sum(shape)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(4353, 128, 1100), (4200, 256, 1040), (1100, 160, 4357)])
def test_large_tiles(shape, dtype):
    # 256 by 256 tiles (bfloat16, k of whole stages), their last rows and columns cut, and what is just not aligned for them
    check(make(*shape, dtype, seed=9))


def test_split_float32_keeps_what_float32_has():
    # values whose 24 bits all matter, sums that cancel to their last ones: three products of 8-bit parts would leave 2^-16
    g = torch.Generator().manual_seed(10)
    x = torch.randn(40, 512, generator=g)
    x[:, 256:] = -x[:, :256] * (1 + 2.0 ** -12)
    w = torch.randn(48, 512, generator=g)
    w[:, 256:] = w[:, :256]
    x, w = x.repeat(5, 1).cuda(), w.cuda()
    _, pre = block.gated_linear(x, w, w, want_pre=True)
    want = f64(x) @ f64(w).t()
    mag = f64(x).abs() @ f64(w).abs().t()
    close(pre[:, :48], want, 514 * U32 * mag, "gate")
    assert float((f64(pre[:, :48]) - want).norm()) <= 4 * U32 * float(mag.norm())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(5, 40, 24), (70, 130, 96), (260, 256, 272)])
def test_strides_and_gelu(shape, dtype):
    check(make(*shape, dtype, seed=2, layout="wide"), "gelu")


@pytest.mark.parametrize("shape", [(0, 8, 8), (3, 0, 8), (3, 8, 0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty(shape, dtype):
    x, wg, wu, dh = make(*shape, dtype, seed=3)
    h, pre = block.gated_linear(x, wg, wu, want_pre=True)
    assert h.shape == (shape[0], shape[2]) and not h.any()
    got = block.gated_linear_vjp(x, wg, wu, pre, dh)
    assert got["d_x"].shape == x.shape and got["d_w_gate"].shape == wg.shape
    assert not any(t.any() for t in got.values())


def test_leading_dimensions_and_outputs():
    x, wg, wu, dh = make(24, 40, 48, BF, seed=4)
    h, pre = block.gated_linear(x, wg, wu, want_pre=True)
    want = block.gated_linear_vjp(x, wg, wu, pre, dh)
    out = torch.full((2, 3, 4, 50), 7.0, device="cuda", dtype=BF)
    h4, none = block.gated_linear(x.reshape(2, 3, 4, 40), wg, wu, out=out[..., 1:49])
    assert none is None and torch.equal(h4.reshape(24, 48), h) and (out[..., [0, 49]] == 7).all()
    both = torch.full((2, 48, 42), 7.0, device="cuda", dtype=BF)
    got = block.gated_linear_vjp(x.reshape(2, 3, 4, 40), wg, wu, pre, dh.reshape(2, 3, 4, 48), w_out=[both[0, :, 1:41], both[1, :, 1:41]])
    assert got["d_x"].shape == (2, 3, 4, 40) and torch.equal(got["d_x"].reshape(24, 40), want["d_x"])
    assert torch.equal(both[0, :, 1:41], want["d_w_gate"]) and torch.equal(both[1, :, 1:41], want["d_w_up"])
    assert (both[..., [0, 41]] == 7).all()
    only = block.gated_linear_vjp(x, wg, wu, pre, dh, want_params=False)
    assert set(only) == {"d_x"} and torch.equal(only["d_x"], want["d_x"])
    only = block.gated_linear_vjp(x, wg, wu, pre, dh, want_x=False)
    assert set(only) == {"d_w_gate", "d_w_up"} and torch.equal(only["d_w_up"], want["d_w_up"])


@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_far_out_gates(activation):
    # act(g) at |g| up to 200: 0 or g, its slope 0 or 1
    x = torch.tensor([[200.0], [-200.0], [60.0], [-60.0], [0.0]], device="cuda")
    one = torch.ones(1, 1, device="cuda")
    h, pre = block.gated_linear(x, one, one, activation, want_pre=True)
    close(h, plain.gated(f64(x), f64(one), f64(one), activation), 1e-2, "h")
    got = block.gated_linear_vjp(x, one, one, pre, torch.ones(5, 1, device="cuda"), activation)
    assert torch.isfinite(got["d_x"]).all()
    assert abs(float(got["d_x"][0]) - 400) < 1e-3 and abs(float(got["d_x"][1])) < 1e-6


def test_nan_and_infinity_stay_in_their_rows():
    x, wg, wu, dh = make(150, 96, 140, BF, seed=5)
    clean, _ = block.gated_linear(x, wg, wu)
    x = x.clone()
    x[149, 5], x[7, 95] = float("nan"), float("inf")
    h, pre = block.gated_linear(x, wg, wu, want_pre=True)
    rows = [r for r in range(150) if r not in (7, 149)]
    assert torch.equal(h[rows], clean[rows]) and torch.isnan(h[149]).all() and not torch.isfinite(h[7]).any()
    got = block.gated_linear_vjp(x, wg, wu, pre, dh)
    assert torch.isfinite(got["d_x"][rows]).all()


def test_gradient_against_differences():
    x, wg, wu, dh = make(3, 4, 5, F32, seed=6)
    for activation in ("silu", "gelu"):
        _, pre = block.gated_linear(x, wg, wu, activation, want_pre=True)
        got = block.gated_linear_vjp(x, wg, wu, pre, dh, activation)
        at = [f64(t) for t in (x, wg, wu)]
        f = lambda *a: (plain.gated(*a, activation) * f64(dh)).sum()  # noqa: E731
        for i, name in enumerate(("d_x", "d_w_gate", "d_w_up")):
            flat = at[i].reshape(-1)
            for j in range(flat.numel()):
                old = float(flat[j])
                flat[j] = old + 1e-5
                up = f(*at)
                flat[j] = old - 1e-5
                down = f(*at)
                flat[j] = old
                assert abs(float(up - down) / 2e-5 - float(got[name].reshape(-1)[j])) < 1e-4, (name, j)


@pytest.mark.parametrize("shape", [(32, 512, 768), (700, 512, 640)])
def test_same_bits_on_every_run_another_stream_and_replayed(shape):
    x, wg, wu, dh = make(*shape, BF, seed=7)

    def both():
        h, pre = block.gated_linear(x, wg, wu, want_pre=True)
        return [h, pre] + list(block.gated_linear_vjp(x, wg, wu, pre, dh).values())

    first = both()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for n in range(3):
        x.copy_(torch.randn_like(x))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n


def test_refusals():
    x, wg, wu, dh = make(6, 8, 10, F32, seed=8)
    _, pre = block.gated_linear(x, wg, wu, want_pre=True)
    for bad in (lambda: block.gated_linear(x.double(), wg, wu), lambda: block.gated_linear(x, wg.bfloat16(), wu),
                lambda: block.gated_linear(x, wg[:, :7], wu[:, :7]), lambda: block.gated_linear(x, wg, wu[:9]),
                lambda: block.gated_linear(x.t(), wg, wu), lambda: block.gated_linear(x, wg.t().contiguous().t(), wu),
                lambda: block.gated_linear(x, wg, wu, "relu"), lambda: block.gated_linear(x, wg, wu.cpu()),
                lambda: block.gated_linear(x, wg, wu, out=x), lambda: block.gated_linear(x, wg, wu, out=dh[:1].expand(6, 10)),
                lambda: block.gated_linear(x, wg[0], wu[0]), lambda: block.gated_linear_vjp(x, wg, wu, None, dh),
                lambda: block.gated_linear_vjp(x, wg, wu, pre[:, :19], dh), lambda: block.gated_linear_vjp(x, wg, wu, pre, dh[:, :9]),
                lambda: block.gated_linear_vjp(x, wg, wu, pre, dh, w_out=[None]),
                lambda: block.gated_linear_vjp(x, wg, wu, pre, dh, want_x=False, out=x)):
        with pytest.raises(ValueError):
            bad()


def test_outputs_in_an_inputs_place_are_refused():
    x, wg, wu, dh = (torch.randn(16, 16, device="cuda") for _ in range(4))
    pre = block.gated_linear(x, wg, wu, want_pre=True)[1]
    with pytest.raises(ValueError, match="share memory"):
        block.gated_linear(x, wg, wu, out=x)
    one = torch.empty_like(x)
    for kw in (dict(out=x), dict(out=dh), dict(w_out=[wg, None]), dict(w_out=[one, one]), dict(out=one, w_out=[None, one])):
        with pytest.raises(ValueError, match="share memory"):
            block.gated_linear_vjp(x, wg, wu, pre, dh, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(70, 1000, 4100), (1500, 130, 1700), (4100, 2040, 40)])
def test_many_narrow_and_wide_tiles(shape, dtype):
    # as many tiles as make them 128 columns wide: of the weights' gradients, of the forward pass, of x's gradient; 256 and more else
    check(make(*shape, dtype, seed=12))


@pytest.mark.parametrize("shape", [(33, 129, 31), (300, 257, 513), (70, 1000, 4100), (4100, 2040, 40), (1300, 64, 70)])
def test_bfloat16_gradients_are_rounded_once(shape):
    # dg and du are off by 2^-16 and float32's roundings (as in check), the products' sums by float32's: of twice as many terms, dg's and du's
    # two bfloat16.  Only the result is rounded to bfloat16.  Few terms (the first and the last shape) show a rounding of each term best
    x, wg, wu, dh = make(*shape, BF, seed=21)
    (R, D), F = x.shape, wg.shape[0]
    got = block.gated_linear_vjp(x, wg, wu, block.gated_linear(x, wg, wu, want_pre=True)[1], dh)
    X, G, U, dH = f64(x), f64(wg), f64(wu), f64(dh)
    g, u = X @ G.t(), X @ U.t()
    eg, eu = (D + 2) * U32 * (X.abs() @ G.abs().t()), (D + 2) * U32 * (X.abs() @ U.abs().t())
    s = torch.sigmoid(g)
    dg, du = dH * u * (s * (1 + g * (1 - s))), dH * g * s
    sg, su = 1.13 * (dH * u).abs(), (dH * g).abs()                   # magnitudes
    one = U16 ** 2 + 32 * U32
    og, ou = one * sg + dH.abs() * (1.13 * eu + u.abs() * eg), one * su + dH.abs() * 1.13 * eg
    for name, w, t in (("d_x", dg @ G + du @ U, og @ G.abs() + ou @ U.abs() + 4 * F * U32 * (sg @ G.abs() + su @ U.abs())),
                       ("d_w_gate", dg.t() @ X, og.t() @ X.abs() + 2 * R * U32 * (sg.t() @ X.abs())),
                       ("d_w_up", du.t() @ X, ou.t() @ X.abs() + 2 * R * U32 * (su.t() @ X.abs()))):
        close(got[name], w, rounded(w, t, BF), name)


def test_bfloat16_gradients_of_huge_and_infinite_values():
    # dg = 3.4e38, which rounds to a bfloat16 infinity, stays finite; an infinite one stays infinite; u = 0 in the other rows
    x, half = torch.ones(70, 1, device="cuda", dtype=BF), torch.full((1, 1), 0.5, device="cuda", dtype=BF)
    pre = torch.zeros(70, 2, device="cuda")
    pre[:, 0] = 2.0
    slope = float(plain.silu(torch.tensor(2.0)) + torch.sigmoid(torch.tensor(2.0)) * (1 - plain.silu(torch.tensor(2.0))))
    pre[0, 1], pre[1, 1] = 3.4e38 / slope, float("inf")
    got = block.gated_linear_vjp(x, half, half * 0, pre, torch.ones(70, 1, device="cuda", dtype=BF))
    want = torch.tensor([1.7e38, float("inf")] + [0.0] * 68, dtype=torch.float64)[:, None]
    close(got["d_x"], want, 1.01 * U16 * 1.7e38, "d_x")


def test_large_tiles_repeat_their_bits():
    # 256 by 256 tiles forward and in both of the gradient's products
    x, wg, wu, dh = make(4100, 2048, 2048, BF, seed=7)

    def both():
        h, pre = block.gated_linear(x, wg, wu, want_pre=True)
        return [h, pre] + list(block.gated_linear_vjp(x, wg, wu, pre, dh).values())

    first = both()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, both()))


def test_pre_is_float32():
    # of bfloat16 inputs too: sums of exact products, off by float32's roundings only
    x, wg, wu, _ = make(300, 128, 96, BF, seed=7)
    _, pre = block.gated_linear(x, wg, wu, want_pre=True)
    for got, w in ((pre[:, :96], wg), (pre[:, 96:], wu)):
        close(got, f64(x) @ f64(w).t(), 130 * U32 * (f64(x).abs() @ f64(w).abs().t()), "pre")


@pytest.mark.parametrize("D", [1, 2, 3, 4])
def test_float32_of_few_terms(D):
    # of the split's nine products three are left out: at most 2 u of a term; sums of D terms are off by D u more.  These values' second and
    # third parts, were they cut off and not rounded, would be the largest there are
    v = 1 + 2.0 ** -7 - 2.0 ** -23
    x, w = torch.full((100, D), v, device="cuda"), torch.full((40, D), v, device="cuda")
    pre = block.gated_linear(x, w, -w, want_pre=True)[1]
    want = f64(x) @ f64(w).t()
    close(pre[:, :40], want, (D + 2) * U32 * want, "gate")
    close(pre[:, 40:], -want, (D + 2) * U32 * want, "up")


def test_float32_products_have_no_bias():
    # one term each, off by at most 3 u, upwards as often as downwards: as the mean of 4096 independent ones that is 6 3 / 64 u at most
    g = torch.Generator().manual_seed(31)
    x, w = torch.randn(4096, 1, generator=g).cuda(), torch.randn(4096, 1, generator=g).cuda()
    pre = block.gated_linear(x, w, w, want_pre=True)[1]
    want = f64(x) @ f64(w).t()
    off = (f64(pre[:, :4096]) - want) / want / U32
    assert float(off.abs().max()) <= 3 and abs(float(off.mean())) <= 18 / 64, (float(off.abs().max()), float(off.mean()))


def test_float32_at_its_lowest_value():
    # values that round to an infinite bfloat16, as masks have them
    low = torch.finfo(F32).min
    x = torch.tensor([[low, 1.0], [-low, -3.0]] * 40, device="cuda")
    w = torch.tensor([[2.0 ** -10, 1.0], [0.25, -(2.0 ** 100)]], device="cuda")
    pre = block.gated_linear(x, w, w, want_pre=True)[1]
    want = f64(x) @ f64(w).t()
    close(pre[:, :2], want, 4 * U32 * (f64(x).abs() @ f64(w).abs().t()), "gate")


@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("far", [17.0, 100.0, 1e15, 1e20, 3e38])
def test_gradients_of_gates_far_out(activation, far):
    # h = act(x) (x 2^-20): 0 for negative x, x^2 2^-20 for positive, whose derivative is x 2^-19 (silu at 17: 1 + 17 e^-17 within 1e-6)
    x = torch.tensor([[far], [-far]], device="cuda")
    one, small = torch.ones(1, 1, device="cuda"), torch.full((1, 1), 2.0 ** -20, device="cuda")
    pre = block.gated_linear(x, one, small, activation, want_pre=True)[1]
    got = block.gated_linear_vjp(x, one, small, pre, torch.ones(2, 1, device="cuda"), activation, want_params=False)["d_x"]
    want = torch.tensor([[f64(x)[0, 0] * 2.0 ** -19], [0.0]], dtype=torch.float64)
    close(got, want, 1e-5 * (want + 17 * 2.0 ** -19), "d_x")


@pytest.mark.parametrize("R", [32, 64, 65, 150])
def test_nan_and_infinity_stay_in_their_rows_in_float32(R):
    # infinite or NaN, by the kernel that the rows take; never finite, never beyond the row
    x, wg, wu, dh = make(R, 96, 140, F32, seed=22)
    clean, pre = block.gated_linear(x, wg, wu, want_pre=True)
    d_clean = block.gated_linear_vjp(x, wg, wu, pre, dh)["d_x"]
    x = x.clone()
    x[R - 1, 5], x[7, 95] = float("nan"), float("inf")
    h, pre = block.gated_linear(x, wg, wu, want_pre=True)
    rows = [r for r in range(R) if r not in (7, R - 1)]
    assert torch.equal(h[rows], clean[rows]) and torch.isnan(h[R - 1]).all()
    assert not torch.isfinite(pre[7]).any()
    got = block.gated_linear_vjp(x, wg, wu, pre, dh)
    assert torch.equal(got["d_x"][rows], d_clean[rows])
    assert not torch.isfinite(got["d_w_up"][:, 95]).any() and torch.isnan(got["d_w_up"][:, 5]).all()
