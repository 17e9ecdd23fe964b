"""Layer normalisation and its gradients (include/pararnn_lm.h) against the plain 64-bit form.

Tolerances (u = 2^-24).  A sum over D values in threads of D/64 or fewer terms and a tree above them is off by at most
(D/64 + 16) u of the sum of magnitudes, so mean and variance, and with them y / max(1, max|s| rstd), by a few times that:
k = 4 (D/64 + 16) u.  The gradient is linear in dy with the same factors: k times max|dy w| rstd times 1 + max n^2
(from the two means).  A parameter sum over N rows: (N/16 + 64) u of the sum of its terms' magnitudes, and the terms'
own k."""
import pytest
import torch

import lm_plain as plain
from lm_plain import U32, close, f64, rounded
from nonlinear_rnn_solve_amd import lm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(N, D, dtype, seed, residual=True, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, res = (rnd(N, D) * 1.5 + shift).to(dtype).cuda(), rnd(N, D).to(dtype).cuda() if residual else None
    w, b = (1 + 0.2 * rnd(D)).cuda(), (0.2 * rnd(D)).cuda()
    return x, res, w, b, rnd(N, D).to(dtype).cuda(), rnd(N, D).to(dtype).cuda() if residual else None


def check(x, res, w, b, dy, dsum, eps=1e-5, **kw):
    dt = x.dtype
    y, s, stats = lm.layer_norm(x, w, b, residual=res, eps=eps, want_stats=True)
    xs = f64(x)
    want_s = xs if res is None else (f64(x) + f64(res)).to(dt).double()
    close(s, want_s, 0.0, "sum")
    leaf = f64(s).requires_grad_()
    lw, lb = f64(w).requires_grad_(), (None if b is None else f64(b).requires_grad_())
    wy, _ = plain.norm(leaf, lw, lb, eps=eps)
    N, D = x.reshape(-1, x.shape[-1]).shape
    rstd = 1 / torch.sqrt(leaf.detach().var(-1, unbiased=False, keepdim=True) + eps)
    size = (leaf.detach().abs().amax(-1, keepdim=True) * rstd).clamp(min=1.0)
    k = 4 * (D / 64 + 16) * U32
    close(y, wy, rounded(wy, k * size * f64(w).abs().max() + U32 * wy.detach().abs(), dt), "y")
    gs = torch.autograd.grad((wy * f64(dy)).sum(), [leaf, lw] + ([] if lb is None else [lb]))
    got = lm.layer_norm_vjp(dy, s, w, stats, d_sum=dsum)
    want = gs[0] if dsum is None else gs[0] + f64(dsum)
    n = (leaf.detach() - leaf.detach().mean(-1, keepdim=True)) * rstd
    scale = rstd * (f64(dy) * f64(w)).abs().amax(-1, keepdim=True) * (1 + (n * n).amax(-1, keepdim=True)) * size
    close(got["d_x"], want, rounded(want, k * scale + 2 * U32 * want.abs(), dt), "d_x")
    rows = (N / 16 + 64) * U32
    nt = (f64(dy) * n).abs().reshape(-1, D).sum(0) + (f64(dy).abs() * size).reshape(-1, D).sum(0)
    close(got["d_weight"], gs[1], (rows + k) * nt, "d_weight")
    close(got["d_bias"], f64(dy).reshape(-1, D).sum(0), rows * f64(dy).abs().reshape(-1, D).sum(0) + 1e-30, "d_bias")


WIDTHS = [1, 2, 7, 16, 33, 64, 100, 128, 129, 250, 256, 300, 511, 512, 1000, 1024, 1025, 2047, 2048, 3000, 4096, 5000, 8192, 8193, 16384]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, dtype):
    check(*make(5, D, dtype, seed=D))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,D", [(1, 512), (2, 64), (3, 1024), (63, 256), (64, 40), (257, 128), (1000, 96), (3001, 24), (700, 1500),
                                 (300, 6000), (20000, 8), (5000, 320)])
def test_rows(N, D, dtype):
    check(*make(N, D, dtype, seed=N + D, residual=N % 2 == 1))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_mean(dtype):
    # the variance is taken about the mean: a shift of 200 spreads costs only the shift's own rounding
    check(*make(9, 777, dtype, seed=1, shift=300.0, residual=False))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_bias_and_eps(dtype):
    x, res, w, _, dy, ds = make(6, 200, dtype, seed=2)
    check(x, res, w, None, dy, ds, eps=0.3)


def test_constant_rows():
    # a row without spread: n = 0, y = bias, and the gradient is that of 1 / sqrt(eps)
    x = torch.full((4, 96), 2.5, device="cuda")
    w, b = torch.ones(96, device="cuda"), torch.arange(96, device="cuda").float()
    y, s, stats = lm.layer_norm(x, w, b, want_stats=True)
    assert torch.equal(y, b.expand(4, -1))
    dy = torch.randn(4, 96, device="cuda")
    g = lm.layer_norm_vjp(dy, s, w, stats)
    want = (dy.double() - dy.double().mean(1, keepdim=True)) / 1e-5 ** 0.5
    close(g["d_x"], want, 64 * U32 * float(want.abs().max()), "d_x")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [96, 95, 1000, 4100])
def test_strides_and_leading_dimensions(D, dtype):
    g = torch.Generator().manual_seed(D)
    big = torch.randn(2, 30, 3 * D + 1, generator=g).to(dtype).cuda()
    x, res = big[..., 1:D + 1], big[..., D + 1:2 * D + 1]
    w, b = torch.randn(D, generator=g).cuda(), torch.randn(D, generator=g).cuda()
    dy = torch.randn(2, 30, D, generator=g).to(dtype).cuda()
    check(x, res, w, b, dy, None)
    # strided outputs, their surroundings untouched
    obuf = torch.full((2, 30, 2 * D + 3), 5.0, dtype=dtype, device="cuda")
    y, s, st = lm.layer_norm(x, w, b, residual=res, want_stats=True)
    lm.layer_norm(x, w, b, residual=res, out=obuf[..., 1:D + 1], sum_out=obuf[..., D + 2:2 * D + 2])
    assert torch.equal(obuf[..., 1:D + 1], y) and torch.equal(obuf[..., D + 2:2 * D + 2], s)
    assert (obuf[..., 0] == 5).all() and (obuf[..., D + 1] == 5).all() and (obuf[..., 2 * D + 2] == 5).all()


@pytest.mark.parametrize("D", [64, 1000, 9000])
def test_in_place(D):
    x, res, w, b, dy, ds = make(33, D, BF, seed=3)
    y, s, stats = lm.layer_norm(x, w, b, residual=res, want_stats=True)
    want = lm.layer_norm_vjp(dy, s, w, stats, d_sum=ds)
    res2 = res.clone()
    y2, s2, _ = lm.layer_norm(x, w, b, residual=res2, sum_out=res2)
    assert s2.data_ptr() == res2.data_ptr() and torch.equal(y, y2) and torch.equal(s, s2)
    for t in (dy, ds):
        src = {"dy": dy.clone(), "ds": ds.clone()}
        out = src["dy"] if t is dy else src["ds"]
        got = lm.layer_norm_vjp(src["dy"], s, w, stats, d_sum=src["ds"], out=out)
        for k in want:
            assert torch.equal(got[k], want[k]), k


def test_bad_values_stay_in_their_row():
    for D in (64, 3000):
        x, _, w, b, dy, _ = make(40, D, F32, seed=4, residual=False)
        y, s, st = lm.layer_norm(x, w, b, want_stats=True)
        g = lm.layer_norm_vjp(dy, s, w, st)["d_x"]
        x2 = x.clone()
        x2[7, 3], x2[11, 5], x2[23, 0] = float("nan"), float("inf"), torch.finfo(F32).min
        y2, s2, st2 = lm.layer_norm(x2, w, b, want_stats=True)
        g2 = lm.layer_norm_vjp(dy, s2, w, st2)["d_x"]
        keep = [n for n in range(40) if n not in (7, 11, 23)]
        assert torch.equal(y[keep], y2[keep]) and torch.equal(g[keep], g2[keep])
        assert torch.isnan(y2[7]).all() and torch.isnan(y2[11]).all()


@pytest.mark.parametrize("N,D", [(0, 16), (0, 5000), (4, 0)])
def test_empty(N, D):
    x = torch.zeros(N, D, device="cuda")
    w = torch.ones(D, device="cuda")
    y, s, stats = lm.layer_norm(x, w, want_stats=True)
    assert y.shape == (N, D)
    g = lm.layer_norm_vjp(x, s, w, stats)
    assert (g["d_weight"] == 0).all() and (g["d_bias"] == 0).all() and g["d_weight"].shape == (D,)


def test_gradients_against_differences():
    x, res, w, b, dy, ds = make(3, 50, F32, seed=5, residual=False)
    y, s, stats = lm.layer_norm(x, w, b, want_stats=True)
    got = lm.layer_norm_vjp(dy, s, w, stats)
    base = [f64(x), f64(w), f64(b)]
    gen = torch.Generator().manual_seed(2)
    loss = lambda t: float((plain.norm(*t)[0] * f64(dy)).sum())  # noqa: E731
    for k, name in enumerate(("d_x", "d_weight", "d_bias")):
        v = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        up, down = list(base), list(base)
        up[k], down[k] = base[k] + 1e-5 * v, base[k] - 1e-5 * v
        want = (loss(up) - loss(down)) / 2e-5
        g = f64(got[name])
        assert abs(float((g * v).sum()) - want) <= 1e-5 * float((g * v).abs().sum()) + 1e-6, name


def test_rows_beyond_32_bit_offsets():
    D = 256
    x, _, w, b, _, _ = make(5, D, BF, seed=6, residual=False)
    want = lm.layer_norm(x, w, b)[0]
    buf = torch.empty(4 * (1 << 30) + D, dtype=BF, device="cuda")
    far = buf.as_strided((5, D), (1 << 30, 1))
    far.copy_(x)
    assert torch.equal(lm.layer_norm(far, w, b)[0], want)
    lm.layer_norm(x, w, b, out=far)
    assert torch.equal(far, want)


@pytest.mark.parametrize("N,D", [(2000, 130), (300, 2500)])
def test_same_bits_stream_and_graph(N, D):
    x, res, w, b, dy, ds = make(N, D, BF, seed=7)

    def run():
        y, s, st = lm.layer_norm(x, w, b, residual=res, want_stats=True)
        return [y, s, *lm.layer_norm_vjp(dy, s, w, st, d_sum=ds).values()]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = run()
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert torch.equal(a, c)
    for _ in range(3):
        dy.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, c in zip(got, run()):
            assert torch.equal(a, c)
        torch.cuda.synchronize()


def test_refusals():
    x, res, w, b, dy, ds = make(4, 32, F32, seed=8)
    for bad in (lambda: lm.layer_norm(x.cpu(), w), lambda: lm.layer_norm(x.half(), w), lambda: lm.layer_norm(x, w[:5]),
                lambda: lm.layer_norm(x, w.bfloat16()), lambda: lm.layer_norm(x, w, residual=res.bfloat16()),
                lambda: lm.layer_norm(x, w, residual=res[:2]), lambda: lm.layer_norm(x.t(), w[:4].contiguous()),
                lambda: lm.layer_norm(x, w, sum_out=res), lambda: lm.layer_norm(x, w, out=x[:2]),
                lambda: lm.layer_norm_vjp(dy, x, w, None), lambda: lm.layer_norm_vjp(dy[:2], x, w, w),
                lambda: lm.layer_norm(x.view(2, 2, 32).transpose(0, 1), w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lm.PararnnError) as e:
        lm.layer_norm(torch.zeros(1, lm.NORM_MAX_D + 1, device="cuda"), torch.zeros(lm.NORM_MAX_D + 1, device="cuda"))
    assert e.value.status == -2
    with pytest.raises(lm.PararnnError) as e:
        lm.layer_norm(x, w, eps=-1.0)
    assert e.value.status == -1


def test_arguments_of_another_shape_are_refused():
    x, res, w, b, dy, ds = make(5, 32, F32, seed=9)
    y, s, stats = lm.layer_norm(x, w, b, residual=res, want_stats=True)
    with pytest.raises(ValueError, match="must be"):
        lm.layer_norm_vjp(dy, s, w, stats.t().contiguous())
    with pytest.raises(ValueError, match="must be"):
        lm.layer_norm(x, w.view(4, 8), b)
    assert torch.equal(lm.layer_norm(x, w[None], b[None], residual=res)[0], y)     # the same order of the same values
    want = lm.layer_norm_vjp(dy, s, w, stats)["d_x"]
    assert torch.equal(lm.layer_norm_vjp(dy, s, w, stats.flatten())["d_x"], want)
    got = lm.layer_norm_vjp(dy.view(5, 1, 32), s.view(5, 1, 32), w, stats.view(5, 1, 2))["d_x"]
    assert torch.equal(got.view(5, 32), want)


def test_written_tensors_tell_autograd():
    x, res, w, b, dy, ds = make(5, 32, F32, seed=10)
    y, stream = torch.empty_like(x), res.clone()
    before = y._version, stream._version, x._version
    _, s, stats = lm.layer_norm(x, w, b, residual=stream, out=y, sum_out=stream, want_stats=True)
    assert (y._version, stream._version, x._version) == (before[0] + 1, before[1] + 1, before[2])
    v = dy._version
    lm.layer_norm_vjp(dy, s, w, stats, out=dy)
    assert dy._version == v + 1


def test_as_many_rows_as_a_launch_holds():
    N, D, P = (1 << 28) - 16, 3, 16
    x, _, w, b, dy, _ = make(P, D, BF, seed=11, residual=False)
    want, _, stats = lm.layer_norm(x, w, b, want_stats=True)
    dwant = lm.layer_norm_vjp(dy, x, w, stats, want_params=False)["d_x"]
    many = lambda t: t.repeat(N // P, 1)  # noqa: E731
    y, s, st = lm.layer_norm(many(x), w, b, want_stats=True)
    assert (y.view(-1, P, D) == want).all() and (st.view(-1, P, 2) == stats).all()
    d = lm.layer_norm_vjp(many(dy), s, w, st, want_params=False)["d_x"]
    assert (d.view(-1, P, D) == dwant).all()
    with pytest.raises(lm.PararnnError) as e:
        lm.layer_norm(x[:1].expand(N + 1, D), w, b, out=y.new_empty(N + 1, D))
    assert e.value.status == -2
