"""Log probabilities of given tokens, entropy, top alternatives and their gradient (include/pararnn_lm.h) against the
plain 64-bit form.

Tolerances (u = 2^-24).  z - m is rounded once, its exponential to a few u plus u |z - m|, whose weight e^(z-m) |z-m| is
below 0.4; the sums of positive terms in threads of V/64 or fewer terms and a tree are off by (V/64 + 16) u relatively: lse
by that plus u |lse|, logp by that plus u (|z_t - m| + |m|).  The entropy's second sum has terms of one sign and size at
most ln V of the first: (V/64 + 16) u (1 + ln V) doubled.  The gradient's p = e^(z - lse) carries lse's error plus u |z - lse|:
relative to |g| + |g_H| (ln V + max |ln p|), times p; below the smallest normal float32, 2^-126, p may be 0."""
import math

import pytest
import torch

import lm_plain as plain
from lm_plain import U32, close, f64, rounded
from nonlinear_rnn_solve_amd import lm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def make(N, V, dtype, seed, scale=2.5, banned=0.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(N, V, generator=g) * scale).to(dtype)
    if banned:
        z = z.masked_fill(torch.rand(N, V, generator=g) < banned, -INF)
        z[:, 0] = 0.0
    t = torch.randint(0, V, (N,), generator=g)
    t[torch.rand(N, generator=g) < 0.2] = -100
    return z.cuda(), t.cuda(), torch.randn(N, generator=g).cuda(), torch.randn(N, generator=g).cuda()


def check(z, t, g, ge, top=0):
    N, V = z.shape
    res = lm.token_logprobs(z, t, top=top)
    lp, ent, lse = plain.logp(f64(z), t.cpu().long())
    m = f64(z).amax(-1)
    base = (V / 64 + 16) * U32
    close(res.lse, lse, base + U32 * (lse.abs() + m.abs()), "lse")
    zt = f64(z).gather(1, t.cpu().long().clamp(min=0)[:, None])[:, 0]
    near = torch.where(torch.isinf(zt), torch.zeros_like(zt), (zt - m).abs())
    close(res.logp, lp, base + 2 * U32 * (near + torch.where(torch.isinf(lp), torch.zeros_like(lp), lp.abs())), "logp")
    close(res.entropy, ent, 2 * base * (1 + math.log(V)), "entropy")
    if top:
        ids = plain.top(f64(z), top)
        assert torch.equal(res.top_ids.cpu(), ids)
        want = (f64(z) - lse[:, None]).gather(1, ids)
        mag = torch.where(torch.isinf(want), torch.zeros_like(want), want.abs())
        close(res.top_logp, want, base + 4 * U32 * (mag + 1), "top_logp")
    else:
        assert res.top_ids is None and res.top_logp is None
    d = lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge)
    l = f64(z) - lse[:, None]
    p = torch.exp(l)
    fl = torch.where(torch.isinf(l), torch.zeros_like(l), l)
    given = (t.cpu() >= 0).double()
    gg, hh = f64(g) * given, (torch.zeros(N, dtype=torch.float64) if ge is None else f64(ge))
    want = -gg[:, None] * p - hh[:, None] * p * (fl + ent[:, None])
    want[torch.arange(N), t.cpu().long().clamp(min=0)] += gg
    # |p'| / p: lse's error, u |l| from z - lse and the exponent's scaling, a few roundings
    rel = base + U32 * (lse.abs()[:, None] + m.abs()[:, None] + 2 * fl.abs() + 8)
    size = gg.abs()[:, None] + hh.abs()[:, None] * (fl.abs() + ent[:, None] + 1)
    tol = (rel * p + 2.0 ** -126) * size + 2 * base * (1 + math.log(V)) * p * hh.abs()[:, None] + U32 * want.abs()
    tol += U32 * 2 * (gg.abs()[:, None] * (want != 0))     # the target's 1 - p
    close(d, want, rounded(want, tol, z.dtype), "d_logits")


SIZES = [(1, 1), (3, 2), (5, 7), (4, 64), (2, 65), (9, 255), (70, 256), (3, 257), (130, 300), (2, 1000), (5, 1024), (3, 2047), (3, 2049),
         (2, 4096), (2, 5001), (3, 8191), (1, 16384), (2, 16385), (2, 32000), (3, 50001), (1, 131072), (2, 130003)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V", SIZES)
def test_sizes(N, V, dtype):
    check(*make(N, V, dtype, seed=N + V), top=min(V, 20))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V", [(6, 300), (4, 5001), (300, 3000), (3, 40000)])
def test_ruled_out_tokens(N, V, dtype):
    z, t, g, ge = make(N, V, dtype, seed=V, banned=0.5)
    z[1, 1:] = -INF            # one token left
    z[2, 7:] = -INF            # fewer left than alternatives asked for
    check(z, t, g, ge, top=20)


@pytest.mark.parametrize("V", [300, 5001])
def test_large_entropy_gradient_with_ruled_out_tokens(V):
    # a power of two scales every product exactly; ln p of a ruled out token is -infinity
    z, t, g, ge = make(5, V, F32, seed=V, banned=0.3)
    res = lm.token_logprobs(z)
    one = lm.token_logprobs_vjp(z, None, res.lse, res.entropy, None, ge)
    large = lm.token_logprobs_vjp(z, None, res.lse, res.entropy, None, ge * 2.0 ** 108)
    assert torch.equal(large, one * 2.0 ** 108) and torch.isfinite(large).all()


@pytest.mark.parametrize("top", [0, 1, 2, 5, 31, 32])
def test_alternative_counts(top):
    for V in (40, 3000, 20011):
        check(*make(4, V, BF, seed=top), top=top)


@pytest.mark.parametrize("V", [33, 300, 2050, 17000, 66000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties_and_orders(V, dtype):
    j = torch.arange(V).float()
    rows = torch.stack([torch.zeros(V), torch.full((V,), -INF).index_fill(0, torch.tensor([0, 3, V - 1]), 1.0),
                        j / V, -j / V, (j % 2), (j % 7 == 0).float(), torch.where(j % 64 < 8, 1 + j / V, 0 * j),
                        torch.where(j < V // 2, -0.0 * j, 0 * j), (j // 500) % 3, torch.where(j % 512 < 16, j, -j)]).to(dtype).cuda()
    res = lm.token_logprobs(rows, None, top=32)
    assert res.logp is None
    assert torch.equal(res.top_ids.cpu(), plain.top(f64(rows), 32))


@pytest.mark.parametrize("V", [3000, 30000, 66000])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top", [1, 31, 32])
def test_large_logits_in_few_columns(V, dtype, top):
    # the large logits fill only some of the positions modulo the stride in which a row is read
    j = torch.arange(V)
    rows = []
    for per in (4, 8, 16):
        for cols in (1, 31, 40):
            rows.append(torch.where((j // per) % 64 < cols, 10 + j / V, -j / V))
    z = torch.stack(rows).to(dtype).cuda()
    assert torch.equal(lm.token_logprobs(z, None, top=top).top_ids.cpu(), plain.top(f64(z), top))


def test_rows_with_nothing_left():
    for V in (5, 700, 9000, 70000):
        z, t, g, ge = make(6, V, F32, seed=V)
        z[2], z[4] = -INF, torch.finfo(F32).min       # nothing left; everything at the type's lowest value
        t[:] = torch.tensor([0, 1, 2, -1, 3, 4])
        res = lm.token_logprobs(z, t, top=3)
        assert res.lse[2] == -INF and res.logp[2] == -INF and res.entropy[2] == 0
        assert (res.top_logp[2] == -INF).all() and res.top_ids[2].tolist() == [0, 1, 2]
        assert res.logp[3] == 0
        # a mask of lowest values all over is a uniform distribution
        close(res.logp[4:5], torch.full((1,), -math.log(V)), 1e-5, "uniform")
        close(res.entropy[4:5], torch.full((1,), math.log(V)), (V / 64 + 16) * U32 * (1 + math.log(V)), "uniform")
        d = lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge)
        assert (d[2] == 0).all() and torch.isfinite(d).all()


def test_lowest_values_as_a_mask():
    for dtype in (BF, F32):
        z, t, g, ge = make(5, 3000, dtype, seed=1)
        z[:, 500:] = torch.finfo(dtype).min
        t[:] = torch.tensor([1, 2, 3, -1, 499])
        ref = lm.token_logprobs(z[:, :500], t)
        res = lm.token_logprobs(z, t)
        close(res.logp, ref.logp, 64 * U32 * 16, "logp")
        close(res.entropy, ref.entropy, 64 * U32 * 16, "entropy")
        d = lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge)
        assert torch.isfinite(d).all() and (d[:, 500:] == 0).all()


def test_bad_values_stay_in_their_row():
    for V in (100, 6000, 50000):
        z, t, g, ge = make(8, V, F32, seed=2)
        ref = lm.token_logprobs(z, t, top=4)
        d = lm.token_logprobs_vjp(z, t, ref.lse, ref.entropy, g, ge)
        z2 = z.clone()
        z2[1, 5], z2[3, 7], z2[6] = float("nan"), INF, float("nan")
        res = lm.token_logprobs(z2, t, top=4)
        d2 = lm.token_logprobs_vjp(z2, t, res.lse, res.entropy, g, ge)
        keep = [0, 2, 4, 5, 7]
        for a, b in zip(ref, res):
            assert torch.equal(a[keep], b[keep])
        assert torch.equal(d[keep], d2[keep])
        for n in (1, 3, 6):
            assert torch.isnan(res.lse[n]) and torch.isnan(res.entropy[n]) and torch.isnan(d2[n]).any()
        assert torch.equal(res.top_ids.cpu(), plain.top(f64(z2), 4))


def test_targets():
    z, t, g, ge = make(6, 50, F32, seed=3)
    t[:] = torch.tensor([0, 49, 50, -1, 7, 2 ** 40])
    r64 = lm.token_logprobs(z, t)
    assert torch.isnan(r64.logp[2]) and torch.isnan(r64.logp[5]) and r64.logp[3] == 0
    t32 = t.clamp(max=1000).to(torch.int32)
    r32 = lm.token_logprobs(z, t32)
    keep = [0, 1, 3, 4]
    assert torch.equal(r64.logp[keep], r32.logp[keep])
    d = lm.token_logprobs_vjp(z, t, r64.lse, r64.entropy, g, ge)
    assert torch.isnan(d[2]).all() and torch.equal(d[keep], lm.token_logprobs_vjp(z, t32, r32.lse, r32.entropy, g, ge)[keep])
    e = lm.token_logprobs_vjp(z, None, r64.lse, r64.entropy, None, ge)     # the entropy alone
    close(e[3], d[3], 0.0, "entropy's gradient")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [100, 2100, 33000])
def test_views_of_a_padded_vocabulary(V, dtype):
    # rows longer than the vocabulary, every alignment of their start
    for pad in (1, 2, 3, 8):
        big, t, g, ge = make(6, V + 2 * pad, dtype, seed=pad)
        z = big[:, pad:pad + V]
        t = t.clamp(max=V - 1)
        check(z, t, g, ge, top=5)
        out = torch.full((6, V + 2 * pad), 3.0, dtype=dtype, device="cuda")
        r = lm.token_logprobs(z, t)
        want = lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g, ge)
        lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g, ge, out=out[:, pad:pad + V])
        assert torch.equal(out[:, pad:pad + V], want) and (out[:, :pad] == 3).all() and (out[:, pad + V:] == 3).all()


def test_leading_dimensions_and_in_place():
    z, t, g, ge = make(6, 1000, BF, seed=4)
    a = lm.token_logprobs(z, t, top=3)
    b = lm.token_logprobs(z.view(2, 3, 1000), t.view(2, 3), top=3)
    assert b.logp.shape == (2, 3) and b.top_ids.shape == (2, 3, 3)
    for p, q in zip(a, b):
        assert torch.equal(p, q.reshape(p.shape))
    want = lm.token_logprobs_vjp(z, t, a.lse, a.entropy, g, ge)
    got = lm.token_logprobs_vjp(z, t, a.lse, a.entropy, g, ge, out=z)
    assert got.data_ptr() == z.data_ptr() and torch.equal(z, want)


def test_large_and_small_logits():
    for scale in (1e-3, 50.0, 1e4):
        check(*make(4, 3001, F32, seed=5, scale=scale), top=5)


def test_without_entropy_gradient():
    z, t, g, _ = make(5, 700, F32, seed=6)
    check(z, t, g, None)


def test_gradient_against_differences():
    z, t, g, ge = make(3, 40, F32, seed=7, scale=1.0)
    res = lm.token_logprobs(z, t)
    d = f64(lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge))
    v = torch.randn(3, 40, generator=torch.Generator().manual_seed(1), dtype=torch.float64)

    def loss(x):
        lp, ent, _ = plain.logp(x, t.cpu())
        return float((lp * f64(g)).sum() + (ent * f64(ge)).sum())

    want = (loss(f64(z) + 1e-5 * v) - loss(f64(z) - 1e-5 * v)) / 2e-5
    assert abs(float((d * v).sum()) - want) <= 1e-5 * float((d * v).abs().sum()) + 1e-7


def test_rows_beyond_32_bit_offsets():
    V = 5000
    z, t, g, ge = make(5, V, BF, seed=8)
    buf = torch.empty(4 * (1 << 30) + V, dtype=BF, device="cuda")
    far = buf.as_strided((5, V), (1 << 30, 1))
    far.copy_(z)
    for a, b in zip(lm.token_logprobs(z, t, top=4), lm.token_logprobs(far, t, top=4)):
        assert torch.equal(a, b)
    r = lm.token_logprobs(z, t)
    want = lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g, ge)
    lm.token_logprobs_vjp(far, t, r.lse, r.entropy, g, ge, out=far)
    assert torch.equal(far, want)


@pytest.mark.parametrize("N,V", [(700, 256), (3, 70000), (40, 4000)])
def test_same_bits_stream_and_graph(N, V):
    z, t, g, ge = make(N, V, BF, seed=9)

    def run():
        r = lm.token_logprobs(z, t, top=8)
        return [*r, lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g, ge)]

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
        z.mul_(-0.75)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, c in zip(got, run()):
            assert torch.equal(a, c)
        torch.cuda.synchronize()


def test_empty():
    z, t = torch.zeros(0, 50, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    r = lm.token_logprobs(z, t, top=3)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 3)
    assert lm.token_logprobs_vjp(z, t, r.lse, r.entropy, r.lse).shape == (0, 50)


def test_refusals():
    z, t, g, ge = make(4, 32, F32, seed=10)
    r = lm.token_logprobs(z, t)
    for bad in (lambda: lm.token_logprobs(z.cpu(), t), lambda: lm.token_logprobs(z.half(), t), lambda: lm.token_logprobs(z, t.float()),
                lambda: lm.token_logprobs(z, t[:2]), lambda: lm.token_logprobs(z, t, top=33), lambda: lm.token_logprobs(z, t, top=-1),
                lambda: lm.token_logprobs(z[:, :4], t, top=5), lambda: lm.token_logprobs(z.t(), t),
                lambda: lm.token_logprobs(z, t.cpu()), lambda: lm.token_logprobs_vjp(z, t, r.lse, r.entropy, None),
                lambda: lm.token_logprobs_vjp(z, t, r.lse, None, g, ge), lambda: lm.token_logprobs_vjp(z, t, r.lse[:2], r.entropy, g),
                lambda: lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g.double()),
                lambda: lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g, out=z.bfloat16())):
        with pytest.raises(ValueError):
            bad()


# The gradient's error must not grow with a common offset of a row's logits: the softmax has none.  z - lse and what the
# gradient adds to it are rounded to u |ln p| each, the exponential's argument as well: 3 u |ln p|, and 48 u for the normaliser's
# own roundings (half a unit of an lse of up to 32: 16 u; its logarithm of up to ln V: 12 u; a few for the exponential).
def gradient_close(d, z, t, g, ge):
    V = z.shape[1]
    base = (V / 64 + 16) * U32
    l = f64(z) - f64(z).amax(-1, keepdim=True)
    l = l - torch.logsumexp(l, -1, keepdim=True)
    p, fl = torch.exp(l), torch.where(torch.isinf(l), torch.zeros_like(l), l)
    ent = -(p * fl).sum(-1)
    gg, hh, at = f64(g) * (t.cpu() >= 0), f64(ge), t.cpu().long().clamp(min=0)
    want = -gg[:, None] * p - hh[:, None] * p * (fl + ent[:, None])
    want[torch.arange(len(gg)), at] += gg
    rel = base + U32 * (3 * fl.abs() + 48)
    size = gg.abs()[:, None] + hh.abs()[:, None] * (fl.abs() + ent[:, None] + 1)
    tol = (rel * p + 2.0 ** -126) * size + 2 * base * (1 + math.log(V)) * p * hh.abs()[:, None] + U32 * want.abs()
    tol += U32 * 2 * (gg.abs()[:, None] * (want != 0))
    close(d, want, rounded(want, tol, z.dtype), "d_logits")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [5, 64, 200, 900, 3000, 9000, 40000])
def test_gradient_of_rows_with_a_common_offset(V, dtype):
    # rows of one tensor with different offsets, all of them exact in the storage type
    gen = torch.Generator().manual_seed(V)
    offsets = [0.0, 64.0, -64.0, 128.0, 0.0, -256.0, 31.0, -40.0] if dtype == BF else \
        [0.0, 2.0 ** 10, -2.0 ** 10, 2.0 ** 15, 0.0, -2.0 ** 15, 31.0, -40.0]
    rows = []
    for o in offsets:
        step = 2.0 ** (math.ceil(math.log2(max(abs(o), 32.0))) - 7) if dtype == BF else 2.0 ** -6
        k = torch.randint(0, 32 if dtype == BF else 1024, (V,), generator=gen)
        rows.append((o + (step * k if o >= 0 else -step * k)).to(dtype))
        assert torch.equal(rows[-1].double(), o + (step if o >= 0 else -step) * k.double())
    z = torch.stack(rows + [torch.zeros(V, dtype=dtype)]).cuda()
    N = len(rows) + 1
    t = torch.randint(0, V, (N,), generator=gen).cuda()
    t[4] = -1
    g, ge = torch.randn(N, generator=gen).cuda(), torch.randn(N, generator=gen).cuda()
    res = lm.token_logprobs(z, t)
    # the forward takes differences from the row's largest logit, which are exact here: the same bits without the offset
    base = lm.token_logprobs((z.float() - z.float().amax(1, keepdim=True)).to(dtype), t)
    assert torch.equal(res.entropy, base.entropy) and torch.equal(res.logp, base.logp)
    d = lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge)
    gradient_close(d, z, t, g, ge)
    wide = torch.zeros(N, V + 3, dtype=dtype, device="cuda")     # rows off their alignment, in place
    wide[:, 1:V + 1] = z
    view = wide[:, 1:V + 1]
    assert torch.equal(lm.token_logprobs_vjp(view, t, res.lse, res.entropy, g, ge, out=view), d)
    assert (wide[:, 0] == 0).all() and (wide[:, V + 1:] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [5, 700, 9000, 70000])
def test_gradient_of_a_row_of_lowest_values(V, dtype):
    # a mask of the lowest value all over leaves a uniform distribution, whose entropy has no gradient
    z, t, g, ge = make(3, V, dtype, seed=V)
    z[1] = torch.finfo(dtype).min
    t[:] = torch.tensor([1, 2, -1])
    res = lm.token_logprobs(z, t)
    d = lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge)
    gradient_close(d, z, t, g, ge)
    one = torch.zeros(V, dtype=torch.float64)
    one[2] = 1
    want = f64(g)[1] * (one - 1 / V)
    tol = 2 * (V / 64 + 64) * U32 * (abs(float(g[1])) + abs(float(ge[1])) * (1 + math.log(V))) / V + 4 * U32 * one * abs(float(g[1]))
    close(d[1], want, rounded(want, tol, dtype), "uniform")


@pytest.mark.parametrize("V", [300, 5000, 40000])
def test_gradient_with_ruled_out_tokens_and_an_offset(V):
    z, t, g, ge = make(6, V, F32, seed=V, banned=0.4)
    z = torch.where(torch.isinf(z), z, torch.round(z * 64) / 64 + 4096.0)
    z[2], z[3, 1:], t[2] = -INF, -INF, 1
    res = lm.token_logprobs(z, t)
    d = lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge)
    assert (d[2] == 0).all()
    keep = [0, 1, 3, 4, 5]
    gradient_close(d[keep], z[keep], t[keep], g[keep], ge[keep])
    z[4, 1] = float("nan")
    res = lm.token_logprobs(z, t)
    d2 = lm.token_logprobs_vjp(z, t, res.lse, res.entropy, g, ge)
    assert torch.isnan(d2[4]).any() and torch.equal(d2[[0, 1, 2, 3, 5]], d[[0, 1, 2, 3, 5]])


@pytest.mark.parametrize("N,V", [((1 << 24) + 16, 2049), ((1 << 23) + 16, 8193)])
def test_gradient_of_more_rows_than_a_launch_has_workgroups(N, V):
    # as many rows as the forward takes, in more pieces than the 2^24 - 1 workgroups of 256 threads that a launch can have
    P = 16
    need = N * V * 2 + (4 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("%d GB of GPU memory needed" % (need >> 30))
    z, t, g, ge = make(P, V, BF, seed=V)
    z[3] = (z[3].float() * 4).round() * 0.25 + 64      # a row with an offset
    want = lm.token_logprobs(z, t)
    dwant = lm.token_logprobs_vjp(z, t, want.lse, want.entropy, g, ge)
    many = lambda a: a.repeat(N // P, *[1] * (a.dim() - 1))  # noqa: E731
    big = torch.empty(N, V, dtype=BF, device="cuda")
    big.view(N // P, P, V).copy_(z)
    out = lm.token_logprobs_vjp(big, many(t), many(want.lse), many(want.entropy), many(g), many(ge), out=big).view(N // P, P, V)
    for part in out.split(1 << 13):
        assert (part == dwant).all()
    del big, out, part
    torch.cuda.empty_cache()


def test_arguments_of_another_shape_are_refused():
    # as many values in another order would be numbers of other rows
    z = torch.randn(3, 5, 40, device="cuda")
    t = torch.zeros(3, 5, dtype=torch.int64, device="cuda")
    r = lm.token_logprobs(z, t)
    g = torch.randn(3, 5, device="cuda")
    want = lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g, g)
    turned = g.t().contiguous()
    for bad in (lambda: lm.token_logprobs_vjp(z, t, r.lse, r.entropy, turned), lambda: lm.token_logprobs_vjp(z, t, turned, r.entropy, g),
                lambda: lm.token_logprobs_vjp(z, t, r.lse, turned, g, g), lambda: lm.token_logprobs_vjp(z, t, r.lse, r.entropy, g, turned)):
        with pytest.raises(ValueError, match="must be"):
            bad()
    for same in (lambda a: a[..., None], lambda a: a[None], lambda a: a.flatten()):     # the same order of the same values
        assert torch.equal(lm.token_logprobs_vjp(z, t, same(r.lse), same(r.entropy), same(g), same(g)), want)


@pytest.mark.parametrize("offset", [0.0, 100.0, -5000.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_from_a_normaliser_of_more_logits(dtype, offset):
    # logits that are a part of their row, with the whole row's lse and entropy: p sums to less than 1, and is not made to
    gen = torch.Generator().manual_seed(11)
    N, V, half = 6, 6000, 2500
    step = 2.0 ** (math.ceil(math.log2(max(abs(offset), 32.0))) - 7) if dtype == BF else 2.0 ** -6
    z = (offset + step * torch.randint(0, 16 if dtype == BF else 512, (N, V), generator=gen)).to(dtype).cuda()
    t = torch.randint(0, half, (N,), generator=gen).cuda()
    g, ge = torch.randn(N, generator=gen).cuda(), torch.randn(N, generator=gen).cuda()
    whole = lm.token_logprobs(z, t)
    part = z[:, :half]
    got = lm.token_logprobs_vjp(part, t, whole.lse, whole.entropy, g, ge)
    # the given lse has its own rounding, u |lse|, which nothing here can know
    want = f64(lm.token_logprobs_vjp(z, t, whole.lse, whole.entropy, g, ge))[:, :half]
    l = f64(part) - f64(whole.lse)[:, None]
    size = torch.exp(l) * (f64(g).abs()[:, None] + f64(ge).abs()[:, None] * (l.abs() + f64(whole.entropy)[:, None] + 1))
    tol = (V / 64 + 64 + 2 * f64(whole.lse).abs()[:, None] + 3 * l.abs()) * U32 * size + 2 * U32 * want.abs()
    close(got, want, rounded(rounded(want, tol, dtype), rounded(want, tol, dtype), dtype), "part of a row")
