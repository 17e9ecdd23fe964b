"""The short causal convolution and its gradients (include/pararnn_block.h) against the plain 64-bit form.

Tolerances.  p is a sum of K + 1 terms: K fused steps, each off by at most u times the magnitudes added so far, (K + 1) u S with
S = |bias| + sum |w x|.  SiLU multiplies p's error by at most 1.1 and adds about 6 roundings (an exponential, a reciprocal and
products, an ulp each): u (1.1 (K + 1) S + 8 |y|).  The gradient of x sums K such products, whose slope's error is the error of p
(slope's slope is at most 0.5) and 8 roundings; the parameters' are sums of B T of them, added in a tree of chunks of at
most 64 steps: 64 u of the terms' magnitudes."""
import pytest
import torch

import block_plain as plain
from block_plain import biggest, grads, leaf
from lm_plain import U32, close, f64, rounded
from nonlinear_rnn_solve_amd import block

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(B, T, D, K, dtype, seed, n=0, state=True, layout="dense"):
    g = torch.Generator().manual_seed(seed)

    def planes(k):
        ts = [torch.randn(B, T, D, generator=g).to(dtype) for _ in range(k)]
        if layout == "slices":
            return list(torch.cat(ts, -1).cuda().split(D, -1))
        if layout == "time-major":
            return [t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in ts]
        return [t.cuda() for t in ts]

    x, dy = planes(2)
    weight, bias = torch.randn(D, K, generator=g).cuda() * 0.5, torch.randn(D, generator=g).cuda()
    shape = (B, n, K - 1, D) if n else (B, K - 1, D)
    s = torch.randn(shape, generator=g).cuda() if state else None
    dl = torch.randn(shape, generator=g).cuda() if state else None
    return x, dy, weight, bias, s, dl


def check(args, cu=None, silu=True):
    x, dy, weight, bias, state, d_last = args
    dt, K = x.dtype, weight.shape[1]
    dcu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    leaves = [leaf(t) for t in (x, weight, bias, state)]
    y, last = plain.conv(*leaves, cu=cu, act=silu)
    S = biggest(f64(bias)) + biggest(f64(weight).abs().sum(1)) * max(biggest(f64(x)), 0.0 if state is None else biggest(f64(state)))
    unit = U32 * (1.1 * (K + 1) * S + 8 * max(1.0, S))
    got_y, got_last = block.causal_conv(x, weight, bias, state=state, cu_seqlens=dcu, silu=silu)
    close(got_y, y, rounded(y, unit, dt), "y")
    close(got_last.reshape(last.shape), last, 0.0, "last")
    ref = grads((y, last), (f64(dy), None if d_last is None else f64(d_last).reshape(last.shape)), leaves)
    got = block.causal_conv_vjp(x, weight, dy, bias, state=state, d_last=d_last, cu_seqlens=dcu, silu=silu)
    # dp = dy slope(p): slopes are at most 1.1
    dp = biggest(f64(dy)) * (1.1 * 8 * U32 + 0.5 * unit)
    tx = K * biggest(f64(weight)) * (dp + 2 * U32 * 1.1 * biggest(f64(dy))) + U32 * (0.0 if d_last is None else biggest(f64(d_last)))
    close(got["d_x"], ref[0], rounded(ref[0], tx, dt), "d_x")
    if state is not None:
        close(got["d_state"].reshape(ref[3].shape), ref[3], tx, "d_state")
    steps = x.shape[0] * x.shape[1]
    size = 1.1 * biggest(f64(dy)) * max(1.0, biggest(f64(x)))
    tw = steps * (dp * max(1.0, biggest(f64(x))) + 64 * U32 * size)
    close(got["d_weight"], ref[1], tw, "d_weight")
    close(got["d_bias"], ref[2], tw, "d_bias")


SHAPES = [(1, 1, 1, 4), (2, 1, 64, 4), (3, 2, 7, 4), (2, 3, 257, 3), (1, 7, 130, 8), (2, 31, 33, 2), (2, 33, 65, 5), (1, 64, 30, 1),
          (2, 65, 70, 4), (1, 300, 1, 4), (1, 129, 2, 6), (2, 513, 48, 7), (1, 2100, 20, 4), (40, 9, 5, 4)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_convolution_and_gradients(shape, dtype):
    check(make(*shape, dtype, seed=sum(shape)))


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("layout", ["slices", "time-major"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layouts(dtype, layout, silu):
    check(make(3, 70, 95, 4, dtype, seed=3, layout=layout), silu=silu)


@pytest.mark.parametrize("cu", [[0, 70], [0, 1, 2, 3, 70], [0, 0, 33, 33, 34, 70, 70], [0, 32, 64, 70], [0, 69, 70], [0, 70, 70, 70]])
@pytest.mark.parametrize("dtype,K", [(BF, 4), (F32, 3), (F32, 8), (F32, 1)])
def test_packed(dtype, K, cu):
    check(make(2, 70, 37, K, dtype, seed=5, n=len(cu) - 1), cu=cu)


def test_many_short_sequences():
    cu = [0]
    while cu[-1] < 1500:
        cu.append(min(1500, cu[-1] + len(cu) % 5))
    check(make(1, 1500, 9, 4, F32, seed=6, n=len(cu) - 1), cu=cu)


def test_no_state_no_bias():
    x, dy, w, _, _, _ = make(2, 40, 10, 4, F32, seed=7)
    y, last = block.causal_conv(x, w)
    ref, rl = plain.conv(f64(x), f64(w))
    close(y, ref, 32 * U32 * max(1.0, biggest(ref)) * 4, "y")
    close(last, rl[:, 0], 0.0, "last")
    got = block.causal_conv_vjp(x, w, dy, want_params=False, want_state=False)
    assert set(got) == {"d_x"}


@pytest.mark.parametrize("cu", [None, [0, 0, 0]])
def test_no_steps(cu):
    x, dy, w, b, s, dl = make(2, 0, 6, 4, F32, seed=8, n=0 if cu is None else 2)
    dcu = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    y, last = block.causal_conv(x, w, b, state=s, cu_seqlens=dcu)
    assert y.shape == x.shape and torch.equal(last, s)
    got = block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl, cu_seqlens=dcu)
    assert torch.equal(got["d_state"], dl) and not got["d_weight"].any() and not got["d_bias"].any()


@pytest.mark.parametrize("T", [1, 2, 5, 200])
def test_state_updated_in_place(T):
    x, _, w, b, s, _ = make(3, T, 41, 4, BF, seed=9)
    want_y, want = block.causal_conv(x, w, b, state=s)
    mine = s.clone()
    y, last = block.causal_conv(x, w, b, state=mine, last=mine)
    assert last is mine and torch.equal(mine, want) and torch.equal(y, want_y)


def test_in_place_with_sequences():
    cu = torch.tensor([0, 5, 5, 90, 91, 200], dtype=torch.int32, device="cuda")
    x, _, w, b, s, _ = make(2, 200, 41, 4, F32, seed=10, n=5)
    want_y, want = block.causal_conv(x, w, b, state=s, cu_seqlens=cu)
    mine = s.clone()
    y, _ = block.causal_conv(x, w, b, state=mine, cu_seqlens=cu, last=mine)
    assert torch.equal(mine, want) and torch.equal(y, want_y)


def test_token_by_token_is_the_whole():
    x, _, w, b, s, _ = make(2, 12, 33, 4, F32, seed=11)
    y, last = block.causal_conv(x, w, b, state=s)
    mine = s.clone()
    for t in range(12):
        one, _ = block.causal_conv(x[:, t:t + 1], w, b, state=mine, last=mine)
        assert torch.equal(one[:, 0], y[:, t])
    assert torch.equal(mine, last)


def test_nan_stays_in_its_sequence_and_channel():
    cu = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device="cuda")
    x, dy, w, b, s, dl = make(1, 60, 8, 4, F32, seed=12, n=3)
    clean, clean_grad = block.causal_conv(x, w, b, state=s, cu_seqlens=cu)[0], None
    x[0, 39, 3] = float("nan")
    y, last = block.causal_conv(x, w, b, state=s, cu_seqlens=cu)
    bad = torch.isnan(y)
    assert bad.sum() == 1 and bad[0, 39, 3] and torch.isnan(last).sum() == 1
    assert torch.equal(y[~bad], clean[~bad])
    got = block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl, cu_seqlens=cu)
    assert torch.isfinite(got["d_x"][:, :20]).all() and torch.isfinite(got["d_x"][:, 40:]).all()
    assert torch.isfinite(got["d_x"][..., [0, 1, 2, 4, 5, 6, 7]]).all()


def test_rows_around_outputs_are_left_alone():
    x, dy, w, b, s, _ = make(2, 21, 10, 4, F32, seed=13)
    big = torch.full((2, 23, 14), 7.0, device="cuda")
    y, _ = block.causal_conv(x, w, b, state=s, out=big[:, 1:22, 2:12])
    want, _ = block.causal_conv(x, w, b, state=s)
    assert torch.equal(big[:, 1:22, 2:12], want)
    keep = torch.ones_like(big, dtype=torch.bool)
    keep[:, 1:22, 2:12] = False
    assert (big[keep] == 7).all()


def test_gradient_against_differences():
    x, dy, w, b, s, dl = make(1, 9, 3, 4, F32, seed=14)
    got = block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl)
    f = lambda x, w, b, s: sum((o * g).sum() for o, g in zip(plain.conv(x, w, b, s), (f64(dy), f64(dl)[:, None])))  # noqa: E731
    at = [f64(t) for t in (x, w, b, s)]
    for k, name in enumerate(("d_x", "d_weight", "d_bias", "d_state")):
        flat = at[k].reshape(-1)
        for i in range(0, flat.numel(), 5):
            old = float(flat[i])
            flat[i] = old + 1e-5
            up = f(*at)
            flat[i] = old - 1e-5
            down = f(*at)
            flat[i] = old
            # second differences of a smooth function of size ~100: 1e-10 each, and float32's own error
            assert abs(float(up - down) / 2e-5 - float(got[name].reshape(-1)[i])) < 1e-4, (name, i)


def test_same_bits_on_every_run_and_on_another_stream():
    args = make(2, 900, 130, 4, BF, seed=15)
    x, dy, w, b, s, dl = args
    first = (block.causal_conv(x, w, b, state=s), block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = (block.causal_conv(x, w, b, state=s), block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[0], again[0]))
    assert all(torch.equal(first[1][k], again[1][k]) for k in first[1])


def test_captured_and_replayed():
    x, dy, w, b, s, dl = make(2, 700, 66, 4, F32, seed=16)
    block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last = block.causal_conv(x, w, b, state=s)
        got = block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl)
    for k in range(3):
        x.copy_(torch.randn_like(x))
        want_y, want_last = block.causal_conv(x, w, b, state=s)
        want = block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(last, want_last)
        assert all(torch.equal(got[n], want[n]) for n in want), k


def test_wrong_offsets_stay_inside():
    # not checked (they are device memory): wrong numbers, nothing outside the arrays
    x, dy, w, b, s, dl = make(1, 64, 8, 4, F32, seed=17, n=4)
    for cu in ([0, 50, 20, 70, 64], [5, -3, 100, 100, 2], [0, 1 << 30, -(1 << 30), 3, 64]):
        dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        block.causal_conv(x, w, b, state=s, cu_seqlens=dcu)
        block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl, cu_seqlens=dcu)
    torch.cuda.synchronize()


def test_refusals():
    x, dy, w, b, s, dl = make(2, 5, 6, 4, F32, seed=18)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    for bad in (lambda: block.causal_conv(x[0], w, b), lambda: block.causal_conv(x.double(), w, b),
                lambda: block.causal_conv(x.transpose(1, 2), w, b), lambda: block.causal_conv(x, w.t(), b),
                lambda: block.causal_conv(x, torch.zeros(6, 9, device="cuda")), lambda: block.causal_conv(x, w.bfloat16(), b),
                lambda: block.causal_conv(x, w, b[:5]), lambda: block.causal_conv(x, w, b, state=s[:, :2]),
                lambda: block.causal_conv(x, w, b, state=s, cu_seqlens=cu), lambda: block.causal_conv(x, w, b, cu_seqlens=cu.long()),
                lambda: block.causal_conv(x, w, b, cu_seqlens=cu.cpu()), lambda: block.causal_conv(x, w, b, out=x[:, :1].expand(2, 5, 6)),
                lambda: block.causal_conv(x, w, b, state=s, last=s[:1]), lambda: block.causal_conv_vjp(x, w, dy.bfloat16(), b),
                lambda: block.causal_conv_vjp(x, w, dy[:, :4], b), lambda: block.causal_conv_vjp(x, w, dy, b, state=s, d_last=dl[:1]),
                lambda: block.causal_conv(x, w, b.cpu())):
        with pytest.raises(ValueError):
            bad()


def test_outputs_in_an_inputs_place_are_refused():
    x, w = torch.randn(2, 9, 8, device="cuda"), torch.randn(8, 4, device="cuda")
    dy = torch.randn_like(x)
    with pytest.raises(ValueError, match="share memory"):
        block.causal_conv(x, w, out=x)
    for t in (x, dy):
        with pytest.raises(ValueError, match="share memory"):
            block.causal_conv_vjp(x, w, dy, out=t)


def test_outputs_that_overlap_something_are_refused():
    # parts of dense tensors, and a state that leaves into a part of the one that entered; the state itself is allowed
    x, w, b = torch.randn(2, 9, 8, device="cuda"), torch.randn(8, 4, device="cuda"), torch.randn(8, device="cuda")
    flat = torch.randn(400, device="cuda")
    state, shifted = flat[:48].view(2, 3, 8), flat[24:72].view(2, 3, 8)
    beside = flat[48:96].view(2, 3, 8)
    inside = flat[100:244].view(2, 9, 8)
    for kw in (dict(state=state, last=shifted), dict(last=x.view(-1)[:48].view(2, 3, 8)), dict(last=x.view(-1)[5:53].view(2, 3, 8)),
               dict(out=inside, last=flat[200:248].view(2, 3, 8)), dict(out=flat[40:184].view(2, 9, 8), state=state)):
        with pytest.raises(ValueError, match="share memory"):
            block.causal_conv(x, w, b, **kw)
    with pytest.raises(ValueError, match="share memory"):
        block.causal_conv_vjp(flat[100:244].view(2, 9, 8), w, x, b, out=flat[150:294].view(2, 9, 8))
    want = block.causal_conv(x, w, b, state=state.clone())[1]
    block.causal_conv(x, w, b, state=state, last=beside)
    assert torch.equal(beside, want)
    block.causal_conv(x, w, b, state=state, last=state)
    assert torch.equal(state, want)
    # slices of one tensor interleave
    both = torch.randn(2, 9, 16, device="cuda")
    y, _ = block.causal_conv(both[..., :8], w, b, out=both[..., 8:])
    assert torch.equal(y, block.causal_conv(both[..., :8].clone(), w, b)[0])
