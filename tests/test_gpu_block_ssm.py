"""The selective state space scan and its gradients (include/pararnn_block.h) against the plain 64-bit recurrence.

Tolerances, u = 2^-24.  softplus and dt A are off by at most 6 u relative; the decay a = exp(dt A) by 4 u + 6 u |dt A|, and a |dt A| is
at most 0.37 for falling exponentials, so 7 u absolute.  The recurrence remembers M = min(T, 1 / min(1 - a)) steps; each adds
the decay's error times |h|, that of dt x B (8 u) and a fused step's rounding, together at most 16 u H with H the largest
|h|, |dt x B|: 16 u M H in the worst case, where all are of one sign, as the errors of one state's decay are (dt A is rounded alike in
similar steps).  y sums N such terms times |C|, plus skip x, times the gate.  The adjoint q obeys the same recurrence with
the largest |C G| + |d_last| in place of |dt x B|, so its products with h have relative errors of both.  Sums over channels or
steps are allowed their terms' magnitudes times the terms' relative error."""
import pytest
import torch

import block_plain as plain
from block_plain import biggest, grads, leaf
from lm_plain import U32, close, f64, rounded
from nonlinear_rnn_solve_amd import block

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, B, T, D, N, dtype, seed, G=1, n=0, state=True, gate=True, extra=True, layout="slices"):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        if layout == "slices":
            self.x, self.z, self.dt = r(B, T, 3 * D).to(dtype).cuda().split(D, -1) if D else [r(B, T, 0).to(dtype).cuda()] * 3
        else:
            self.x, self.z, self.dt = (r(T, B, D).to(dtype).cuda().transpose(0, 1) for _ in range(3))
        low = r(B, T, 3 + 2 * G * N).to(dtype).cuda()
        self.b, self.c = (t.unflatten(-1, (G, N)) for t in (low[..., 3:3 + G * N], low[..., 3 + G * N:]))
        if G == 1:
            self.b, self.c = self.b[:, :, 0], self.c[:, :, 0]
        self.A = (-torch.arange(1, N + 1) * torch.exp(0.1 * r(D, N))).cuda()
        self.skip, self.dt_bias = (r(D).cuda(), (r(D) - 3).cuda()) if extra else (None, None)
        shape = (B, n, D, N) if n else (B, D, N)
        self.h0 = r(*shape).cuda() if state else None
        self.dy, self.d_last = r(B, T, D).to(dtype).cuda(), r(*shape).cuda() if state else None
        if not gate:
            self.z = None

    def rest(self, cu=None):
        return dict(skip=self.skip, z=self.z, dt_bias=self.dt_bias, h0=self.h0,
                    cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))

    def forward(self, cu=None, **kw):
        return block.selective_scan(self.x, self.dt, self.A, self.b, self.c, **self.rest(cu), **kw)

    def backward(self, carry, cu=None, **kw):
        return block.selective_scan_vjp(self.x, self.dt, self.A, self.b, self.c, carry, self.dy, d_last=self.d_last,
                                        **self.rest(cu), **kw)

    def leaves(self):
        return [leaf(t) for t in (self.x, self.dt, self.A, self.b, self.c, self.skip, self.z, self.dt_bias, self.h0)]


def check(k, cu=None):
    dt = k.x.dtype
    leaves = k.leaves()
    y, last = plain.ssm(*leaves, cu=cu)
    got_y, got_last, carry = k.forward(cu, want_carry=True)
    x, delta, A, b, c, skip, z, bias, h0 = [None if t is None else t.detach() for t in leaves]
    T = x.shape[1]
    step = torch.nn.functional.softplus(delta if bias is None else delta + bias)
    a = torch.exp(step[..., None] * A)
    M = min(max(1, T), 1 / max(1e-7, float((1 - a).min()))) if a.numel() else 1
    # the states, their inputs, the adjoints and theirs, from the plain form
    with torch.no_grad():
        gate = torch.ones_like(x) if z is None else plain.silu(z)
        G = f64(k.dy) * gate
        H = max(biggest(step * x) * biggest(b) * M, 0.0 if h0 is None else biggest(h0), 1e-3)
        Q = max(biggest(G) * biggest(c) * M, 0.0, 1e-3) + (0.0 if k.d_last is None else biggest(f64(k.d_last)))
    N = A.shape[1]
    rel = 16 * U32 * M
    ty = (rel * H * N * biggest(c) + 4 * U32 * biggest(x) * (0 if skip is None else biggest(skip))) * max(1.0, biggest(gate)) + \
        8 * U32 * biggest(y)
    close(got_y, y, rounded(y, ty, dt), "y")
    close(got_last.reshape(last.shape), last, rel * H, "h_last")
    want = grads((y, last), (f64(k.dy), None if k.d_last is None else f64(k.d_last).reshape(last.shape)), leaves)
    got = k.backward(carry, cu)
    names = ("d_x", "d_dt", "d_A", "d_b", "d_c", "d_skip", "d_z", "d_dt_bias", "d_h0")
    D, S, X = x.shape[2], biggest(step), max(1.0, biggest(x))
    e = 2 * rel * Q * H                             # of one product of adjoint and state
    dd = N * e * biggest(A) + N * rel * Q * biggest(b) * X
    tol = {"d_x": N * rel * Q * biggest(b) * S + 8 * U32 * biggest(G) * (0 if skip is None else biggest(skip)),
           "d_dt": dd, "d_A": x.shape[0] * T * e * S, "d_b": D * 2 * rel * Q * S * X, "d_c": D * rel * H * biggest(G),
           "d_skip": x.shape[0] * T * 16 * U32 * biggest(G) * X, "d_z": biggest(f64(k.dy)) * 1.1 * (ty / max(1.0, biggest(gate)) + 8 * U32 * H * N * max(1.0, biggest(c))),
           "d_dt_bias": x.shape[0] * T * dd, "d_h0": rel * Q}
    for name, w in zip(names, want):
        if w is None:
            assert name in ("d_skip", "d_dt_bias", "d_h0") or name not in got
            continue
        g = got[name].reshape(w.shape)
        t = tol[name]
        close(g, w, rounded(w, t, dt) if name in ("d_x", "d_dt", "d_z", "d_b", "d_c") else t, name)
        if dt == F32 and w.numel() > 8:             # the whole is far nearer than its worst element may be
            assert float((f64(g) - w).norm()) <= 2e-5 * float(w.norm()) + 1e-12, (name, float((f64(g) - w).norm() / w.norm()))


SHAPES = [(1, 1, 1, 1), (2, 1, 64, 16), (3, 2, 7, 4), (2, 5, 65, 3), (1, 15, 130, 16), (2, 16, 33, 2), (2, 17, 65, 5), (1, 33, 64, 8),
          (2, 64, 70, 16), (1, 65, 3, 32), (1, 130, 66, 9), (2, 200, 20, 1), (1, 1030, 5, 16), (1, 700, 70, 17), (2, 333, 12, 4), (5, 48, 64, 31)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_scan_and_gradients(shape, dtype):
    check(Case(*shape, dtype, seed=sum(shape)))


@pytest.mark.parametrize("N", range(1, 33))
def test_every_number_of_states(N):
    check(Case(1, 21, 10, N, F32, seed=N))


@pytest.mark.parametrize("G,D", [(2, 6), (3, 201), (2, 256), (5, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups(G, D, dtype):
    check(Case(2, 40, D, 6, dtype, seed=G, G=G))


@pytest.mark.parametrize("kw", [dict(state=False), dict(gate=False), dict(extra=False), dict(state=False, gate=False, extra=False),
                                dict(layout="time-major")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_options_and_layouts(kw, dtype):
    check(Case(2, 75, 67, 16, dtype, seed=4, **kw))


@pytest.mark.parametrize("cu", [[0, 150], [0, 1, 2, 3, 150], [0, 0, 33, 33, 34, 150, 150], [0, 16, 64, 150], [0, 149, 150],
                                [0, 150, 150, 150], [0, 128, 144, 150], [0, 15, 16, 17, 31, 32, 33, 150]])
@pytest.mark.parametrize("dtype,N", [(BF, 16), (F32, 3), (F32, 1)])
def test_packed(dtype, N, cu):
    check(Case(2, 150, 37, N, dtype, seed=5, n=len(cu) - 1), cu=cu)


@pytest.mark.parametrize("step", [16, 80, 112])
def test_sequences_that_end_where_a_tile_or_a_segment_does(step):
    cu = list(range(0, 640, step)) + [640]
    check(Case(1, 640, 70, 4, F32, seed=5, n=len(cu) - 1), cu=cu)


def test_packed_without_states():
    check(Case(2, 150, 37, 5, F32, seed=5, n=4, state=False), cu=[0, 3, 70, 70, 150])


def test_many_short_sequences():
    cu = [0]
    while cu[-1] < 600:
        cu.append(min(600, cu[-1] + len(cu) % 5))
    check(Case(1, 600, 9, 4, F32, seed=6, n=len(cu) - 1), cu=cu)


@pytest.mark.parametrize("cu", [None, [0, 0, 0]])
def test_no_steps(cu):
    k = Case(2, 0, 6, 4, F32, seed=8, n=0 if cu is None else 2)
    y, last, carry = k.forward(cu, want_carry=True)
    assert y.shape == k.x.shape and torch.equal(last, k.h0)
    got = k.backward(carry, cu)
    assert torch.equal(got["d_h0"], k.d_last) and not got["d_A"].any() and not got["d_skip"].any()


@pytest.mark.parametrize("cu", [None, [0, 5, 5, 90, 91, 999, 2000], [0, 1000, 2000], [0, 64, 2000, 2000]])
@pytest.mark.parametrize("T", [1, 3, 2000])
def test_state_updated_in_place(T, cu):
    if cu is not None:
        if T < 2000:
            pytest.skip("the offsets are of the long row")
    k = Case(2, T, 41, 16, BF, seed=9, n=0 if cu is None else len(cu) - 1)
    want_y, want, _ = k.forward(cu)
    k.h0 = k.h0.clone()
    y, last, _ = k.forward(cu, h_last=k.h0)
    assert last is k.h0 and torch.equal(last, want) and torch.equal(y, want_y)


def test_token_by_token_is_the_whole():
    k = Case(2, 40, 33, 16, F32, seed=11)
    y, last, _ = k.forward()
    h = k.h0.clone()
    for t in range(40):
        s = slice(t, t + 1)
        one, _, _ = block.selective_scan(k.x[:, s], k.dt[:, s], k.A, k.b[:, s], k.c[:, s], skip=k.skip, z=k.z[:, s],
                                         dt_bias=k.dt_bias, h0=h, h_last=h)
        assert torch.equal(one[:, 0], y[:, t]), t
    assert torch.equal(h, last)


def test_nan_and_infinity_stay_in_their_sequence_and_channel():
    cu = [0, 200, 400, 600]
    k = Case(1, 600, 70, 16, F32, seed=12, n=3)
    clean = k.forward(cu)[0]
    x = k.x.clone()
    x[0, 399, 3], x[0, 230, 66] = float("nan"), float("inf")
    k.x = x
    y, last, carry = k.forward(cu, want_carry=True)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 399, 3] = hit[0, 230:400, 66] = True
    assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[0, 399, 3])
    assert torch.isfinite(last[:, [0, 2]]).all() and not torch.isfinite(last[:, 1, 3]).any()
    got = k.backward(carry, cu)
    for name in ("d_x", "d_dt", "d_z"):
        assert torch.isfinite(got[name][:, :200]).all() and torch.isfinite(got[name][:, 400:]).all(), name
    keep = [d for d in range(70) if d not in (3, 66)]
    assert torch.isfinite(got["d_x"][..., keep]).all() and torch.isfinite(got["d_A"][keep]).all()


def test_extreme_steps():
    # dt pre-activations far out: a step of zero holds the state, a huge one forgets it
    k = Case(1, 40, 8, 4, F32, seed=13)
    k.dt = k.dt.clone()
    k.dt[0, 10:20], k.dt[0, 30] = -200.0, 150.0
    y, last, carry = k.forward(want_carry=True)
    want, wl = plain.ssm(*[t.detach() if t is not None else None for t in k.leaves()])
    close(y, want, 1e-4 * max(1.0, biggest(want)), "y")
    got = k.backward(carry)
    assert all(torch.isfinite(t).all() for t in got.values())


def test_rows_around_outputs_are_left_alone():
    k = Case(2, 21, 10, 4, F32, seed=14)
    big = torch.full((2, 23, 14), 7.0, device="cuda")
    k.forward(out=big[:, 1:22, 2:12])
    assert torch.equal(big[:, 1:22, 2:12], k.forward()[0])
    big[:, 1:22, 2:12] = 7
    assert (big == 7).all()


def test_gradients_into_slices():
    k = Case(2, 50, 10, 4, BF, seed=15)
    carry = k.forward(want_carry=True)[2]
    want = k.backward(carry)
    wide, low = torch.zeros(2, 50, 30, device="cuda", dtype=BF), torch.zeros(2, 50, 8, device="cuda", dtype=BF)
    got = k.backward(carry, out=[wide[..., :10], wide[..., 10:20], wide[..., 20:], low[..., :4], low[..., 4:]])
    assert got["d_x"].data_ptr() == wide.data_ptr()
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_gradient_against_differences():
    k = Case(1, 7, 3, 2, F32, seed=16)
    got = k.backward(k.forward(want_carry=True)[2])
    at = [f64(t) for t in (k.x, k.dt, k.A, k.b, k.c, k.skip, k.z, k.dt_bias, k.h0)]
    f = lambda *a: sum((o * g).sum() for o, g in zip(plain.ssm(*a), (f64(k.dy), f64(k.d_last)[:, None])))  # noqa: E731
    for i, name in enumerate(("d_x", "d_dt", "d_A", "d_b", "d_c", "d_skip", "d_z", "d_dt_bias", "d_h0")):
        flat = at[i].reshape(-1) if at[i].is_contiguous() else None
        if flat is None:
            at[i] = at[i].contiguous()
            flat = at[i].reshape(-1)
        for j in range(0, flat.numel(), 3):
            old = float(flat[j])
            flat[j] = old + 1e-5
            up = f(*at)
            flat[j] = old - 1e-5
            down = f(*at)
            flat[j] = old
            assert abs(float(up - down) / 2e-5 - float(got[name].reshape(-1)[j])) < 2e-4, (name, j)


def test_same_bits_on_every_run_and_on_another_stream():
    k = Case(2, 900, 130, 16, BF, seed=17)

    def both():
        y, last, carry = k.forward(want_carry=True)
        return [y, last, carry] + list(k.backward(carry).values())

    first = both()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_and_replayed():
    k = Case(2, 1200, 66, 16, F32, seed=18)

    def both():
        y, last, carry = k.forward(want_carry=True)
        return [y, last] + list(k.backward(carry).values())

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for n in range(3):
        k.dy.copy_(torch.randn_like(k.dy))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n


def test_wrong_offsets_stay_inside():
    k = Case(1, 640, 8, 4, F32, seed=19, n=4)
    for cu in ([0, 500, 200, 700, 640], [5, -3, 1000, 1000, 2], [0, 1 << 30, -(1 << 30), 3, 640]):
        carry = k.forward(cu, want_carry=True)[2]
        k.backward(carry, cu)
    torch.cuda.synchronize()


def test_refusals():
    k = Case(2, 5, 6, 4, F32, seed=20)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    scan = lambda **kw: block.selective_scan(**{**dict(x=k.x, dt=k.dt, A=k.A, b=k.b, c=k.c), **kw})  # noqa: E731
    for bad in (dict(x=k.x[0]), dict(x=k.x.double()), dict(dt=k.dt.bfloat16()), dict(dt=k.dt[:, :4]), dict(A=k.A.t()), dict(A=k.A[:5]),
                dict(A=torch.zeros(6, 33, device="cuda")), dict(b=k.b[..., :3]), dict(b=k.b.bfloat16()), dict(c=k.c[:1]),
                dict(b=k.b[:, :, None].expand(2, 5, 4, 4), c=k.c[:, :, None].expand(2, 5, 4, 4)), dict(skip=k.skip[:5]),
                dict(z=k.z[..., :5]), dict(dt_bias=k.dt_bias.cpu()), dict(h0=k.h0[:1]), dict(h0=k.h0, cu_seqlens=cu),
                dict(cu_seqlens=cu.long()), dict(h_last=k.h0[:1]), dict(out=k.x[:, :1].expand(2, 5, 6))):
        with pytest.raises(ValueError):
            scan(**bad)
    carry = k.forward(want_carry=True)[2]
    for bad in (lambda: k.backward(None), lambda: k.backward(carry[:, :, :3]), lambda: k.backward(carry, out=[None] * 4),
                lambda: k.backward(carry, out=[k.x[:, :1].expand(2, 5, 6)] + [None] * 4)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("B,T,D,cu", [(2, 5, 33, None), (2, 21, 65, None), (1, 1003, 64, None), (1, 1003, 40, [0, 18, 18, 519, 1003])])
def test_state_that_forgets_at_once(B, T, D, cu):
    # exp(s A) is 0 for A = -inf and for -1e30 alike (s > 1e-20 here): the same bits
    k = Case(B, T, D, 5, F32, 71, n=len(cu) - 1 if cu else 0)
    k.A[:, 2] = -1e30
    want = k.forward(cu)[:2]
    k.A[:, 2] = float("-inf")
    for a, w in zip(k.forward(cu)[:2], want):
        assert torch.isfinite(a).all() and torch.equal(a, w)


def test_outputs_in_an_inputs_place_are_refused():
    k = Case(1, 20, 8, 4, F32, 72)
    carry = k.forward(want_carry=True)[2]
    for t in (k.x, k.z, k.dt):
        with pytest.raises(ValueError, match="share memory"):
            k.forward(out=t)
    one = torch.empty_like(k.dy)
    for out in ([k.dy] + [None] * 4, [one, one, None, None, None], [None, None, None, k.b, None]):
        with pytest.raises(ValueError, match="share memory"):
            k.backward(carry, out=out)


@pytest.mark.parametrize("B,T,D,cu", [(2, 5, 33, None), (2, 21, 65, None), (2, 33, 64, None), (1, 1003, 64, None), (1, 1003, 40, [0, 18, 18, 519, 1003])])
def test_gradients_of_a_state_that_forgets_at_once(B, T, D, cu):
    # as forward: A = -inf gives the bits of A = -1e30, and nothing past a row's end or its last channel reaches the sums
    k = Case(B, T, D, 5, F32, 71, n=len(cu) - 1 if cu else 0)
    k.A[:, 2] = -1e30
    want = k.backward(k.forward(cu, want_carry=True)[2], cu)
    k.A[:, 2] = float("-inf")
    got = k.backward(k.forward(cu, want_carry=True)[2], cu)
    for name in set(want) - {"d_dt", "d_dt_bias"}:
        assert torch.isfinite(got[name]).all() and torch.equal(got[name], want[name]), name


def test_one_channels_infinite_state_leaves_the_others_sums():
    # the last channel's state is infinite: lanes past it must not make a NaN of the sums over channels, where its own term is infinite
    k = Case(1, 40, 65, 4, F32, 74, gate=False)
    k.h0 = k.h0.clone()
    k.h0[0, 64, 1] = float("inf")
    k.dy = torch.ones_like(k.dy)
    got = k.backward(k.forward(want_carry=True)[2])
    assert torch.isposinf(got["d_c"][..., 1]).all() and torch.isfinite(got["d_c"][..., [0, 2, 3]]).all()
    assert torch.isfinite(got["d_b"]).all() and torch.isfinite(got["d_x"]).all()


@pytest.mark.parametrize("T,quiet", [(1003, 990), (4003, 3900)])
def test_growth_past_float32_in_a_quiet_row(T, quiet):
    # rates of 1 and steps of log 2: 2^T over the row.  x is zero up to step `quiet`, so the states are, and stay below 2^115 after it; the
    # steps before the last are cut into segments, each of which would multiply a zero by an infinity
    k = Case(1, T, 40, 3, F32, 75, state=False)
    k.A = torch.ones_like(k.A)
    k.dt, k.dt_bias, k.x = torch.zeros_like(k.dt), torch.zeros_like(k.dt_bias), k.x.clone()
    k.x[:, :quiet] = 0
    y, last, carry = k.forward(want_carry=True)
    want, wl = plain.ssm(*[t.detach() if t is not None else None for t in k.leaves()])
    assert not y[:, :quiet].any() and torch.isfinite(y).all()
    # each of the steps after it adds 16 u of the largest state so far (as above), and the state doubles: 2 x 16 u of its magnitudes
    magnitudes = plain.ssm(*[t.detach().abs() if t is not None and i not in (1, 2, 7) else t if t is None else t.detach() for i, t in enumerate(k.leaves())])[1]
    close(last, wl[:, 0], 16 * U32 * (T - quiet) * magnitudes[:, 0], "h_last")
    # the other way: only the first steps have a gradient, so nothing flows back to them
    k.dy = k.dy.clone()
    k.dy[:, T - quiet:] = 0
    got = k.backward(carry)
    assert all(torch.isfinite(t).all() for t in got.values())
    assert not got["d_x"][:, T - quiet:].any() and got["d_x"][:, :T - quiet].any()


def test_growth_past_float32_of_a_small_state():
    # h = 2^-100 grows by 2^150 over a row of several segments: 2^50, though the factor is infinite
    T = 2000
    k = Case(1, T, 64, 4, F32, 76)
    k.A, k.dt, k.dt_bias = torch.full_like(k.A, 150 / T), torch.zeros_like(k.dt), torch.zeros_like(k.dt_bias)
    k.x, k.h0 = torch.zeros_like(k.x), torch.full_like(k.h0, 2.0 ** -100)
    y, last, _ = k.forward()
    # log 2 and A are off by 3 u together, so the exponent 104 = 150 log 2 by 312 u; each of its steps adds 4 u
    close(last, torch.full((1, 64, 4), 2.0 ** 50, dtype=torch.float64), 2.0 ** 50 * U32 * (312 + 4 * T), "h_last")


def test_a_single_steps_stride_means_nothing():
    # [B, 1, D] planes whose (unused) step is 2^24 elements and more, forward and backward, outputs too
    k = Case(3, 1, 8, 4, F32, 77)
    y, last, carry = k.forward(want_carry=True)
    want = k.backward(carry)

    def far(t):
        s = torch.empty(t.numel(), device="cuda")
        v = torch.as_strided(s, t.shape, (t.shape[2], 1 << 24, 1))
        return v.copy_(t)

    k.x, k.dt, k.z, k.b, k.c, k.dy = (far(t) for t in (k.x, k.dt, k.z, k.b, k.c, k.dy))
    got_y, got_last, got_carry = k.forward(want_carry=True, out=far(torch.zeros_like(y)))
    assert torch.equal(got_y, y) and torch.equal(got_last, last) and torch.equal(got_carry, carry)
    got = k.backward(carry, out=[far(torch.zeros_like(want[n])) for n in ("d_x", "d_dt", "d_z", "d_b", "d_c")])
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_outputs_that_overlap_something_are_refused():
    k = Case(2, 20, 8, 4, F32, 78)
    flat = torch.randn(1000, device="cuda")
    k.h0 = flat[:64].view(2, 8, 4)
    for kw in (dict(h_last=flat[32:96].view(2, 8, 4)), dict(h_last=flat[200:264].view(2, 8, 4), out=flat[240:560].view(2, 20, 8)),
               dict(out=flat[60:380].view(2, 20, 8))):
        with pytest.raises(ValueError, match="share memory"):
            k.forward(**kw)
    k.skip = flat[600:608]
    with pytest.raises(ValueError, match="share memory"):
        k.forward(h_last=flat[590:654].view(2, 8, 4))
    carry = k.forward(want_carry=True)[2]
    for out in ([None, flat[:320].view(2, 20, 8), None, None, None], [flat[500:820].view(2, 20, 8), None, None, None, None]):
        with pytest.raises(ValueError, match="share memory"):
            k.backward(carry, out=out)
    want = k.forward()[1]
    _, last, _ = k.forward(h_last=flat[64:128].view(2, 8, 4))
    assert torch.equal(last, want)
    _, last, _ = k.forward(h_last=k.h0)
    assert torch.equal(k.h0, want)
