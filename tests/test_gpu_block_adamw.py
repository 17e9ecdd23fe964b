"""The AdamW step over many tensors (include/pararnn_block.h) against the plain 64-bit form.

Tolerances, u = 2^-24: a moment is two products and a sum, 3 u of the terms' magnitudes; the update is made of about 8 roundings,
relative to its own size, plus what the moments' errors do to it.  The sum m may cancel: its error 3 u (b1 |m0| + (1 - b1) |g|) is
relative to its terms and not to m, so the update's is relative to R, the update made of the terms' magnitudes, which is at least
|update|.  v has no cancellation.  So 16 u R holds for all of it.  A moment in 8 bits is one of the two codes next to its value."""
import pytest
import torch

import block_plain as plain
from lm_plain import U16, U32, close, f64
from nonlinear_rnn_solve_amd import block

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SIZES = [(1,), (255,), (256,), (257,), (33, 65), (5000,), (16385,), (3, 1, 7), (0,), (40001,)]


def make(sizes, seed, pt=F32, gt=F32):
    g = torch.Generator().manual_seed(seed)
    params = [torch.randn(s, generator=g).to(pt).cuda() for s in sizes]
    grads = [(torch.randn(s, generator=g) * 1e-2).to(gt).cuda() for s in sizes]
    return params, grads


def places(params):
    at, out = 0, []
    for p in params:
        out.append(slice(at, at + p.numel()))
        at += -(-p.numel() // block.ADAMW_BLOCK) * block.ADAMW_BLOCK
    return out, at


def magnitudes(o, g, om, v, step, grad_scale=1.0):
    """R: the update with the magnitudes of m's terms in m's place; v is the new one."""
    (b1, b2), lr = HYPER["betas"], HYPER["lr"]
    m = b1 * om.reshape(o.shape).abs() + (1 - b1) * (f64(g) * grad_scale).abs()
    return lr * (m / (1 - b1 ** step)) / (torch.sqrt(v / (1 - b2 ** step)) + HYPER["eps"])


def check_params(params, old, want, reach):
    for p, o, w, r in zip(params, old, want, reach):
        tol = 16 * U32 * (o.abs() + r) + 1e-12
        if p.dtype == BF:
            tol = tol + U16 * (w.abs() + tol)
        close(p, w, tol, "param")


@pytest.mark.parametrize("pt,gt", [(F32, F32), (F32, BF), (BF, BF), (BF, F32)])
def test_steps_in_32_bits(pt, gt):
    params, grads = make(SIZES, 1, pt, gt)
    where, total = places(params)
    assert block.adamw_state_size(params) == total
    m, v = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
    for step in (1, 2, 3):
        old, om, ov = [f64(p) for p in params], f64(m), f64(v)
        block.adamw_step(params, grads, m, v, step, grad_scale=0.5, **HYPER)
        want = [plain.adamw(o, f64(g), om[w].reshape(o.shape), ov[w].reshape(o.shape), step, grad_scale=0.5, **HYPER)
                for o, g, w in zip(old, grads, where)]
        check_params(params, old, [x[0] for x in want],
                     [magnitudes(o, g, om[w], x[2], step, 0.5) for o, g, w, x in zip(old, grads, where, want)])
        for x, w, g in zip(want, where, grads):
            close(m[w], x[1].reshape(-1), 4 * U32 * (om[w].abs() + f64(g).abs().reshape(-1)), "m")
            close(v[w], x[2].reshape(-1), 4 * U32 * x[2].reshape(-1) + 1e-40, "v")
        grads = [torch.randn_like(g.float()).to(gt) * 1e-2 for g in grads]


def test_many_tensors_and_mixed_types():
    # more than one launch's worth, of all four pairs of types
    g = torch.Generator().manual_seed(2)
    params, grads = [], []
    for k in range(300):
        n = int(torch.randint(1, 700, (1,), generator=g))
        params.append(torch.randn(n, generator=g).to((F32, BF)[k % 2]).cuda())
        grads.append(torch.randn(n, generator=g).to((F32, BF)[k // 2 % 2]).cuda())
    where, total = places(params)
    m, v = torch.zeros(total, device="cuda"), torch.zeros(total, device="cuda")
    old = [f64(p) for p in params]
    block.adamw_step(params, grads, m, v, 1, **HYPER)
    zero = [torch.zeros_like(o) for o in old]
    want = [plain.adamw(o, f64(g), z, z, 1, **HYPER) for o, g, z in zip(old, grads, zero)]
    check_params(params, old, [x[0] for x in want], [magnitudes(o, g, z, x[2], 1) for o, g, z, x in zip(old, grads, zero, want)])


@pytest.mark.parametrize("gt", [F32, BF])
def test_steps_in_8_bits(gt):
    params, grads = make(SIZES, 3, F32, gt)
    where, total = places(params)
    m, v = (torch.zeros(total, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(total // 256, device="cuda") for _ in range(2))
    tables = {"m": plain.values(15), "v": plain.values(31)}
    decode = lambda code, scale, t: t[code.cpu().long()] * f64(scale).repeat_interleave(256)  # noqa: E731
    for step in (1, 2, 3, 4):
        old, om, ov = [f64(p) for p in params], decode(m, ms, tables["m"]), decode(v, vs, tables["v"])
        block.adamw_step(params, grads, m, v, step, m_scale=ms, v_scale=vs, seed=7, **HYPER)
        want = [plain.adamw(o, f64(g), om[w].reshape(o.shape), ov[w].reshape(o.shape), step, **HYPER)
                for o, g, w in zip(old, grads, where)]
        check_params(params, old, [x[0] for x in want],
                     [magnitudes(o, g, om[w], x[2], step) for o, g, w, x in zip(old, grads, where, want)])
        for name, code, scale, k in (("m", m, ms, 1), ("v", v, vs, 2)):
            full = torch.zeros(total, dtype=torch.float64)
            for x, w in zip(want, where):
                full[w] = x[k].reshape(-1)
            most = full.abs().reshape(-1, 256).amax(1)
            # the smallest power of two that holds the block (float32's rounding of the largest value moves none here)
            e = torch.ceil(torch.log2(most.clamp(min=1e-30) / 1.875)).clamp(min=-80)
            assert torch.equal(f64(scale), torch.where(most > 0, 2.0 ** e, torch.full_like(e, 2.0 ** -80))), name
            y = full / f64(scale).repeat_interleave(256)
            got, table = tables[name][code.cpu().long()], tables[name].unique().sort().values
            below = table[torch.searchsorted(table, y * (1 - 8 * U32 * y.sign()), right=True) - 1]
            at = torch.searchsorted(table, y - y.abs() * 8 * U32, right=True) - 1
            lo, hi = table[at.clamp(min=0)], table[(at + 1).clamp(max=len(table) - 1)]
            # one of the two codes next to the value (or a third, where float32's error moves it over a code)
            ok = ((got >= lo) & (got <= hi)) | ((got - y).abs() <= (hi - lo) * (1 + 1e-6)) | (got == below)
            assert ok.all(), (name, step)
        am, av = block.adamw_moments(m, v, ms, vs)
        assert torch.equal(f64(am), decode(m, ms, tables["m"])) and torch.equal(f64(av), decode(v, vs, tables["v"]))
        grads = [torch.randn_like(g.float()).to(gt) * 1e-2 for g in grads]


def test_rounding_keeps_the_mean():
    # one value in every block next to its largest: the mean of 2^18 independent roundings of a value x between two codes a step
    # s apart is off by 6 s / 2 / 2^9 with a probability of 2e-9, and by the 16 bits' 2^-16 s
    n = 1 << 18
    p = [torch.zeros(n, device="cuda")]
    g = torch.full((n,), 0.0123, device="cuda")
    g[::256] = 1.0
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(n // 256, device="cuda") for _ in range(2))
    block.adamw_step(p, [g], m, v, 1, betas=(0.0, 0.0), m_scale=ms, v_scale=vs, seed=11)
    am, av = block.adamw_moments(m, v, ms, vs)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::256] = False
    for got, x in ((am, 0.0123), (av, 0.0123 ** 2)):
        some = f64(got)[rest.cpu()]
        step = float(some.max() - some.min())
        assert 0 < step <= x / 8 + 1e-12 and len(some.unique()) == 2
        assert abs(float(some.mean()) - x) <= step * (6 / 2 / 2 ** 9 + 2 ** -15), (float(some.mean()), x)
    # the two moments' numbers are independent of each other: up together as often as chance has it
    um, uv = f64(am)[rest.cpu()] > 0.0123, f64(av)[rest.cpu()] > 0.0123 ** 2
    joint, apart = float((um & uv).double().mean()), float(um.double().mean() * uv.double().mean())
    assert abs(joint - apart) < 6 / 2 / 2 ** 9


def test_seed_and_step_change_the_rounding():
    def run(step, seed):
        params, grads = make([(4096,)], 4)
        m, v = (torch.zeros(4096, dtype=torch.uint8, device="cuda") for _ in range(2))
        ms, vs = (torch.zeros(16, device="cuda") for _ in range(2))
        block.adamw_step(params, grads, m, v, step, m_scale=ms, v_scale=vs, seed=seed, **HYPER)
        return torch.cat([m, v])

    base = run(1, 0)
    assert torch.equal(base, run(1, 0))
    for other in (run(2, 0), run(1, 1), run(1, 1 << 40), run((1 << 32) + 1, 0)):
        assert 0.05 < float((base != other).float().mean()) < 0.6


def test_nan_and_extremes():
    n = 1024
    params, grads = make([(n,)], 5)
    grads[0][300] = float("nan")
    grads[0][600] = float("inf")
    grads[0][800:1024] = 0.0
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(n // 256, device="cuda") for _ in range(2))
    block.adamw_step(params, grads, m, v, 1, m_scale=ms, v_scale=vs, **HYPER)
    am, av = block.adamw_moments(m, v, ms, vs)
    assert torch.isnan(am[256:768]).all() and torch.isnan(av[256:768]).all()
    assert torch.isfinite(am[:256]).all() and torch.isfinite(av[768:]).all() and not am[800:].any()
    assert torch.isnan(params[0][300]) and torch.isfinite(params[0][:256]).all()
    # gradients beyond what a moment's scale holds: huge and tiny ones
    params, _ = make([(512,)], 6)
    grads = [torch.cat([torch.full((256,), 1e18), torch.full((256,), 1e-25)]).cuda()]
    m, v = (torch.zeros(512, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros(2, device="cuda") for _ in range(2))
    block.adamw_step(params, grads, m, v, 1, m_scale=ms, v_scale=vs, **HYPER)
    am, av = block.adamw_moments(m, v, ms, vs)
    assert torch.isfinite(am).all() and torch.isfinite(av).all() and torch.isfinite(params[0]).all()
    assert ((f64(am[:256]) - 1e17).abs() <= 1e17 / 8).all() and ((f64(av[:256]) - 5e34).abs() <= 5e34 / 8).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_elements_past_a_tensors_end(bits):
    params, grads = make([(300,), (5,)], 7)
    backing = torch.full((400,), 7.0, device="cuda")
    backing[:300] = params[0]
    params[0] = backing[:300]
    kind = torch.uint8 if bits == 8 else F32
    m, v = (torch.full((768,), 9, dtype=kind, device="cuda") for _ in range(2))
    kw = dict(m_scale=torch.ones(3, device="cuda"), v_scale=torch.ones(3, device="cuda")) if bits == 8 else {}
    block.adamw_step(params, grads, m, v, 1, **kw, **HYPER)
    assert (backing[300:] == 7).all()
    for t in (m, v):
        assert (t[300:512] == (0 if bits == 8 else 9)).all() and (t[517:] == (0 if bits == 8 else 9)).all()


def test_unaligned_tensors():
    for pt, gt in ((F32, F32), (BF, BF)):
        flat, gflat = torch.randn(5000, device="cuda").to(pt), torch.randn(5000, device="cuda").to(gt)
        params, grads = [flat[1:1000], flat[1001:4998]], [gflat[3:1002], gflat[1003:5000]]
        copy = [p.clone() for p in params]
        m, v = (torch.zeros(block.adamw_state_size(params), device="cuda") for _ in range(2))
        m2, v2 = m.clone(), v.clone()
        ends = flat[[0, 1000, 4998, 4999]].clone()
        block.adamw_step(params, grads, m, v, 1, **HYPER)
        block.adamw_step(copy, [g.clone() for g in grads], m2, v2, 1, **HYPER)
        assert all(torch.equal(a, b) for a, b in zip(params, copy)) and torch.equal(m, m2) and torch.equal(v, v2)
        assert torch.equal(flat[[0, 1000, 4998, 4999]], ends)


@pytest.mark.parametrize("bits", [8, 32])
def test_device_numbers_and_replays(bits):
    def state():
        params, grads = make(SIZES, 8)
        total = block.adamw_state_size(params)
        m, v = (torch.zeros(total, dtype=torch.uint8 if bits == 8 else F32, device="cuda") for _ in range(2))
        kw = dict(m_scale=torch.zeros(total // 256, device="cuda"), v_scale=torch.zeros(total // 256, device="cuda")) if bits == 8 else {}
        return params, grads, m, v, kw

    hyper = dict(betas=(0.9, 0.95), weight_decay=0.1, seed=3)
    a, b = state(), state()
    step, lr, scale = (torch.tensor(x, device="cuda") for x in (0, 0.0, 1.0))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            block.adamw_step(a[0], a[1], a[2], a[3], step, lr=lr, grad_scale=scale, **a[4], **hyper)
    torch.cuda.current_stream().wait_stream(side)
    for n in range(1, 5):
        step.fill_(n), lr.fill_(n * 0.25), scale.fill_(0.5 ** n)
        for g, h in zip(a[1], b[1]):
            g.copy_(torch.randn_like(g))
            h.copy_(g)
        graph.replay()
        block.adamw_step(b[0], b[1], b[2], b[3], n, lr=n * 0.25, grad_scale=0.5 ** n, **b[4], **hyper)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a[0] + [a[2], a[3]], b[0] + [b[2], b[3]])), n


def test_follows_torch():
    # torch's AdamW on the same gradients in float64: 50 steps of float32 stay within 50 steps' roundings
    params, _ = make([(700,), (33, 9)], 9)
    ref = [f64(p).requires_grad_() for p in params]
    opt = torch.optim.AdamW(ref, lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m, v = (torch.zeros(block.adamw_state_size(params), device="cuda") for _ in range(2))
    for step in range(1, 51):
        grads = [torch.randn_like(p) for p in params]
        for r, g in zip(ref, grads):
            r.grad = f64(g)
        opt.step()
        block.adamw_step(params, grads, m, v, step, **HYPER)
    for p, r in zip(params, ref):
        close(p, r, 50 * 16 * U32 * (r.detach().abs() + 50 * 3e-3), "param")


def test_written_tensors_count_as_modified():
    params, grads = make([(10,)], 10)
    m, v = (torch.zeros(256, device="cuda") for _ in range(2))
    before = params[0]._version, m._version
    block.adamw_step(params, grads, m, v, 1)
    assert params[0]._version > before[0] and m._version > before[1]
    leaf = torch.nn.Parameter(torch.ones(10, device="cuda"))
    block.adamw_step([leaf], grads, m, v, 1)
    assert not torch.equal(leaf.detach(), torch.ones(10, device="cuda"))


def test_refusals():
    params, grads = make([(10,), (20, 3)], 11)
    m, v = (torch.zeros(512, device="cuda") for _ in range(2))
    m8, v8, s = m.to(torch.uint8), v.to(torch.uint8), torch.ones(2, device="cuda")
    for bad in (lambda: block.adamw_step(params, grads[:1], m, v, 1), lambda: block.adamw_step(params, [grads[0], grads[1].t()], m, v, 1),
                lambda: block.adamw_step([params[0], params[1].t()], [grads[0], grads[1].t()], m, v, 1),
                lambda: block.adamw_step([params[0], params[0]], [grads[0], grads[0]], m, v, 1),
                lambda: block.adamw_step([params[1].view(-1)[:20], params[1].view(-1)[19:40]], [grads[1].view(-1)[:20], grads[1].view(-1)[19:40]], m, v, 1),
                lambda: block.adamw_step([p.half() for p in params], grads, m, v, 1), lambda: block.adamw_step(params, [g.cpu() for g in grads], m, v, 1),
                lambda: block.adamw_step(params, grads, m[:256], v, 1), lambda: block.adamw_step(params, grads, m, v8, 1),
                lambda: block.adamw_step(params, grads, m.bfloat16(), v, 1), lambda: block.adamw_step(params, grads, m8, v8, 1),
                lambda: block.adamw_step(params, grads, m8, v8, 1, m_scale=s, v_scale=s[:1]), lambda: block.adamw_step(params, grads, m, v, 1, m_scale=s),
                lambda: block.adamw_step(params, grads, m, v, torch.ones(1, device="cuda")), lambda: block.adamw_step(params, grads, m, v, 1, lr=torch.ones(2, device="cuda")),
                lambda: block.adamw_moments(m, v, s, s), lambda: block.adamw_moments(m8[:100], v8[:100], s, s), lambda: block.adamw_moments(m8, v8, s, None)):
        with pytest.raises(ValueError):
            bad()
    for bad in (dict(step=0), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0), dict(lr=float("nan")), dict(weight_decay=float("inf"))):
        with pytest.raises(block.PararnnError):
            block.adamw_step(params, grads, m, v, **{"step": 1, **bad})
    block.adamw_step([], [], m[:0], v[:0], 1)


def test_moments_that_share_memory_are_refused():
    p, g = torch.zeros(600, device="cuda"), torch.ones(600, device="cuda")
    n = block.adamw_state_size([p])
    m = torch.zeros(n, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        block.adamw_step([p], [g], m, m, 1)
    q = torch.zeros(n, device="cuda")[:600]
    with pytest.raises(ValueError, match="overlap"):
        block.adamw_step([q], [g], q.new_empty(0).set_(q.untyped_storage()), m, 1)
    m8, v8, s = (torch.zeros(k, dtype=t, device="cuda") for k, t in ((n, torch.uint8), (n, torch.uint8), (n // 256, torch.float32)))
    with pytest.raises(ValueError, match="overlap"):
        block.adamw_step([p], [g], m8, v8, 1, m_scale=s, v_scale=s)
    assert not p.any() and not m8.any()


@pytest.mark.parametrize("lr,decay", [(1e-6, 0.1), (1e-7, 0.25), (1e-5, 0.01), (1e-4, 0.1), (1e-3, 0.1)])
def test_small_decays(lr, decay):
    # without gradients p is taken p lr decay, off by 4 u of that (lr, decay, their product, the product), and rounded once: by half a step
    p = torch.randn(1 << 16, generator=torch.Generator().manual_seed(12)).cuda()
    want = f64(p) * (1 - lr * decay)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    block.adamw_step([p], [torch.zeros_like(p)], m, v, 1, lr=lr, weight_decay=decay)
    half = 2.0 ** (torch.floor(torch.log2(want.abs())) - 24)
    close(p, want, half + 5 * U32 * lr * decay * want.abs(), "param")


@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_infinite_parameters_stay(decay):
    p = torch.tensor([float("inf"), float("-inf"), 1.0], device="cuda")
    m, v = (torch.zeros(256, device="cuda") for _ in range(2))
    block.adamw_step([p], [torch.tensor([0.5, 0.0, 0.0], device="cuda")], m, v, 1, lr=0.5, weight_decay=decay)
    assert p[:2].tolist() == [float("inf"), float("-inf")]
    close(p[2:], torch.tensor([1.0 - 0.5 * decay], dtype=torch.float64), U32, "param")        # one rounding below 1, and decay's own


def test_rounding_of_ties():
    # 17/16 is halfway between two codes: m goes up where the element's number is 2^19 / 2^20 or more, v where it is more.  One in 2^16 is just that
    def mix(x):
        x = (x ^ (x >> 16)) * 0x7FEB352D & 0xFFFFFFFF
        x = (x ^ (x >> 15)) * 0x846CA68B & 0xFFFFFFFF
        return x ^ (x >> 16)

    n, seed, step = 1 << 21, 7, 3
    h = mix(torch.arange(n) ^ mix(mix(torch.tensor(seed) ^ mix(torch.tensor(step)))))
    for power, name in ((1, "m"), (2, "v")):
        g = torch.full((n,), float(torch.tensor(17 / 16, dtype=torch.float64) ** (1 / power)), device="cuda")
        assert float(g[0] ** power) == 17 / 16
        p = [torch.zeros(n, device="cuda")]
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        ms, vs = (torch.zeros(n // 256, device="cuda") for _ in range(2))
        block.adamw_step(p, [g], m, v, step, betas=(0.0, 0.0), m_scale=ms, v_scale=vs, seed=seed)
        number = (h & 0xFFFF if name == "m" else h >> 16) << 4
        assert int((number == 1 << 19).sum()) > 0
        up = number >= 1 << 19 if name == "m" else number > 1 << 19
        assert torch.equal(f64(block.adamw_moments(m, v, ms, vs)[name == "v"]), torch.where(up, 9 / 8, 1.0).double()), name


def test_moments_that_no_scale_holds():
    # v = 3.3e38 asks for a scale of 2^128: NaN, as for an infinity, and not an infinity beside NaNs; 3.1e38 has 2^127
    for big, held in ((3.3e38 ** 0.5, False), (3.1e38 ** 0.5, True)):
        p, g = torch.zeros(512, device="cuda"), torch.zeros(512, device="cuda")
        g[3] = big
        m, v = (torch.zeros(512, dtype=torch.uint8, device="cuda") for _ in range(2))
        ms, vs = (torch.zeros(2, device="cuda") for _ in range(2))
        block.adamw_step([p], [g], m, v, 1, betas=(0.9, 0.0), m_scale=ms, v_scale=vs)
        av = block.adamw_moments(m, v, ms, vs)[1]
        assert not av[256:].any()
        if held:
            assert float(vs[0]) == 2.0 ** 127 and abs(float(av[3]) - 3.1e38) <= 2.0 ** 124 and not av[4:].any()
        else:
            assert torch.isnan(vs[0]) and torch.isnan(av[:256]).all()
