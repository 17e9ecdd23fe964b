"""Host-side checks of the language-model operators' C ABI (include/pararnn_lm.h) and of their plain forms, without a GPU."""
import ctypes
import os
import re
import shutil
import subprocess
import sys
import sysconfig

import pytest
import torch

import lm_abi
import lm_plain as plain
from nonlinear_rnn_solve_amd import build, lm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pararnn_lm.h")
P = 1 << 20          # an aligned address that is never read
WS, BIG = 1 << 24, 1 << 50


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(lm.LIB_PATH):
        build.build(verbose=False)
    return lm_abi.load(lm.LIB_PATH)


def declared():
    txt = open(HEADER).read()
    return set(re.findall(r"^\s*(?:size_t|pararnn_status|int64_t|int)\s+(pararnn_lm_\w+)\s*\(", txt, re.M))


def test_library_exports_every_declared_function(lib):
    names = declared()
    assert len(names) == 11, names
    out = subprocess.run(["nm", "-D", "--defined-only", lm.LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r"\bT (pararnn_\w+)", out)) == names
    for n in names:
        assert hasattr(lib, n), n


def test_constants_and_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "layout.c"
    fields = ["sizeof(pararnn_lm_scan)"] + ["offsetof(pararnn_lm_scan, %s)" % f for f in
                                            "c B x sx lam h0 cu_seqlens n_seqs".split()] + \
        ["sizeof(pararnn_lm_scan_grad)"] + ["offsetof(pararnn_lm_scan_grad, %s)" % f for f in
                                            "dh d_last d_x sdh sdx sdi d_lam d_h0".split()] + \
        ["(size_t)PARARNN_LM_SCAN_CHUNK", "(size_t)PARARNN_LM_NORM_MAX_D", "(size_t)PARARNN_LM_MAX_TOP",
         "(size_t)PARARNN_LM_ABI_VERSION"]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pararnn_lm.h"\nint main(void){%s return 0;}\n'
                   % "".join('printf("%%zu ", %s);' % f for f in fields))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [lm_abi.SCAN.size, 4, 8, 32, 56, 104, 112, 120, 128, lm_abi.SCAN_GRAD.size, 8, 16, 24, 48, 64, 96, 112, 120,
                   lm.SCAN_CHUNK, lm.NORM_MAX_D, lm.MAX_TOP, lm.ABI_VERSION]


def scan_problem(dtype=0, c=8.0, B=2, T=300, D=64, x=P, r=P, i=P, st=(64, 64), lam=P, h0=0, cu=0, n=1):
    return lm_abi.SCAN.pack(dtype, c, B, T, D, x, r, i, *(st * 3), lam, h0, cu, n)


def test_scan_validation(lib):
    sh = lm_abi.PAIR.pack(300 * 64, 64)
    run = lambda prob, h=P, last=None, carry=None, ws=WS, n=BIG: lib.pararnn_lm_gated_scan(  # noqa: E731
        prob, h, sh, last, carry, ws, n, None)
    assert run(None) == -1
    for bad in (dict(dtype=2), dict(dtype=-1), dict(c=0.0), dict(c=-3.0), dict(c=float("inf")), dict(c=float("nan")), dict(B=-1),
                dict(T=-1), dict(D=-5), dict(B=1 << 40, T=1 << 40), dict(x=0), dict(r=0), dict(i=0), dict(x=P + 2), dict(lam=0),
                dict(lam=P + 1), dict(h0=P + 2), dict(cu=P + 2), dict(cu=P, n=0), dict(cu=P, n=-1), dict(cu=P, T=1 << 31),
                dict(st=(-1, 64)), dict(st=(1 << 62, 64), B=64), dict(st=(64, 1 << 61))):
        assert run(scan_problem(**bad)) == -1, bad
    assert run(scan_problem(dtype=1, x=P + 2, r=P + 2, i=P + 2, B=1 << 31, D=1)) == -2    # element alignment is enough
    assert run(scan_problem(B=1 << 31, T=1)) == -2
    assert run(scan_problem(), h=0) == -1
    assert run(scan_problem(), h=P + 1) == -1
    assert run(scan_problem(), last=P + 2) == -1
    assert run(scan_problem(), carry=P + 2) == -1
    assert run(scan_problem(), ws=None) == -3
    assert run(scan_problem(), ws=WS + 8) == -3
    assert run(scan_problem(), n=16) == -3
    assert run(scan_problem(B=0)) == 0 and run(scan_problem(D=0)) == 0
    assert lib.pararnn_lm_gated_scan(scan_problem(), P, None, None, None, WS, BIG, None) == -1
    assert lib.pararnn_lm_scan_workspace_bytes(2, 300, 64) > 0
    assert lib.pararnn_lm_scan_workspace_bytes(-1, 300, 64) == 0
    assert [lib.pararnn_lm_scan_chunks(t) for t in (0, 1, lm.SCAN_CHUNK, lm.SCAN_CHUNK + 1)] == [0, 1, 1, 2]


def test_scan_gradient_validation(lib):
    def grad(carry=P, dh=P, dl=0, dx=P, dr=P, di=P, st=64, dlam=0, dh0=0):
        return lm_abi.SCAN_GRAD.pack(carry, dh, dl, dx, dr, di, *([st] * 8), dlam, dh0)

    run = lambda prob, g, ws=WS, n=BIG: lib.pararnn_lm_gated_scan_vjp(prob, g, ws, n, None)  # noqa: E731
    assert run(scan_problem(), None) == -1
    assert run(scan_problem(c=0.0), grad()) == -1
    for bad in (dict(carry=0), dict(dh=0), dict(dx=0), dict(dr=0), dict(di=0), dict(dh=P + 2), dict(dl=P + 2), dict(dlam=P + 2),
                dict(dh0=P + 1), dict(st=-1), dict(st=1 << 61)):
        assert run(scan_problem(), grad(**bad)) == -1, bad
    assert run(scan_problem(B=0, lam=0), grad(dlam=P)) == -1      # d_lam needs lam, rows or not
    assert run(scan_problem(), grad(), n=16) == -3
    assert run(scan_problem(), grad(), ws=None) == -3


def test_norm_validation(lib):
    def fwd(dtype=0, N=4, D=64, x=P, xs=64, res=None, rs=64, w=P, b=None, eps=1e-5, y=P, ys=64, s=None, ss=64, stats=None):
        return lib.pararnn_lm_layer_norm(dtype, N, D, x, xs, res, rs, w, b, eps, y, ys, s, ss, stats, None)

    for bad in (dict(dtype=3), dict(N=-1), dict(D=-1), dict(x=None), dict(x=P + 2), dict(w=None), dict(y=None), dict(eps=-1.0),
                dict(eps=float("nan")), dict(res=P), dict(s=P), dict(res=P + 2, s=P), dict(xs=-1), dict(ys=-1), dict(b=P + 1),
                dict(res=P, s=P, rs=-1), dict(res=P, s=P, ss=-1), dict(stats=P + 2), dict(N=1 << 40, D=1 << 40), dict(xs=1 << 61)):
        assert fwd(**bad) == -1, bad
    assert fwd(D=lm.NORM_MAX_D + 1) == -2
    assert fwd(N=1 << 31, D=1, xs=1, ys=1) == -2 and fwd(N=1 << 22, D=5000) == -2
    assert fwd(N=0) == 0 and fwd(D=0) == 0

    def bwd(dtype=0, N=4, D=64, dy=P, s=P, w=P, stats=P, ds=None, dx=P, st=64, dw=None, db=None, ws=WS, n=BIG):
        return lib.pararnn_lm_layer_norm_vjp(dtype, N, D, dy, st, s, st, w, stats, ds, st, dx, st, dw, db, ws, n, None)

    for bad in (dict(dtype=3), dict(N=-1), dict(dy=None), dict(s=None), dict(w=None), dict(stats=None), dict(dx=None), dict(ds=P + 2),
                dict(dx=P + 1), dict(st=-1), dict(dw=P + 2), dict(db=P + 2)):
        assert bwd(**bad) == -1, bad
    assert bwd(D=lm.NORM_MAX_D + 1) == -2
    assert bwd(n=16) == -3 and bwd(ws=None) == -3 and bwd(ws=WS + 4) == -3
    assert bwd(D=0) == 0
    assert lib.pararnn_lm_layer_norm_vjp_workspace_bytes(4, -1) == 0


def test_logprobs_validation(lib):
    def fwd(dtype=0, N=4, V=100, z=P, st=100, t=P, tb=8, lse=P, lp=P, ent=P, top=0, tl=None, ti=None, ws=WS, n=BIG):
        return lib.pararnn_lm_token_logprobs(dtype, N, V, z, st, t, tb, lse, lp, ent, top, tl, ti, ws, n, None)

    for bad in (dict(dtype=2), dict(N=-1), dict(V=-1), dict(V=1 << 31, N=1), dict(z=None), dict(z=P + 2), dict(st=-1), dict(tb=2),
                dict(t=P + 4), dict(lp=None), dict(t=None), dict(lse=P + 2), dict(ent=P + 1), dict(top=-1), dict(top=33, tl=P, ti=P),
                dict(top=5, V=4, tl=P, ti=P), dict(top=3, tl=P), dict(top=3, ti=P), dict(top=3, tl=P, ti=P + 4), dict(st=1 << 61)):
        assert fwd(**bad) == -1, bad
    assert fwd(n=16) == -3 and fwd(ws=None) == -3 and fwd(ws=WS + 16) == -3
    assert fwd(N=1 << 26, V=5, st=5) == -2 and fwd(N=1 << 22, V=40000) == -2
    assert fwd(N=0) == 0
    assert lib.pararnn_lm_token_logprobs_workspace_bytes(4, 100, 33) == 0
    assert lib.pararnn_lm_token_logprobs_workspace_bytes(4, 100, 32) > 0

    def bwd(dtype=0, N=4, V=100, z=P, st=100, t=P, tb=4, lse=P, ent=P, g=P, ge=P, d=P, ds=100):
        return lib.pararnn_lm_token_logprobs_vjp(dtype, N, V, z, st, t, tb, lse, ent, g, ge, d, ds, None)

    for bad in (dict(dtype=2), dict(N=-1), dict(z=None), dict(lse=None), dict(g=None), dict(ent=None), dict(d=None), dict(d=P + 2),
                dict(ds=-1), dict(ge=P + 2), dict(t=P + 2), dict(tb=3)):
        assert bwd(**bad) == -1, bad
    assert bwd(N=0) == 0 and bwd(V=0) == 0


def test_binding_is_built_for_the_library(lib):
    b = lm.load_library()
    assert (b.ABI_VERSION, b.SCAN_CHUNK, b.NORM_MAX_D, b.MAX_TOP) == (lm.ABI_VERSION, lm.SCAN_CHUNK, lm.NORM_MAX_D, lm.MAX_TOP)
    assert lib.pararnn_lm_abi_version() == lm.ABI_VERSION


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        lm.gated_scan(x, x, x, torch.zeros(8))
    with pytest.raises(ValueError, match="GPU tensor"):
        lm.layer_norm(x, torch.zeros(8))
    with pytest.raises(ValueError, match="GPU tensor"):
        lm.token_logprobs(x, torch.zeros(2, 4, dtype=torch.int64))


def test_plain_scan_is_the_recurrence_and_differentiates():
    g = torch.Generator().manual_seed(1)
    leaves = [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_() for s in ((2, 9, 3),) * 3 + ((3,), (2, 4, 3))]
    cu = [0, 2, 2, 7, 9]
    x, r, i, lam, h0 = (t.detach() for t in leaves)
    h, last = plain.scan(x, r, i, lam, h0, cu=cu)
    a = torch.exp(-8 * torch.log1p(torch.exp(lam)) / (1 + torch.exp(-r)))
    state = h0[:, 0]
    for t in range(9):
        if t in (2, 7):
            state = h0[:, {2: 2, 7: 3}[t]]
        state = a[:, t] * state + torch.sqrt(1 - a[:, t] ** 2) * x[:, t] / (1 + torch.exp(-i[:, t]))
        assert torch.allclose(h[:, t], state, atol=1e-12)
    assert torch.allclose(last[:, 1], h0[:, 1]) and torch.allclose(last[:, 3], state)
    assert torch.autograd.gradcheck(lambda *t: plain.scan(*t, cu=cu), leaves)


def test_plain_norm_and_logprobs_against_torch():
    g = torch.Generator().manual_seed(2)
    x, w, b = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 33), (33,), (33,)))
    assert torch.allclose(plain.norm(x, w, b)[0], torch.nn.functional.layer_norm(x, (33,), w, b), atol=1e-12)
    t = torch.tensor([0, 32, -1, 5, 7])
    lp, ent, lse = plain.logp(x, t)
    d = torch.distributions.Categorical(logits=x)
    assert torch.allclose(ent, d.entropy()) and lp[2] == 0
    assert torch.allclose(lp[t >= 0], d.log_prob(t.clamp(min=0))[t >= 0])
    assert plain.top(torch.tensor([[1.0, float("nan"), 3.0, 1.0, -float("inf")]]), 5).tolist() == [[2, 0, 3, 1, 4]]


class _Finished:
    returncode = 0

    def communicate(self):
        return "", None


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_the_libraries_build_without_torch_or_a_host_compiler(missing, monkeypatch, capsys):
    # the C ABI needs hipcc only; what the Python binding needs is looked for before anything is started
    commands = []
    monkeypatch.setattr(build, "_start", lambda cmd, *a, **k: commands.append(cmd) or _Finished())
    for name in ("replace", "remove"):
        monkeypatch.setattr(build.os, name, lambda *a: None)
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr(shutil, "which", lambda *a, **k: None)
    assert build.build(verbose=False) == build.LIB
    made = [c[c.index("-o") + 1] for c in commands]
    for lib in (build.LIB, build.STRESS_LIB, build.LM_LIB, build.LM_STRESS_LIB):
        assert any(m.startswith(lib) for m in made), lib
    assert not any("lm_binding" in " ".join(c) for c in commands)
    assert missing in capsys.readouterr().out


def test_the_binding_is_of_this_interpreter():
    assert build.LM_BINDING == lm.BINDING_PATH and build.LM_BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_launch_limits_count_whole_workgroups(lib):
    # a launch has fewer than 2^32 threads, the last workgroup's idle rows included: one row more than its limit
    def fwd(N, D):
        return lib.pararnn_lm_layer_norm(0, N, D, P, D, None, 0, P, None, 1e-5, P, D, None, 0, None, None)

    for D, rows in ((1, 16), (256, 16), (257, 4), (1024, 4)):
        limit = rows * ((1 << 24) - 1)
        for N in (limit + 1, limit + rows):
            assert fwd(N, D) == -2, (N, D)
