"""Host-side checks of the block operators' C ABI (include/pararnn_block.h) and of their plain forms, without a GPU."""
import ctypes
import os
import re
import struct
import subprocess

import pytest
import torch

import block_plain as plain
from nonlinear_rnn_solve_amd import block, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pararnn_block.h")
P = 1 << 20          # an aligned address that is never read
WS, BIG = 1 << 24, 1 << 50

# the structs as the C compiler lays them out
CONV = struct.Struct("@ii4qP2q4Pq")
CONV_GRAD = struct.Struct("@3P4q3P")
SSM = struct.Struct("@i5q3P6q2P6q5Pq")
SSM_GRAD = struct.Struct("@8P14q4P")
TENSOR = struct.Struct("@2P2q2i")
ADAMW = struct.Struct("@i6dq3PQ4P")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(block.LIB_PATH):
        build.build(verbose=False)
    lib = ctypes.CDLL(block.LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    for name, res, args in (
            ("abi_version", i32, []),
            ("conv_workspace_bytes", sz, [i64] * 4),
            ("causal_conv", i32, [vp] * 5),
            ("causal_conv_vjp", i32, [vp, vp, vp, sz, vp]),
            ("ssm_chunks", i64, [i64]),
            ("ssm_workspace_bytes", sz, [i64] * 5 + [i32]),
            ("selective_scan", i32, [vp] * 6 + [sz, vp]),
            ("selective_scan_vjp", i32, [vp, vp, vp, sz, vp]),
            ("gated_linear_workspace_bytes", sz, [i32, i64, i64, i64, i32]),
            ("gated_linear", i32, [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp]),
            ("gated_linear_vjp", i32, [i32, i32, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp, i64, vp, sz, vp]),
            ("adamw", i32, [vp, vp, i64, vp]),
            ("adamw_moments", i32, [i64] + [vp] * 7)):
        fn = getattr(lib, "pararnn_block_" + name)
        fn.restype, fn.argtypes = res, args
    return lib


def test_library_exports_every_declared_function(lib):
    names = set(re.findall(r"^\s*(?:size_t|pararnn_status|int64_t|int)\s+(pararnn_block_\w+)\s*\(", open(HEADER).read(), re.M))
    assert len(names) == 13, names
    out = subprocess.run(["nm", "-D", "--defined-only", block.LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r"\bT (pararnn_\w+)", out)) == names


def test_constants_and_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "layout.c"
    off = lambda s, fields: ["sizeof(pararnn_block_%s)" % s] + ["offsetof(pararnn_block_%s, %s)" % (s, f) for f in fields.split()]  # noqa: E731
    fields = off("conv", "silu B K x sx weight bias state cu_seqlens n_seqs") + off("conv_grad", "d_last d_x sdy sdx d_weight d_state") + \
        off("ssm", "B N G x z sx sz b c sb sc A h0 cu_seqlens n_seqs") + off("ssm_grad", "dy d_x d_c sdy sdb sdc d_A d_h0") + \
        off("adamw_tensor", "grad numel offset grad_dtype") + off("adamw_args", "beta1 lr step lr_ptr step_ptr seed m v_scale") + \
        ["(size_t)PARARNN_BLOCK_" + c for c in ("MAX_TAPS", "MAX_STATES", "SSM_CHUNK", "ADAMW_BLOCK", "ABI_VERSION")]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pararnn_block.h"\nint main(void){%s return 0;}\n'
                   % "".join('printf("%%zu ", (size_t)(%s));' % f for f in fields))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [CONV.size, 4, 8, 32, 40, 48, 64, 72, 80, 88, 96] + [CONV_GRAD.size, 8, 16, 24, 40, 56, 72] + \
        [SSM.size, 8, 32, 40, 48, 64, 72, 104, 120, 128, 136, 160, 184, 208, 216, 224] + [SSM_GRAD.size, 8, 24, 56, 64, 128, 152, 176, 200] + \
        [TENSOR.size, 8, 16, 24, 36] + [ADAMW.size, 8, 40, 56, 64, 80, 88, 96, 120] + \
        [block.MAX_TAPS, block.MAX_STATES, block.SSM_CHUNK, block.ADAMW_BLOCK, block.ABI_VERSION]


def test_binding_is_built_for_the_library(lib):
    b = block.load_library()
    assert (b.ABI_VERSION, b.MAX_TAPS, b.MAX_STATES, b.SSM_CHUNK, b.ADAMW_BLOCK) == \
        (block.ABI_VERSION, block.MAX_TAPS, block.MAX_STATES, block.SSM_CHUNK, block.ADAMW_BLOCK)
    assert lib.pararnn_block_abi_version() == block.ABI_VERSION
    assert build.BLOCK_BINDING == block.BINDING_PATH


def conv(dtype=0, silu=1, B=2, T=300, D=64, K=4, x=P, st=(64, 64), w=P, b=0, s=0, cu=0, n=1):
    return CONV.pack(dtype, silu, B, T, D, K, x, *st, w, b, s, cu, n)


def test_conv_validation(lib):
    sy = struct.pack("@2q", 300 * 64, 64)
    run = lambda p, y=P, last=None: lib.pararnn_block_causal_conv(p, y, sy, last, None)  # noqa: E731
    assert run(None) == -1 and lib.pararnn_block_causal_conv(conv(), P, None, None, None) == -1
    for bad in (dict(dtype=2), dict(silu=2), dict(B=-1), dict(T=-1), dict(D=-1), dict(K=0), dict(K=-3), dict(B=1 << 40, T=1 << 40), dict(x=0),
                dict(x=P + 2), dict(w=0), dict(w=P + 1), dict(b=P + 2), dict(s=P + 2), dict(cu=P + 2), dict(cu=P, n=0), dict(cu=P, T=1 << 31),
                dict(st=(-1, 64)), dict(st=(1 << 61, 64), B=64), dict(st=(64, 1 << 61)), dict(cu=P, n=1 << 58)):
        assert run(conv(**bad)) == -1, bad
    assert run(conv(K=9)) == -2 and run(conv(B=1 << 34, T=8, D=4)) == -2
    assert run(conv(), y=0) == -1 and run(conv(), y=P + 2) == -1 and run(conv(), last=P + 2) == -1
    assert run(conv(B=0)) == 0 and run(conv(D=0)) == 0

    def grad(dy=P, dl=0, dx=P, st=64, dw=P, db=0, ds=0):
        return CONV_GRAD.pack(dy, dl, dx, st, st, st, st, dw, db, ds)

    run = lambda p, g, ws=WS, n=BIG: lib.pararnn_block_causal_conv_vjp(p, g, ws, n, None)  # noqa: E731
    assert run(conv(), None) == -1 and run(conv(silu=3), grad()) == -1
    for bad in (dict(dy=0), dict(dx=0), dict(dy=P + 2), dict(dl=P + 2), dict(dw=P + 1), dict(db=P + 2), dict(ds=P + 2), dict(st=-1), dict(st=1 << 61)):
        assert run(conv(), grad(**bad)) == -1, bad
    assert run(conv(), grad(), ws=None) == -3 and run(conv(), grad(), ws=WS + 8) == -3 and run(conv(), grad(), n=64) == -3
    assert run(conv(K=9), grad()) == -2 and run(conv(D=0), grad()) == 0
    need = lib.pararnn_block_conv_workspace_bytes
    assert need(2, 300, 64, 4) > 0 and need(2, 300, 64, 9) == 0 and need(-1, 300, 64, 4) == 0 and need(1 << 40, 1 << 40, 1, 4) == 0


def ssm(dtype=0, B=2, T=300, D=64, N=16, G=1, x=P, dl=P, z=P, st=64, b=P, c=P, st3=16, A=P, skip=0, bias=0, h0=0, cu=0, n=1):
    return SSM.pack(dtype, B, T, D, N, G, x, dl, z, *([st] * 6), b, c, *([st3] * 6), A, skip, bias, h0, cu, n)


def test_ssm_validation(lib):
    sy = struct.pack("@2q", 300 * 64, 64)
    run = lambda p, y=P, last=None, carry=None, ws=WS, n=BIG: lib.pararnn_block_selective_scan(p, y, sy, last, carry, ws, n, None)  # noqa: E731
    assert run(None) == -1
    for bad in (dict(dtype=2), dict(B=-1), dict(T=-1), dict(D=-1), dict(N=0), dict(G=0), dict(G=3), dict(G=128), dict(B=1 << 40, T=1 << 40), dict(x=0),
                dict(x=P + 2), dict(dl=0), dict(z=P + 2), dict(b=0), dict(c=P + 2), dict(A=0), dict(skip=P + 2), dict(bias=P + 1), dict(h0=P + 2),
                dict(cu=P + 2), dict(cu=P, n=0), dict(cu=P, T=1 << 31), dict(st=-1), dict(st=1 << 61), dict(st3=-1), dict(st3=1 << 61),
                dict(N=1 << 60), dict(cu=P, n=1 << 56)):
        assert run(ssm(**bad)) == -1, bad
    assert run(ssm(N=1 << 40)) == -2 and run(ssm(N=33)) == -2 and run(ssm(T=(1 << 31) - 1, B=1, D=1)) == -2 and run(ssm(B=1 << 31, T=1, D=1)) == -2
    assert run(ssm(), y=0) == -1 and run(ssm(), last=P + 2) == -1 and run(ssm(), carry=P + 1) == -1
    assert run(ssm(), ws=None) == -3 and run(ssm(), ws=WS + 8) == -3 and run(ssm(), n=64) == -3
    assert run(ssm(B=0)) == 0 and run(ssm(D=0)) == 0

    def grad(carry=P, dy=P, dl=0, dx=P, dd=P, dz=P, db=P, dc=P, st=64, st3=16, dA=0, ds=0, dbias=0, dh=0):
        return SSM_GRAD.pack(carry, dy, dl, dx, dd, dz, db, dc, *([st] * 8), *([st3] * 6), dA, ds, dbias, dh)

    run = lambda p, g, ws=WS, n=BIG: lib.pararnn_block_selective_scan_vjp(p, g, ws, n, None)  # noqa: E731
    assert run(ssm(), None) == -1 and run(ssm(dtype=5), grad()) == -1
    for bad in (dict(carry=0), dict(dy=0), dict(dl=P + 2), dict(dx=0), dict(dd=0), dict(dz=0), dict(db=0), dict(dc=P + 2), dict(st=-1), dict(st3=-1),
                dict(dA=P + 2), dict(ds=P + 2), dict(dbias=P + 2), dict(dh=P + 2)):
        assert run(ssm(), grad(**bad)) == -1, bad
    assert run(ssm(z=0), grad(dz=0), n=64) == -3 and run(ssm(), grad(), ws=None) == -3
    assert run(ssm(N=33), grad()) == -2 and run(ssm(D=0), grad()) == 0
    assert [lib.pararnn_block_ssm_chunks(t) for t in (-1, 0, 1, 16, 17)] == [0, 0, 1, 1, 2]
    need = lib.pararnn_block_ssm_workspace_bytes
    assert need(2, 300, 64, 16, 1, 1) > 0 and need(2, 300, 64, 33, 1, 1) == 0 and need(2, 300, 64, 16, 3, 0) == 0 and need(-1, 3, 64, 16, 1, 0) == 0


def test_gated_linear_validation(lib):
    def fwd(dtype=0, act=0, R=4, D=8, F=6, x=P, sx=8, g=P, sg=8, u=P, su=8, h=P, sh=6, pre=None, ws=WS, n=BIG):
        return lib.pararnn_block_gated_linear(dtype, act, R, D, F, x, sx, g, sg, u, su, h, sh, pre, ws, n, None)

    for bad in (dict(dtype=2), dict(act=2), dict(act=-1), dict(R=-1), dict(D=-1), dict(F=-1), dict(x=None), dict(x=P + 2), dict(g=None), dict(u=P + 2),
                dict(h=None), dict(pre=P + 2), dict(sx=-1), dict(sg=-1), dict(su=1 << 61), dict(sh=-1), dict(R=1 << 30, D=1 << 30, F=1 << 30, dtype=7)):
        assert fwd(**bad) == -1, bad
    assert fwd(R=1 << 31) == -2 and fwd(D=1 << 31) == -2 and fwd(F=1 << 31) == -2
    assert fwd(R=0) == 0 and fwd(F=0) == 0

    def bwd(dtype=0, act=0, R=4, D=8, F=6, x=P, g=P, u=P, pre=P, dh=P, dx=P, dg=P, du=P, st=8, ws=WS, n=BIG):
        return lib.pararnn_block_gated_linear_vjp(dtype, act, R, D, F, x, st, g, st, u, st, pre, dh, st, dx, st, dg, st, du, st, ws, n, None)

    for bad in (dict(dtype=2), dict(act=2), dict(R=-1), dict(x=None), dict(g=P + 2), dict(u=None), dict(pre=None), dict(dh=None), dict(dx=P + 2),
                dict(dg=None), dict(du=None), dict(dg=P + 1), dict(st=-1), dict(st=1 << 61)):
        assert bwd(**bad) == -1, bad
    assert bwd(ws=None) == -3 and bwd(ws=WS + 8) == -3 and bwd(n=64) == -3 and bwd(R=1 << 31) == -2
    assert bwd(dx=None, dg=None, du=None) == 0
    need = lib.pararnn_block_gated_linear_workspace_bytes
    assert need(0, 4, 8, 6, 1) > need(1, 4, 8, 6, 1) > 0 and need(2, 4, 8, 6, 1) == 0 and need(0, -1, 8, 6, 1) == 0 and need(0, 1 << 31, 8, 6, 1) == 0


def test_adamw_validation(lib):
    def run(count=1, tensors=True, param=P, grad=P, numel=300, offset=0, pt=0, gt=0, bits=32, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, lr=1e-3, gs=1.0,
            step=1, lrp=0, gsp=0, stepp=0, m=P, v=P, ms=0, vs=0):
        a = ADAMW.pack(bits, b1, b2, eps, wd, lr, gs, step, lrp, gsp, stepp, 0, m, v, ms, vs)
        return lib.pararnn_block_adamw(a, TENSOR.pack(param, grad, numel, offset, pt, gt) if tensors else None, count, None)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(count=-1), dict(tensors=False), dict(param=0), dict(param=P + 2), dict(grad=0), dict(grad=P + 1), dict(numel=-1), dict(offset=-256),
                dict(offset=255), dict(pt=2), dict(gt=-1), dict(bits=16), dict(b1=1.0), dict(b1=-0.1), dict(b2=nan), dict(eps=-1.0), dict(eps=inf),
                dict(wd=nan), dict(lr=inf), dict(gs=nan), dict(step=0), dict(lrp=P + 2), dict(gsp=P + 1), dict(stepp=P + 4), dict(m=0), dict(v=P + 2),
                dict(bits=8), dict(bits=8, ms=P), dict(bits=8, ms=P, vs=P + 2), dict(numel=1 << 61)):
        assert run(**bad) == -1, bad
    assert run(numel=1 << 40) == -2
    assert run(count=0, tensors=False) == 0 and run(numel=0, param=0, grad=0, m=0, v=0) == 0
    assert lib.pararnn_block_adamw(None, None, 0, None) == -1
    mom = lambda n=512, m=P, v=P, ms=P, vs=P, mo=P, vo=P: lib.pararnn_block_adamw_moments(n, m, v, ms, vs, mo, vo, None)  # noqa: E731
    for bad in (dict(n=-256), dict(n=100), dict(m=0), dict(v=0), dict(ms=0), dict(vs=P + 2), dict(mo=0), dict(vo=P + 1)):
        assert mom(**bad) == -1, bad
    assert mom(n=0) == 0 and mom(n=1 << 50) == -2


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        block.causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="GPU tensor"):
        block.selective_scan(x, x, torch.zeros(8, 4), x[..., :4], x[..., :4])
    with pytest.raises(ValueError, match="GPU tensor"):
        block.gated_linear(x, torch.zeros(3, 8), torch.zeros(3, 8))
    with pytest.raises(ValueError, match="GPU tensor"):
        block.adamw_step([x], [x], torch.zeros(256), torch.zeros(256), 1)
    assert block.adamw_state_size([torch.zeros(1), torch.zeros(0), torch.zeros(257, 2)]) == 256 + 3 * 256


def test_plain_forms_against_torch_and_differences():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64).requires_grad_()  # noqa: E731
    x, w, b = r(2, 9, 3), r(3, 4), r(3)
    y, last = plain.conv(x, w, b, act=False)
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (3, 0)), w[:, None], b, groups=3).transpose(1, 2)
    assert torch.allclose(y, want) and torch.equal(last[:, 0], x[:, -3:])
    assert torch.allclose(plain.silu(x), torch.nn.functional.silu(x)) and torch.allclose(plain.gelu(x), torch.nn.functional.gelu(x, approximate="tanh"))
    cu = [0, 2, 2, 7, 9]
    assert torch.autograd.gradcheck(lambda *t: plain.conv(*t, cu=cu), (x, w, b, r(2, 4, 3, 3)))
    args = (r(2, 9, 4), r(2, 9, 4), r(4, 2), r(2, 9, 2, 2), r(2, 9, 2, 2), r(4), r(2, 9, 4), r(4), r(2, 4, 4, 2))
    assert torch.autograd.gradcheck(lambda *t: plain.ssm(*t, cu=cu), args)
    # a scan of one state whose step is s is the recurrence h = exp(s A) h + s x b
    one = torch.ones(1, 5, 1, dtype=torch.float64)
    y, _ = plain.ssm(one, one * 0, torch.tensor([[-2.0]], dtype=torch.float64), one, one)
    s = torch.log(torch.tensor(2.0, dtype=torch.float64))
    assert torch.allclose(y[0, :, 0], torch.stack([s * (torch.exp(-2 * s) ** torch.arange(k + 1)).sum() for k in range(5)]))
    assert plain.values(15)[127] == 1.875 and plain.values(31)[255] == 1.875 and plain.values(15)[129] == -2.0 ** -17 and plain.values(31)[1] == 2.0 ** -33


def test_ssm_steps_too_far_apart(lib):
    # 2^24 elements between two steps; between one and none nothing is (without a GPU the launch itself then fails)
    sy = struct.pack("@2q", 1 << 26, 1 << 24)
    run = lambda p: lib.pararnn_block_selective_scan(p, P, sy, None, None, WS, BIG, None)  # noqa: E731
    assert run(ssm(B=1, T=2)) == -2 and run(ssm(B=1, T=300, st=1 << 24)) == -2
    if not torch.cuda.is_available():
        assert run(ssm(B=1, T=1)) == run(ssm(B=1, T=1, st=1 << 24, st3=1 << 25)) == -4


def test_gated_linear_launch_limit(lib):
    # 4096 by 3000 large tiles are 2^32.55 threads in workgroups of 512; 4096 by 2000 are 2^31.97 (without a GPU their launch then fails)
    run = lambda F: lib.pararnn_block_gated_linear(1, 0, 1 << 20, 64, F, P, 64, P, 64, P, 64, P, F, None, None, 0, None)  # noqa: E731
    assert run(128 * 3000) == -2
    if not torch.cuda.is_available():
        assert run(128 * 2000) == -4
