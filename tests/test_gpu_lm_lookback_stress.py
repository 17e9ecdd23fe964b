"""The gated recurrence under its look-back stress build: the same source, but tiles pause for pseudo-random times before they
publish words, so that words come in orders that the plain build rarely or never sees.  What is composed with what is
fixed, so the results must be the plain library's, bit for bit."""
import pytest
import torch

import lm_abi
from nonlinear_rnn_solve_amd import build, lm

pytestmark = pytest.mark.gpu


def scan(lib, x, r, i, lam, h0, cu, dh, d_last):
    B, T, D = x.shape
    n = 1 if cu is None else cu.numel() - 1
    st = x.stride()
    p = lm_abi.SCAN.pack(1, 8.0, B, T, D, x.data_ptr(), r.data_ptr(), i.data_ptr(), *([st[0], st[1]] * 3), lam.data_ptr(),
                         h0.data_ptr(), 0 if cu is None else cu.data_ptr(), n)
    h = torch.empty_like(x)
    last, carry = torch.empty_like(h0), torch.empty(B, lib.pararnn_lm_scan_chunks(T), D, device="cuda")
    ws = torch.empty(lib.pararnn_lm_scan_workspace_bytes(B, T, D), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.pararnn_lm_gated_scan(p, h.data_ptr(), lm_abi.PAIR.pack(st[0], st[1]), last.data_ptr(), carry.data_ptr(),
                                     ws.data_ptr(), ws.numel(), stream) == 0
    d = [torch.empty_like(x) for _ in range(3)]
    d_lam, d_h0 = torch.empty_like(lam), torch.empty_like(h0)
    g = lm_abi.SCAN_GRAD.pack(carry.data_ptr(), dh.data_ptr(), d_last.data_ptr(), *(t.data_ptr() for t in d),
                              *([st[0], st[1]] * 4), d_lam.data_ptr(), d_h0.data_ptr())
    assert lib.pararnn_lm_gated_scan_vjp(p, g, ws.data_ptr(), ws.numel(), stream) == 0
    torch.cuda.synchronize()
    return [h, last, carry, *d, d_lam, d_h0]


@pytest.mark.parametrize("B,T,D,n", [(1, 8192, 192, 0), (3, 1500, 100, 0), (1, 4000, 129, 6), (2, 600, 1030, 0)])
def test_stress_build_gives_the_same_bits(B, T, D, n):
    print("[stress]", B, T, D, n, flush=True)
    g = torch.Generator(device="cuda").manual_seed(T + D)
    x, r, i, dh = (torch.randn(B, T, D, generator=g, device="cuda").bfloat16() for _ in range(4))
    lam = torch.randn(D, generator=g, device="cuda") - 8
    h0, d_last = (torch.randn(B, max(n, 1), D, generator=g, device="cuda") for _ in range(2))
    cu = None
    if n:
        cuts = torch.randint(0, T, (n - 1,), generator=g, device="cuda").sort().values
        cu = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).int()
    plain = scan(lm_abi.load(lm.LIB_PATH), x, r, i, lam, h0, cu, dh, d_last)
    stress = lm_abi.load(build.LM_STRESS_LIB)
    for _ in range(3):
        for a, b in zip(plain, scan(stress, x, r, i, lam, h0, cu, dh, d_last)):
            assert torch.equal(a, b)
