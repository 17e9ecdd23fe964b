"""The block operators together, as examples/selective_lm.py runs them: a packed training step against the same model in plain
64-bit torch, the optimizer's step on its gradients, generation against scoring the whole sequence, and packed documents against
each by itself."""
import os
import sys

import pytest
import torch

import block_plain
import lm_plain as plain
from lm_plain import f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import selective_lm  # noqa: E402

pytestmark = pytest.mark.gpu


def plain_loss(p, tokens, targets, cu, blocks, rank):
    stream = p["embed"][tokens]
    out = torch.zeros_like(stream)
    for k in range(blocks):
        q = {n.split(".", 2)[2]: t for n, t in p.items() if n.startswith("layers.%d." % k)}
        y, stream = plain.norm(out, q["norm1"], q["bias1"], residual=stream)
        x, z = (y @ q["into"].t()).chunk(2, -1)
        x, _ = block_plain.conv(x, q["taps"], q["taps_bias"], cu=cu)
        low = x @ q["low"].t()
        n = q["log_A"].shape[1]
        y, _ = block_plain.ssm(x, low[..., :rank] @ q["steps"].t(), -torch.exp(q["log_A"]), low[..., rank:rank + n], low[..., rank + n:],
                               skip=q["skip"], z=z, dt_bias=q["dt_bias"], cu=cu)
        y, stream = plain.norm(y @ q["back"].t(), q["norm2"], q["bias2"], residual=stream)
        out = block_plain.gated(y, q["gate"], q["up"]) @ q["down"].t()
    y, _ = plain.norm(out, p["norm"], p["bias"], residual=stream)
    logp, _, _ = plain.logp(y @ p["embed"].t(), targets)
    return -logp.sum() / (targets >= 0).sum()


def test_training_step_against_the_plain_model():
    # float32: every operator is within ~1e-5 of its terms' sizes, and the model is two dozen of them deep
    vocab, blocks, rank = 37, 2, 3
    model = selective_lm.SelectiveLM(vocab, 24, blocks, states=5, rank=rank, dtype=torch.float32, seed=3)
    tokens, targets, cu = selective_lm.documents(vocab, 3, 90, 4, torch.Generator().manual_seed(5))
    loss = model.loss(tokens, targets, cu)
    loss.backward()
    params = {n: f64(t).requires_grad_() for n, t in model.named_parameters()}
    want = plain_loss(params, tokens.cpu(), targets.cpu(), cu.tolist(), blocks, rank)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 1e-5 * abs(float(want.detach()))
    for n, t in model.named_parameters():
        a, b = f64(t.grad), params[n].grad
        assert float((a - b).norm()) <= 2e-4 * float(b.norm()) + 1e-9, n
    # the step on these gradients
    old, grads = {n: f64(t) for n, t in model.named_parameters()}, {n: f64(t.grad) for n, t in model.named_parameters()}
    opt = selective_lm.AdamW(model.parameters(), lr=1e-3, betas=(0.9, 0.95), weight_decay=0.1)
    opt.step()
    for n, t in model.named_parameters():
        z = torch.zeros_like(old[n])
        want, _, _ = block_plain.adamw(old[n], grads[n], z, z, 1, 1e-3, (0.9, 0.95), 1e-8, 0.1)
        assert float((f64(t) - want).abs().max()) <= 16 * plain.U32 * float(old[n].abs().max() + 1e-3), n


def test_generation_follows_the_whole_sequence():
    model = selective_lm.SelectiveLM(50, 64, 2, dtype=torch.float32, seed=4)
    prompt = torch.randint(0, 50, (3, 19), generator=torch.Generator().manual_seed(6)).cuda()
    got = model.generate(prompt, 7)
    with torch.no_grad():
        logits, _ = model(torch.cat([prompt, got], 1))
    for n in range(7):     # each token is the most probable one after all before it (up to rounding at a tie)
        row = logits[:, 18 + n]
        assert torch.all(row.gather(1, got[:, n:n + 1])[:, 0] >= row.amax(1) - 1e-4)


@pytest.mark.parametrize("bits", [8, 32])
def test_a_short_training_run(bits):
    model = selective_lm.SelectiveLM(29, 64, 2, seed=5)
    losses = selective_lm.train(model, 5, 29, rows=4, total=128, count=3, bits=bits)
    assert losses.shape == (5,) and torch.isfinite(losses).all()
    assert all(torch.isfinite(p).all() for p in model.parameters())


def test_packed_documents_do_not_meet():
    # the states that a document leaves and its logits are those of the document alone
    model = selective_lm.SelectiveLM(31, 32, 2, dtype=torch.float32, seed=6)
    tokens, _, cu = selective_lm.documents(31, 2, 100, 3, torch.Generator().manual_seed(8))
    with torch.no_grad():
        logits, states = model(tokens, cu)
        for j, (a, b) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
            alone, last = model(tokens[:, a:b])
            assert float((logits[:, a:b] - alone).abs().max()) <= 1e-4
            for (c, h), (c1, h1) in zip(states, last):
                assert float((c[:, j] - c1).abs().max()) <= 1e-4 and float((h[:, j] - h1).abs().max()) <= 1e-4


def test_second_derivatives_are_refused():
    # the gradients' operators have none: a gradient of a gradient must not come out without their part
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g).cuda().requires_grad_()  # noqa: E731
    x, low, w = r(2, 5, 8), r(2, 5, 3 + 2 * 4), r(8, 4)
    calls = {
        "conv": (selective_lm.CausalConv.apply(x, w, r(8), None, None), x),
        "scan": (selective_lm.SelectiveScan.apply(x, r(2, 5, 8), -w.exp(), low, 3, r(8), r(2, 5, 8), r(8), None, None), x),
        "product": (selective_lm.GatedLinear.apply(x, r(16, 8), r(16, 8)), x),
        "norm": (selective_lm.LayerNorm.apply(x, r(2, 5, 8), r(8), r(8)), x),
        "logprobs": (selective_lm.TokenLogprobs.apply(low, torch.zeros(2, 5, dtype=torch.int64, device="cuda")), low),
    }
    for name, (out, leaf) in calls.items():
        loss = sum(t.square().sum() for t in (out if isinstance(out, tuple) else (out,)))
        (first,) = torch.autograd.grad(loss, leaf, create_graph=True)
        assert torch.isfinite(first).all(), name
        with pytest.raises(RuntimeError, match="once_differentiable"):
            first.sum().backward()
