"""The three language-model operators together, as examples/gated_lm.py runs them: a packed training step against the same
model in plain 64-bit torch, generation against scoring the whole sequence, and a short training run."""
import os
import sys

import pytest
import torch

import lm_plain as plain
from lm_plain import f64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gated_lm  # noqa: E402

pytestmark = pytest.mark.gpu


def plain_loss(params, tokens, targets, cu, blocks, entropy_weight):
    stream = params["embed"][tokens]
    out = torch.zeros_like(stream)
    for k in range(blocks):
        y, stream = plain.norm(out, params["weight.%d" % k], params["bias.%d" % k], residual=stream)
        x, r, i = (y @ params["into.%d" % k].t()).chunk(3, -1)
        h, _ = plain.scan(x, r, i, params["lam.%d" % k], cu=cu)
        out = h @ params["back.%d" % k].t()
    y, _ = plain.norm(out, params["weight.%d" % blocks], params["bias.%d" % blocks], residual=stream)
    logp, ent, _ = plain.logp(y @ params["embed"].t(), targets)
    return -(logp.sum() + entropy_weight * ent.sum()) / (targets >= 0).sum()


def test_training_step_against_the_plain_model():
    # float32: every operator is within ~1e-5 of its terms' sizes, and the model is a dozen of them deep
    vocab, blocks = 37, 2
    model = gated_lm.GatedLM(vocab, 24, blocks, dtype=torch.float32, seed=3)
    tokens, targets, cu = gated_lm.documents(vocab, 3, 90, 4, torch.Generator().manual_seed(5))
    loss = model.loss(tokens, targets, cu, entropy_weight=0.01)
    loss.backward()
    params = {n: f64(p).requires_grad_() for n, p in model.named_parameters()}
    want = plain_loss(params, tokens.cpu(), targets.cpu(), cu.tolist(), blocks, 0.01)
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 1e-5 * abs(float(want.detach()))
    for n, p in model.named_parameters():
        a, b = f64(p.grad), params[n].grad
        assert float((a - b).norm()) <= 1e-4 * float(b.norm()) + 1e-9, n


def test_generation_follows_the_whole_sequence():
    model = gated_lm.GatedLM(50, 64, 2, dtype=torch.float32, seed=4)
    prompt = torch.randint(0, 50, (3, 19), generator=torch.Generator().manual_seed(6)).cuda()
    got = model.generate(prompt, 7)
    with torch.no_grad():
        logits, _ = model(torch.cat([prompt, got], 1))
    for n in range(7):     # greedy: each token is the most probable one after all before it (up to rounding at a tie)
        row = logits[:, 18 + n]
        best = row.amax(1)
        assert torch.all(row.gather(1, got[:, n:n + 1])[:, 0] >= best - 1e-4)


def test_a_short_training_run_learns():
    model = gated_lm.GatedLM(29, 64, 2, seed=5)
    losses = gated_lm.train(model, 60, 29, rows=4, total=128, count=3)
    assert torch.isfinite(losses).all()
    assert float(losses[-5:].mean()) < 0.6 * float(losses[:5].mean())


def test_a_second_backward_pass_is_refused():
    # the logits' gradient has taken the logits' place: a second pass over the graph has nothing to start from
    model = gated_lm.GatedLM(29, 16, 1, dtype=torch.float32, seed=6)
    tokens, targets, cu = gated_lm.documents(29, 2, 40, 2, torch.Generator().manual_seed(7))
    loss = model.loss(tokens, targets, cu)
    loss.backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
