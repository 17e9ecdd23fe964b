"""A small recurrent language model on the operators of nonlinear_rnn_solve_amd.lm: packed training and generation.

    python examples/gated_lm.py --steps 200

Each block normalises the residual stream (layer_norm with its residual sum), projects it to the three planes of the
gated recurrence (gated_scan, packed documents in one row) and projects the states back; the head scores the next token
(token_logprobs).  Training follows the gradients of all three through torch's autograd; generation carries the float32
states of the recurrence from token to token and samples among the most probable tokens.  The matrix products are
torch's.  The documents are synthetic: arithmetic sequences modulo the vocabulary, so a trained model can continue one.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nonlinear_rnn_solve_amd import lm  # noqa: E402


class GatedScan(torch.autograd.Function):
    """(h, h_last) of lm.gated_scan; proj holds x, r and i side by side, and so does its gradient."""

    @staticmethod
    def forward(ctx, proj, lam, h0, cu):
        x, r, i = proj.chunk(3, -1)
        h, h_last, carry = lm.gated_scan(x, r, i, lam, h0=h0, cu_seqlens=cu, want_carry=True)
        ctx.save_for_backward(proj, lam, h0, cu, carry)
        return h, h_last

    @staticmethod
    def backward(ctx, dh, d_last):
        proj, lam, h0, cu, carry = ctx.saved_tensors
        d_proj = torch.empty_like(proj)
        g = lm.gated_scan_vjp(*proj.chunk(3, -1), lam, carry, dh.contiguous(), h0=h0, d_last=d_last.contiguous(),
                              cu_seqlens=cu, out=d_proj.chunk(3, -1), want_h0=h0 is not None)
        return d_proj, g["d_lam"], g.get("d_h0"), None


class LayerNorm(torch.autograd.Function):
    """(y, s) of lm.layer_norm for s = x + residual."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias):
        y, s, stats = lm.layer_norm(x, weight, bias, residual=residual, want_stats=True)
        ctx.save_for_backward(s, weight, stats)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, weight, stats = ctx.saved_tensors
        g = lm.layer_norm_vjp(dy.contiguous(), s, weight, stats, d_sum=ds.contiguous())
        return g["d_x"], g["d_x"], g["d_weight"], g["d_bias"]


class TokenLogprobs(torch.autograd.Function):
    """(logp, entropy) of lm.token_logprobs; the gradient overwrites the logits (a second backward pass raises)."""

    @staticmethod
    def forward(ctx, logits, targets):
        t = lm.token_logprobs(logits, targets)
        ctx.save_for_backward(logits, targets, t.lse, t.entropy)
        return t.logp, t.entropy

    @staticmethod
    def backward(ctx, g, ge):
        logits, targets, lse, entropy = ctx.saved_tensors
        return lm.token_logprobs_vjp(logits, targets, lse, entropy, g.contiguous(), ge.contiguous(), out=logits.detach()), None


class GatedLM(torch.nn.Module):
    def __init__(self, vocab, width, blocks, dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def matrix(rows, cols):
            return torch.nn.Parameter((torch.randn(rows, cols, generator=g) / cols ** 0.5).to(device))

        self.dtype, self.width, self.blocks = dtype, width, blocks
        self.embed = matrix(vocab, width)
        self.into = torch.nn.ParameterList(matrix(3 * width, width) for _ in range(blocks))
        self.back = torch.nn.ParameterList(matrix(width, width) for _ in range(blocks))
        # decays between 0.9 and 0.999 at an open gate
        a = torch.rand(blocks, width, generator=g, dtype=torch.float64) * 0.099 + 0.9
        lam = torch.log(torch.expm1(-torch.log(a) / 8)).float().to(device)
        self.lam = torch.nn.ParameterList(torch.nn.Parameter(v.clone()) for v in lam)
        self.weight = torch.nn.ParameterList(torch.nn.Parameter(torch.ones(width, device=device)) for _ in range(blocks + 1))
        self.bias = torch.nn.ParameterList(torch.nn.Parameter(torch.zeros(width, device=device)) for _ in range(blocks + 1))

    def forward(self, tokens, cu=None, states=None):
        """Logits [B, T, V] of the tokens that follow `tokens` [B, T], and the blocks' states."""
        stream = self.embed[tokens].to(self.dtype)
        out, last = torch.zeros_like(stream), []
        for k in range(self.blocks):
            y, stream = LayerNorm.apply(out, stream, self.weight[k], self.bias[k])
            proj = y @ self.into[k].to(self.dtype).t()
            h, h_last = GatedScan.apply(proj, self.lam[k], None if states is None else states[k], cu)
            last.append(h_last)
            out = h @ self.back[k].to(self.dtype).t()
        y, _ = LayerNorm.apply(out, stream, self.weight[-1], self.bias[-1])
        return y @ self.embed.to(self.dtype).t(), last

    def loss(self, tokens, targets, cu=None, entropy_weight=0.0):
        logits, _ = self(tokens, cu)
        logp, entropy = TokenLogprobs.apply(logits, targets)
        return -(logp.sum() + entropy_weight * entropy.sum()) / (targets >= 0).sum().clamp(min=1)

    @torch.no_grad()
    def generate(self, prompt, count, top=1, generator=None):
        """`count` tokens after prompt [B, T], each sampled among the `top` most probable ones; the prompt in one call,
        then token by token with the states updated in place."""
        logits, states = self(prompt)
        got = []
        for _ in range(count):
            t = lm.token_logprobs(logits[:, -1], top=top)
            pick = torch.multinomial(t.top_logp.exp(), 1, generator=generator)
            token = t.top_ids.gather(1, pick)
            got.append(token)
            stream = self.embed[token].to(self.dtype)
            out = torch.zeros_like(stream)
            for k in range(self.blocks):
                y, stream, _ = lm.layer_norm(out, self.weight[k], self.bias[k], residual=stream, sum_out=stream)
                x, r, i = (y @ self.into[k].to(self.dtype).t()).chunk(3, -1)
                h, _, _ = lm.gated_scan(x, r, i, self.lam[k], h0=states[k], h_last=states[k])
                out = h @ self.back[k].to(self.dtype).t()
            y, _, _ = lm.layer_norm(out, self.weight[-1], self.bias[-1], residual=stream, sum_out=stream)
            logits = y @ self.embed.to(self.dtype).t()
        return torch.cat(got, 1)


def documents(vocab, rows, total, count, generator):
    """`rows` rows of `count` packed documents each (the same cuts in every row): tokens, targets (the last token of a
    document has none) and the cuts."""
    cuts = torch.randint(4, total - 3, (count - 1,), generator=generator).sort().values
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([total])])
    tokens = torch.empty(rows, total, dtype=torch.int64)
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        start = torch.randint(vocab, (rows, 1), generator=generator)
        step = torch.randint(1, 4, (rows, 1), generator=generator)
        tokens[:, a:b] = (start + step * torch.arange(b - a)) % vocab
    targets = torch.cat([tokens[:, 1:], torch.full((rows, 1), -1)], 1)
    targets[:, cu[1:-1] - 1] = -1
    return tokens.cuda(), targets.cuda(), cu.to(torch.int32).cuda()


def train(model, steps, vocab, rows=8, total=256, count=4, lr=3e-3, seed=1, every=0):
    """AdamW over fresh documents; the losses."""
    g = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr)
    losses = []
    for n in range(steps):
        tokens, targets, cu = documents(vocab, rows, total, count, g)
        loss = model.loss(tokens, targets, cu, entropy_weight=1e-4)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if every and n % every == 0:
            print("step %4d  loss %.4f" % (n, float(losses[-1])), flush=True)
    return torch.stack(losses)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--vocab", type=int, default=97)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=2)
    a = ap.parse_args()
    model = GatedLM(a.vocab, a.width, a.blocks)
    train(model, a.steps, a.vocab, every=max(1, a.steps // 10))
    prompt = torch.tensor([[5, 7, 9, 11, 13, 15], [90, 93, 96, 2, 5, 8]]) % a.vocab
    print("continuing 5 7 9 11 13 15 and 90 93 96 2 5 8:", model.generate(prompt.cuda(), 6).tolist())


if __name__ == "__main__":
    main()
