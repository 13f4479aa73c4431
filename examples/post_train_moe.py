"""Post-training a small mixture-of-experts language model on one GPU, end to
end through the framework: the router and the losses turn the model's outputs
into gradients (objectives.Router, TokenLogprobs, PolicyLoss, PreferenceLoss),
the shard step packs, clips and applies them (step.ShardStep). Embedding,
experts and output projection are plain torch products.

    python examples/post_train_moe.py [--steps N]

Two phases on synthetic data: policy updates on one batch of sampled tokens
whose advantage is +1 for even tokens and -1 for odd ones, then preference
updates on pairs of sequences. Prints each step's losses.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fsdp_buffer_layout_gb300 import vsf as V  # noqa: E402
from fsdp_buffer_layout_gb300.objectives import (  # noqa: E402
    PolicyLoss, PreferenceLoss, Router, TokenLogprobs)
from fsdp_buffer_layout_gb300.step import ShardStep, TensorSpec  # noqa: E402


class Route(torch.autograd.Function):
    """The router for autograd: gates (differentiable) and the choice. The
    balance loss pulls on the logits in backward with its own weight."""

    @staticmethod
    def forward(ctx, logits, router):
        idx, gates, _, balance = router.forward(logits)
        ctx.router, ctx.call = router, router.calls
        ctx.save_for_backward(logits)
        ctx.mark_non_differentiable(idx, balance)
        return gates, idx, balance

    @staticmethod
    def backward(ctx, d_gates, _idx, _balance):
        logits, = ctx.saved_tensors
        return ctx.router.backward(logits, d_gates.contiguous(), call=ctx.call), None


class TinyMoE:
    """embed -> router -> top-k of E experts (one hidden layer) -> project.
    Parameters are bf16 tensors; their gradients go to a ShardStep as they are."""

    def __init__(self, vocab=2048, hidden=128, inner=256, experts=8, top_k=2, tokens=256, seed=0,
                 lr=2e-4, balance=1e-2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        shapes = {"embed": (vocab, hidden), "router": (experts, hidden),
                  "up": (experts, inner, hidden), "down": (experts, hidden, inner),
                  "head": (vocab, hidden)}
        self.params = {n: (torch.randn(s, device="cuda", generator=g) * s[-1] ** -0.5)
                       .bfloat16().requires_grad_() for n, s in shapes.items()}
        self.router = Router(tokens, experts, top_k, balance=balance)
        # rows of 32 quantised together, as for the layers of the larger workloads
        specs = [TensorSpec(s, V.VSF_GRAN_ROWS, 32) if s[0] >= 32 or len(s) == 3
                 else TensorSpec(s, V.VSF_GRAN_ELEM) for s in shapes.values()]
        self.shard = ShardStep(specs, m=4, g_coll=128, lr=lr, weight_decay=0.0, max_norm=1.0, world=1)
        for t, p in enumerate(self.params.values()):
            self.shard.load_master(t, p.detach().float())
        self.count = 0

    def logits(self, inputs):
        """Logits [tokens, vocab] and the balance loss for input tokens."""
        p = self.params
        x = p["embed"][inputs]
        gates, idx, balance = Route.apply(x @ p["router"].t(), self.router)
        mixed = torch.zeros_like(x, dtype=torch.float32)
        for e in range(p["router"].shape[0]):
            token, slot = torch.nonzero(idx == e, as_tuple=True)
            hidden = torch.relu(x[token] @ p["up"][e].t())
            out = (hidden @ p["down"][e].t()).float() * gates[token, slot, None]
            mixed = mixed.index_add(0, token, out)
        return (x + mixed.bfloat16()) @ p["head"].t(), balance

    def update(self, logits, d_logits):
        """Backward from the logits' gradient, then one shard step."""
        grads = torch.autograd.grad(logits, list(self.params.values()), d_logits)
        self.count += 1
        with torch.no_grad():
            self.shard.step([g.contiguous() for g in grads],
                            [p.detach() for p in self.params.values()], self.count)
        return grads


def policy_phase(model, steps, tokens, log=print):
    """Returns the batch's mean advantage-weighted log ratio after the steps."""
    g = torch.Generator(device="cuda").manual_seed(1)
    vocab = model.params["embed"].shape[0]
    inputs = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
    logprobs = TokenLogprobs(tokens, vocab)
    with torch.no_grad():
        start, _ = model.logits(inputs)
        targets = torch.multinomial(torch.softmax(start.float(), 1), 1, generator=g).flatten()
        old = logprobs(start, targets).clone()
    advantages = torch.where(targets % 2 == 0, 1.0, -1.0)
    weights = torch.ones(tokens, device="cuda")
    weights[-tokens // 8:] = 0.0  # padding
    loss = PolicyLoss(tokens, vocab, clip_low=0.2, clip_high=0.3, kl_beta=0.02)
    logp = old
    for step in range(steps):
        logits, balance = model.logits(inputs)
        stats, logp, d_logits = loss(logits.detach(), targets, old, advantages, ref_logp=old,
                                     weights=weights)
        model.update(logits, d_logits)
        log("policy %d: loss %.5f policy %.5f kl %.6f balance %.5f" % (
            step, stats[0], stats[1], stats[2], balance))
    with torch.no_grad():
        logp = logprobs(model.logits(inputs)[0], targets)
    return ((logp - old) * advantages * weights).sum().item() / weights.sum().item()


def preference_phase(model, steps, pairs, length, log=print):
    """Returns the mean reward margin before and after the steps."""
    g = torch.Generator(device="cuda").manual_seed(2)
    vocab, tokens = model.params["embed"].shape[0], 2 * pairs * length
    inputs = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
    targets = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
    starts = torch.arange(0, tokens + 1, length, device="cuda")
    with torch.no_grad():
        reference = TokenLogprobs(tokens, vocab)(model.logits(inputs)[0], targets).clone()
    loss = PreferenceLoss(pairs, tokens, vocab, beta=0.1)
    margins = []
    for step in range(steps + 1):
        logits, balance = model.logits(inputs)
        stats, _, _, d_logits = loss(logits.detach(), targets, starts, ref_logp=reference)
        margins.append(stats[1].item())
        log("preference %d: loss %.5f margin %.5f balance %.5f" % (
            step, stats[0], stats[1], balance))
        if step < steps:
            model.update(logits, d_logits)
    return margins[0], margins[-1]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    model = TinyMoE()
    print("policy: mean advantage-weighted log ratio %.4f" % policy_phase(model, a.steps, 256))
    print("preference: margin %.4f -> %.4f" % preference_phase(model, a.steps, 4, 32))
    model.shard.close()


if __name__ == "__main__":
    main()
