"""The post-training example: the operators together, through the shard step.

The model's gradients (through the router and the policy loss) against torch's
autograd on the same model with plain forms of both in fp32: the products run
in bf16 on either side, so gradients agree to bf16's rounding of the logits'
gradient and of each product's result, a few times 2^-8 of a tensor's norm."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_policy_and_preference_phases_learn():
    import post_train_moe as P
    model = P.TinyMoE()
    lines = []
    try:
        assert P.policy_phase(model, 6, 256, log=lines.append) > 0.02
        before, after = P.preference_phase(model, 6, 4, 32, log=lines.append)
        # the reference is the model itself, rounded to fp32: half a unit of the
        # last place of 8..16, 2^-21, for each of a pair's 64 tokens, times beta
        assert abs(before) <= 0.1 * 64 * 2.0**-21 and after > 0.02
        assert len(lines) == 13 and model.shard.device_error() == 0
    finally:
        model.shard.close()


def test_gradients_against_plain_autograd():
    import post_train_moe as P
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    model = P.TinyMoE(vocab=512, tokens=64, balance=0.05)
    try:
        g = torch.Generator(device="cuda").manual_seed(3)
        inputs = torch.randint(0, 512, (64,), device="cuda", generator=g)
        targets = torch.randint(0, 512, (64,), device="cuda", generator=g)
        adv = torch.randn(64, device="cuda", generator=g)
        logits, balance = model.logits(inputs)
        old = torch.log_softmax(logits.detach().float(), 1).gather(1, targets[:, None])[:, 0]
        loss = PolicyLoss(64, 512, kl_beta=0.1)
        stats, _, d_logits = loss(logits.detach(), targets, old, adv, ref_logp=old - 0.3)
        got = torch.autograd.grad(logits, list(model.params.values()), d_logits)

        # the same with plain forms
        p = model.params
        x = p["embed"][inputs]
        r = (x @ p["router"].t()).float()
        probs = torch.softmax(r, 1)
        idx = torch.sort(r, dim=1, descending=True, stable=True).indices[:, :2]
        picked = probs.gather(1, idx)
        gates = picked / picked.sum(1, keepdim=True)
        counts = torch.bincount(idx.flatten(), minlength=8).float()
        plain_balance = 0.05 * 8 / (2 * 64 * 64) * (counts * probs.sum(0)).sum()
        mixed = torch.zeros(64, x.shape[1], device="cuda")
        for e in range(8):
            token, slot = torch.nonzero(idx == e, as_tuple=True)
            out = (torch.relu(x[token] @ p["up"][e].t()) @ p["down"][e].t()).float()
            mixed = mixed.index_add(0, token, out * gates[token, slot, None])
        y = ((x + mixed.bfloat16()) @ p["head"].t()).float()
        logp = torch.log_softmax(y, 1).gather(1, targets[:, None])[:, 0]
        ratio = torch.exp(logp - old)
        u = old - 0.3 - logp
        plain = (-torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv)
                 + 0.1 * (torch.exp(u) - u - 1)).mean()
        want = torch.autograd.grad(plain + plain_balance, list(p.values()))
        assert abs(balance.item() - plain_balance.item()) < 1e-5 * plain_balance.item()
        assert abs(stats[0].item() - plain.item()) < 1e-4
        for name, a, b in zip(p, got, want):
            off = (a.float() - b.float()).norm() / b.float().norm()
            assert off < 6 * 2.0**-8, (name, off.item())
    finally:
        model.shard.close()
