"""The post-training example on the framework's experts and token scores: the
operators together, as a training step calls them.

Gradients of the same model with the experts as torch products: both sides round
to bf16 after each product, the gates' sum and its gradient, and the residual, some
eight times between a parameter and the logits, each by half a step at most (2^-8
of a value), so two results differ by less than 8 2^-8 of a tensor's norm."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts,top_k,hidden,inner", [(8, 2, 128, 256), (13, 3, 72, 200), (4, 4, 64, 96)])
def test_gradients_against_torch_products(experts, top_k, hidden, inner):
    import post_train_moe as P
    sizes = dict(vocab=512, hidden=hidden, inner=inner, experts=experts, top_k=top_k, tokens=96)
    models = [P.TinyMoE(kernels=k, **sizes) for k in (True, False)]
    try:
        g = torch.Generator(device="cuda").manual_seed(5)
        inputs = torch.randint(0, 512, (96,), device="cuda", generator=g)
        d_logits = (torch.randn(96, 512, device="cuda", generator=g) / 96).bfloat16()
        out = []
        for m in models:
            logits, _ = m.logits(inputs)
            out.append((logits.detach(), torch.autograd.grad(logits, list(m.params.values()), d_logits)))
        bound = 8 * 2.0**-8
        a, b = (o[0].float() for o in out)
        assert (a - b).norm() < bound * b.norm()
        for name, a, b in zip(models[0].params, out[0][1], out[1][1]):
            assert torch.isfinite(a).all()
            assert (a.float() - b.float()).norm() < bound * b.float().norm(), name
        assert models[0].experts.up.device_error() == models[0].experts.down.device_error() == 0
    finally:
        for m in models:
            m.shard.close()


def test_the_example_runs_on_the_kernels():
    import post_train_moe as P
    model = P.TinyMoE(kernels=True)
    lines = []
    try:
        P.policy_phase(model, 3, 256, log=lines.append, entropy_bonus=0.01)
        P.preference_phase(model, 2, 4, 32, log=lines.append)
        assert len(lines) == 9 and not any("nan" in line for line in lines)
        assert model.shard.device_error() == 0
        assert model.experts.up.device_error() == model.experts.down.device_error() == 0
    finally:
        model.shard.close()


def test_backward_refuses_another_forward():
    """The experts' buffers hold the last forward call's rows."""
    import post_train_moe as P
    model = P.TinyMoE(vocab=256, hidden=64, inner=64, tokens=32, kernels=True)
    try:
        inputs = torch.arange(32, device="cuda")
        first, _ = model.logits(inputs)
        model.logits(inputs + 7)
        with pytest.raises(ValueError, match="has followed"):
            torch.autograd.grad(first, model.params["up"], torch.zeros_like(first))
    finally:
        model.shard.close()


def test_the_whole_layer_in_a_graph():
    """Router, dispatch, products and scores captured once, replayed on new tokens: the
    bits of eager calls."""
    from fsdp_buffer_layout_gb300.experts import Dispatch, ExpertLinear
    from fsdp_buffer_layout_gb300.objectives import Router, TokenScores
    tokens, experts, top_k, hidden, inner, vocab = 200, 16, 4, 256, 384, 1024
    g = torch.Generator(device="cuda").manual_seed(9)

    def rand(*shape):
        return (torch.randn(*shape, device="cuda", generator=g) * shape[-1] ** -0.5).bfloat16()

    up, down, head, gate = rand(experts, inner, hidden), rand(experts, hidden, inner), rand(vocab, hidden), \
        rand(experts, hidden)
    x = [torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16() for _ in range(3)]
    targets = torch.randint(-1, vocab, (tokens,), device="cuda", generator=g)
    one = torch.ones(tokens, device="cuda")

    class Layer:
        def __init__(self, stream=None):
            self.router = Router(tokens, experts, top_k, stream=stream)
            self.to = Dispatch(tokens, experts, top_k, hidden, stream=stream)
            self.up = ExpertLinear(tokens * top_k, experts, inner, hidden, stream=stream)
            self.down = ExpertLinear(tokens * top_k, experts, hidden, inner, stream=stream)
            self.scores = TokenScores(tokens, vocab, top_k=3, stream=stream)

        def __call__(self, x):
            idx, gates, _, _ = self.router.forward(x @ gate.t())
            starts, _, _ = self.to.sort(idx)
            rows = self.to.gather(x)
            h = torch.relu(self.up.forward(rows, up, starts))
            y = self.down.forward(h, down, starts)
            out = self.to.combine(y, gates)
            logits = out @ head.t()
            logp, entropy, top, top_logp = self.scores.forward(logits, targets)
            d = self.scores.backward(logits, targets, d_logp=one, d_entropy=one)
            d_y, d_gates = self.to.combine_backward(d @ head, y, gates)
            d_h = self.down.backward_input(d_y, down, starts) * (h > 0)
            d_x = self.to.gather_backward(self.up.backward_input(d_h, up, starts))
            return (out, logp, entropy, top, top_logp, d, d_gates, d_x,
                    self.up.backward_weight(d_h, rows, starts), self.down.backward_weight(d_y, h, starts))

    eager = Layer()
    want = [[t.clone() for t in eager(v)] for v in x]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    layer, fixed = Layer(stream), x[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        layer(fixed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = layer(fixed)
    for v, w in zip(x, want):
        torch.cuda.synchronize()
        fixed.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, w):
            assert torch.equal(a, b)
