"""The router on the GPU against the 64-bit reference.

Tolerances: scores are fp32 from expf (2 ulp) with sums of at most 512 terms,
16 by a thread and 5 by shuffles: within 2^-19 relative. Gates divide two such
sums. The balance loss sums shares kept to 2^-40. A gradient element is a
difference of two fp32 sums of at most 512 products, each within 2^-18 of its
terms' sizes, then rounded (bf16: 2^-8).
"""
import math

import numpy as np
import pytest
import torch

import objective_reference as R

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
REL = 2.0**-18


def host(x):
    return x.double().cpu().numpy()


def make(rng, tokens, experts, dtype, k, score, bias, pad=0, shift=0, spread=1.5):
    """Logits whose choice does not hang on rounding (with a bias: gaps of
    2e-6 between scores; without one the logits themselves decide)."""
    ld = experts + pad
    buf = torch.zeros(shift + max(tokens, 1) * ld, dtype=dtype, device="cuda")
    x = torch.as_strided(buf, (tokens, experts), (ld, 1), shift)
    at = np.arange(tokens)
    for _ in range(50):
        if len(at) == 0:
            break
        new = torch.from_numpy((rng.normal(size=(len(at), experts)) * spread).astype(np.float32))
        x[torch.from_numpy(at).cuda()] = new.to(dtype).cuda()
        if bias is None or experts == 1:
            break
        v = host(x)[at]
        s = np.exp(R.log_softmax(v)) if score == "softmax" else 1 / (1 + np.exp(-v))
        top = -np.sort(-(s + bias), axis=1)[:, :k + 1]
        at = at[(top[:, :-1] - top[:, 1:]).min(1) < 2e-6]
    return x


CASES = [  # tokens, experts, k, dtype, score, renorm, bias, sequences, masked, pad, shift
    (1, 1, 1, BF16, "softmax", True, False, None, False, 0, 0),
    (1, 8, 2, BF16, "softmax", True, False, None, False, 0, 0),
    (5, 7, 7, FP32, "sigmoid", True, True, None, True, 1, 1),
    (64, 32, 4, BF16, "softmax", True, False, None, False, 0, 0),
    (300, 33, 3, BF16, "softmax", False, True, (0, 100, 100, 300), True, 3, 1),
    (1000, 64, 6, FP32, "softmax", True, True, (0, 1, 1000), True, 0, 0),
    (777, 127, 8, BF16, "sigmoid", False, False, (5, 500, 700), True, 0, 1),
    (2049, 256, 8, FP32, "sigmoid", True, True, (0, 0, 513, 2049, 2049), True, 0, 0),
    (130, 257, 5, BF16, "softmax", True, False, None, False, 0, 0),
    (300, 512, 32, FP32, "sigmoid", True, True, (0, 17, 300), True, 2, 3),
    (9000, 8, 2, BF16, "softmax", True, False, (0, 4000, 9000), True, 0, 0),
    (5000, 16, 1, FP32, "softmax", False, False, None, True, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:5]))
def test_route_and_gradient(case):
    from fsdp_buffer_layout_gb300.objectives import Router
    tokens, experts, k, dtype, score, renorm, biased, starts, masked, pad, shift = case
    rng = np.random.default_rng(tokens + experts)
    bias = (0.05 * rng.normal(size=experts)).astype(np.float32) if biased else None
    x = make(rng, tokens, experts, dtype, k, score, bias, pad, shift)
    live = (rng.random(tokens) < 0.8).astype(np.uint8) if masked else None
    dg = rng.normal(size=(tokens, k)).astype(np.float32)
    if masked:
        x[torch.from_numpy(live == 0).cuda()] = math.nan
        dg[live == 0] = np.nan
    op = Router(tokens, experts, k, dtype=dtype, score=score, renorm=renorm, route_scale=1.5,
                balance=0.3, sequences=1 if starts is None else len(starts) - 1)
    more = dict(live=None if live is None else torch.from_numpy(live).cuda(),
                seq_starts=None if starts is None else torch.tensor(starts, device="cuda"))
    idx, gates, counts, loss = op.forward(x, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                                          **more)
    b64 = None if bias is None else bias.astype(np.float64)
    clean = np.nan_to_num(host(x))
    i, g, c, l, grad = R.route(clean, k, score, renorm, 1.5, float(np.float32(0.3)), b64, live,
                               starts, dg, 0.5)
    assert np.array_equal(idx.cpu().numpy(), i)
    assert np.array_equal(counts.cpu().numpy(), c)
    assert (np.abs(host(gates) - g) <= 2 * REL * np.abs(g) + 1e-30).all()
    assert abs(loss.item() - l) <= REL * abs(l) + experts * 2.0**-40
    got = op.backward(x, torch.from_numpy(dg).cuda(), loss_scale=0.5, **more)
    dgn = np.nan_to_num(dg)
    # sizes of the terms: the gates' pull and the balance term on each score
    s = np.exp(R.log_softmax(clean)) if score == "softmax" else 1 / (1 + np.exp(-clean))
    pull = np.zeros_like(clean)
    for t in range(tokens):
        if i[t, 0] >= 0:
            picked = s[t, i[t]]
            down = picked.sum() if renorm else 1.0
            pull[t, i[t]] = 1.5 * (np.abs(dgn[t]) + (np.abs(dgn[t]) @ picked / down if renorm else 0)) / down
    seq_c = op.seq_counts.cpu().numpy().max(0) * float(op.seq_coef.max())
    pull += 0.5 * seq_c / (1 if score == "softmax" else s.sum(1, keepdims=True))
    size = s * (pull + (s * pull).sum(1, keepdims=True))
    lim = 8 * REL * size + (2.0**-8 if dtype == BF16 else 2.0**-23) * np.abs(grad) + 1e-30
    err = np.abs(host(got) - grad)
    assert (err <= lim).all(), (err / lim).max()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_ties_infinities_and_nan(dtype):
    """Equal logits go to the lowest expert, -0 equals +0, -inf is taken last
    but before NaN, and every index stays in range."""
    from fsdp_buffer_layout_gb300.objectives import Router
    inf, nan = math.inf, math.nan
    rows = [[1, 1, 1, 1, 1], [0.0, -0.0, 0.0, -1, 1], [-inf, 2, -inf, -inf, 1], [nan, 1, nan, -inf, 0],
            [-1, -0.0, 0.0, -2, -3], [nan] * 5]
    x = torch.tensor(rows, dtype=dtype, device="cuda")
    op = Router(6, 5, 3, dtype=dtype)
    idx, gates, counts, loss = op.forward(x)
    assert idx.tolist() == [[0, 1, 2], [4, 0, 1], [1, 4, 0], [1, 4, 3], [1, 2, 0], [0, 1, 2]]
    assert torch.isnan(gates).any(1).tolist() == [False, False, False, True, False, True]
    assert counts.sum().item() == 18 and math.isnan(loss.item())
    # the next call starts afresh
    assert math.isfinite(op.forward(x[:3])[3].item())
    grad = op.backward(x[:3], torch.ones(3, 3, device="cuda"))
    assert torch.isfinite(grad).all() and grad[2, 0].item() == 0


@pytest.mark.parametrize("experts,k", [(5, 5), (8, 8), (15, 3), (32, 4), (32, 12), (40, 8), (64, 8), (64, 32),
                                       (100, 6), (128, 8), (128, 30), (200, 8), (256, 8), (256, 32), (400, 10),
                                       (512, 8), (512, 20)])
def test_ties_go_to_the_lowest_expert(experts, k):
    """Few different logits, so that the K-th place is mostly a tie; all equal
    in the last rows; some -inf (after every finite logit) and NaN (last)."""
    from fsdp_buffer_layout_gb300.objectives import Router
    rng = np.random.default_rng(experts + k)
    x = rng.integers(0, 3, (500, experts)).astype(np.float32)
    x[100:200][rng.random((100, experts)) < 0.9] = -math.inf
    x[450:] = 1.0
    x[150:250][rng.random((100, experts)) < 0.5] = math.nan
    order = np.where(np.isnan(x), 10.0, np.where(np.isinf(x), 5.0, -x))
    want = np.argsort(order, axis=1, kind="stable")[:, :k]
    for dtype in (BF16, FP32):
        idx = Router(500, experts, k, dtype=dtype).forward(torch.from_numpy(x).to("cuda", dtype))[0]
        assert np.array_equal(idx.cpu().numpy(), want)

def test_nothing_live_and_no_tokens():
    from fsdp_buffer_layout_gb300.objectives import Router
    op = Router(70, 12, 3, dtype=FP32, balance=0.1)
    x = torch.full((70, 12), math.nan, device="cuda")
    dead = torch.zeros(70, dtype=torch.uint8, device="cuda")
    idx, gates, counts, loss = op.forward(x, live=dead)
    assert (idx == -1).all() and (gates == 0).all() and (counts == 0).all() and loss.item() == 0
    assert (op.backward(x, torch.ones(70, 3, device="cuda"), live=dead) == 0).all()
    idx, gates, counts, loss = op.forward(x[:0])
    assert idx.shape == (0, 3) and (counts == 0).all() and loss.item() == 0
    assert op.backward(x[:0]).shape == (0, 12)


def test_same_bits_again_in_place_on_a_stream_and_in_a_graph():
    from fsdp_buffer_layout_gb300.objectives import Router
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.normal(size=(4000, 64)).astype(np.float32)).cuda()
    dg = torch.from_numpy(rng.normal(size=(4000, 4)).astype(np.float32)).cuda()
    starts = torch.tensor([0, 11, 3000, 4000], device="cuda")

    def run(op, grad=None):
        out = list(op.forward(x, seq_starts=starts))
        return out + [op.backward(x, dg, seq_starts=starts, grad=grad)]

    kw = dict(dtype=FP32, balance=0.1, score="sigmoid", sequences=3)
    want = [t.clone() for t in run(Router(4000, 64, 4, **kw))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    op = Router(4000, 64, 4, stream=side, **kw)
    for _ in range(3):
        got = run(op)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(op)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(run(Router(4000, 64, 4, **kw), grad=x)[4], want[4])  # over the logits


def test_balance_alone_and_gates_alone():
    """Without d_gates only the balance loss pulls; with loss_scale 0 only the
    gates do."""
    from fsdp_buffer_layout_gb300.objectives import Router
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.normal(size=(50, 10)).astype(np.float32)).cuda()
    dg = rng.normal(size=(50, 2)).astype(np.float32)
    op = Router(50, 10, 2, dtype=FP32, balance=0.2)
    op.forward(x)
    a = R.route(host(x), 2, "softmax", True, 1.0, float(np.float32(0.2)))[4]
    b = R.route(host(x), 2, "softmax", True, 1.0, 0.0, d_gates=dg)[4]
    assert np.abs(host(op.backward(x)) - a).max() < 1e-7 + 8 * REL * np.abs(a).max()
    got = op.backward(x, torch.from_numpy(dg).cuda(), loss_scale=0.0)
    assert np.abs(host(got) - b).max() < 8 * REL * np.abs(dg).max()


def test_python_refusals():
    from fsdp_buffer_layout_gb300.objectives import Router
    x = torch.zeros(4, 8, device="cuda")
    op = Router(4, 8, 2, dtype=FP32)
    for bad in (x.bfloat16(), x[:, :7], torch.zeros(5, 8, device="cuda"), x.cpu()):
        with pytest.raises(ValueError):
            op.forward(bad)
    with pytest.raises(ValueError):
        op.forward(x, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        op.forward(x, live=torch.ones(4, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        op.backward(x, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        Router(4, 8, 2, dtype=FP32, sequences=2).forward(x)
    with pytest.raises(ValueError):
        Router(4, 8, 2, score="tanh")


@pytest.mark.parametrize("experts,k", [(3, 3), (9, 8), (16, 9), (24, 4), (32, 20), (32, 5), (48, 8), (64, 8),
                                       (64, 12), (128, 3), (128, 8), (128, 11), (512, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_route_several_tokens_a_warp(experts, k, score, dtype):
    """Several tokens a warp up to 8 choices of up to 64, or of 128 experts, else
    one; full rows and others."""
    test_route_and_gradient((1037, experts, k, dtype, score, True, True, (0, 5, 5, 700, 1030), True, 0, 0))


@pytest.mark.parametrize("sequences", [1, 31, 32, 33, 700])
def test_many_sequences(sequences):
    """The walk through the sequences' starts, empty ones among them, and the
    finish by the last CTA or by a launch of its own."""
    from fsdp_buffer_layout_gb300.objectives import Router
    rng = np.random.default_rng(sequences)
    starts = np.sort(rng.integers(0, 3001, sequences + 1))
    starts[0] = 0
    x = make(rng, 3000, 40, FP32, 3, "softmax", None)
    op = Router(3000, 40, 3, dtype=FP32, balance=0.2, sequences=sequences)
    more = dict(seq_starts=torch.tensor(starts, device="cuda"))
    i, g, c, l, grad = R.route(host(x), 3, "softmax", True, 1.0, float(np.float32(0.2)), starts=starts)
    for _ in range(2):
        idx, gates, counts, loss = op.forward(x, **more)
        assert np.array_equal(idx.cpu().numpy(), i) and np.array_equal(counts.cpu().numpy(), c)
        assert abs(loss.item() - l) <= REL * abs(l) + 40 * sequences * 2.0**-40
    got = host(op.backward(x, **more))
    assert np.abs(got - grad).max() <= 8 * REL * max(np.abs(grad).max(), 0.2 * 40 / 3)
