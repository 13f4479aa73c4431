"""Token log probabilities, policy loss and preference loss on the GPU against
the 64-bit reference.

Tolerances, from the arithmetic: a term exp(x - m) of a row's sum is within
2^-22 (ex2.approx) plus the rounding of its argument, t 2^-24 with a
sum-weighted |t| of at most log2 V, of its value; a thread adds at most
V / 256 + 40 of them in fp32 (2^-24 each). So the sum, and with it ln p
absolutely, is within tol(V); ln p is then rounded to fp32. A gradient element
is a (1[v = y] - p), where a's relative error is at most the loss's slope's
and p's twice tol(V) plus the 2^-22 + |t| 2^-24 (|t| <= 60 where p matters) of
its own term; bf16 (8 significant bits) rounds by 2^-8 of the value at most.
"""
import math

import numpy as np
import pytest
import torch

import objective_reference as R

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def tol(vocab):
    return 2.0**-22 + (math.log2(vocab) + 1) * 2.0**-23 + (vocab / 256 + 40) * 2.0**-24


def make_logits(rng, tokens, vocab, dtype, pad=0, shift=0, scale=2.5):
    """Rows of stride vocab + pad that start `shift` elements into a buffer."""
    ld = vocab + pad
    buf = torch.empty(shift + max(tokens, 1) * ld, dtype=dtype, device="cuda")
    buf.copy_(torch.from_numpy(rng.normal(size=buf.numel()).astype(np.float32) * scale))
    return torch.as_strided(buf, (tokens, vocab), (ld, 1), shift)


def host(x):
    return x.double().cpu().numpy()


def dev(a, dtype=torch.float32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def check_logp(got, want, vocab):
    lim = tol(vocab) + 2.0**-24 * np.abs(want) + 1e-9
    assert (np.abs(host(got) - want) <= lim).all(), np.abs(host(got) - want).max()


def check_grad(got, want, dtype, vocab, row_scale):
    """row_scale: per row, the sizes of the terms that make up a."""
    err = np.abs(host(got) - want)
    rel = 2 * tol(vocab) + 2.0**-22 + 60 * 2.0**-24 + (2.0**-8 if dtype == BF16 else 2.0**-23)
    lim = rel * np.abs(want) + row_scale[:, None] * (8 * tol(vocab)) * (np.abs(want) > 0) + 1e-30
    # at the target 1 - p cancels: its error is that of p
    lim += (row_scale * 4 * tol(vocab))[:, None] * (np.abs(want) == np.abs(want).max(1, keepdims=True))
    assert (err <= lim).all(), (err / lim).max()


SHAPES = [  # tokens, vocab, dtype, pad, shift
    (1, 1, BF16, 0, 0), (3, 2, FP32, 0, 0), (5, 31, BF16, 2, 1), (1, 1000, FP32, 0, 3),
    (7, 257, BF16, 0, 0), (17, 4096, BF16, 0, 0), (9, 5003, FP32, 1, 1), (4, 32000, BF16, 0, 0),
    (3, 32000, FP32, 0, 0), (6, 50021, BF16, 3, 5), (3, 65537, FP32, 2, 1),
    (2, 131072, BF16, 0, 0), (2, 131075, FP32, 5, 2), (2, 300001, BF16, 0, 0),
    (200, 640, BF16, 0, 0), (700, 96, FP32, 0, 0),
]


@pytest.mark.parametrize("tokens,vocab,dtype,pad,shift", SHAPES)
def test_token_logprobs(tokens, vocab, dtype, pad, shift):
    from fsdp_buffer_layout_gb300.objectives import TokenLogprobs
    rng = np.random.default_rng(vocab)
    x = make_logits(rng, tokens, vocab, dtype, pad, shift)
    y = rng.integers(0, vocab, tokens)
    if tokens > 2:
        y[1] = -100
    for inv_t in (1.0, 1.25):
        op = TokenLogprobs(tokens, vocab, dtype=dtype, inv_temperature=inv_t)
        got = op(x, dev(y, torch.int64))
        check_logp(got, R.logprobs(host(x), y, inv_t), vocab)
        assert op.device_error() == 0


def policy_case(tokens, vocab, dtype, pad=0, shift=0, seed=0, masked=True):
    rng = np.random.default_rng(seed + vocab)
    x = make_logits(rng, tokens, vocab, dtype, pad, shift)
    y = rng.integers(0, vocab, tokens)
    w = rng.uniform(0.5, 1.5, tokens).astype(np.float32)
    if masked and tokens > 3:
        y[2], w[3] = -1, 0.0
    lp = R.logprobs(host(x), np.maximum(y, 0))
    ratio = np.exp(0.3 * rng.normal(size=tokens))
    for end in (0.8, 1.25):  # away from the ends of the clipping range
        ratio = np.where(np.abs(ratio - end) < 0.02, ratio + 0.05, ratio)
    old = (lp - np.log(ratio)).astype(np.float32)
    ref = (lp + 0.3 * rng.normal(size=tokens)).astype(np.float32)
    adv = rng.normal(size=tokens).astype(np.float32)
    return x, y, w, old, ref, adv


def policy_scale(lp, old, adv, ref, w, beta, f, inv_t):
    return np.abs(f * inv_t * w) * (np.abs(np.exp(lp - old) * adv) + beta * (1 + np.exp(ref - lp)))


@pytest.mark.parametrize("tokens,vocab,dtype,pad,shift", SHAPES)
@pytest.mark.parametrize("beta,mean,in_place", [(0.1, True, False), (0.0, False, True)])
def test_policy_loss(tokens, vocab, dtype, pad, shift, beta, mean, in_place):
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    x, y, w, old, ref, adv = policy_case(tokens, vocab, dtype, pad, shift)
    stats, lp, grad, _ = R.policy(host(x), y, old, adv, ref, w, 0.2, 0.25, beta, 1.0, 0.5, mean)
    op = PolicyLoss(tokens, vocab, dtype=dtype, clip_low=0.2, clip_high=0.25, kl_beta=beta,
                    scale=0.5, mean=mean)
    got = op(x, dev(y, torch.int64), dev(old), dev(adv), ref_logp=dev(ref) if beta else None,
             weights=dev(w), grad=x if in_place else None)
    check_logp(got[1], lp, vocab)
    f = 0.5 / stats[3] if mean else 0.5
    big = policy_scale(lp, old, adv, ref, w, beta, f, 1.0)
    check_grad(got[2], grad, dtype, vocab, big)
    lim = big.sum() * 4 * tol(vocab) + 2.0**-22 * np.abs(stats)
    assert (np.abs(host(got[0]) - stats) <= lim).all(), (host(got[0]), stats)
    assert op.device_error() == 0


def pair_starts(lengths):
    return np.cumsum([0] + list(lengths))


@pytest.mark.parametrize("vocab,dtype,pad,lengths,lead", [
    (33, FP32, 0, (1, 1), 0), (1000, BF16, 0, (5, 0, 3, 2), 2), (32000, BF16, 0, (4, 3), 0),
    (5003, FP32, 1, (7, 1, 0, 2, 9, 4), 1), (70001, BF16, 2, (2, 3), 0), (96, BF16, 0, (300, 411), 5),
])
@pytest.mark.parametrize("kind,average", [("sigmoid", False), ("squared", True)])
def test_preference_loss(vocab, dtype, pad, lengths, lead, kind, average):
    from fsdp_buffer_layout_gb300.objectives import PreferenceLoss
    rng = np.random.default_rng(vocab + len(lengths))
    starts = pair_starts(lengths) + lead
    tokens = int(starts[-1]) + lead  # tokens in no sequence before and after
    x = make_logits(rng, tokens, vocab, dtype, pad)
    y, w = rng.integers(0, vocab, tokens), rng.uniform(0.5, 1.5, tokens).astype(np.float32)
    if tokens > 4:
        y[-2] = -100
    ref = (R.logprobs(host(x), y) + 0.3 * rng.normal(size=tokens)).astype(np.float32)
    pairs = len(lengths) // 2
    op = PreferenceLoss(pairs, tokens, vocab, dtype=dtype, kind=kind, beta=0.3, smoothing=0.1,
                        margin=0.2, average=average, inv_temperature=0.9, scale=0.5)
    stats, rewards, lp, grad = op(x, dev(y, torch.int64), dev(starts, torch.int64),
                                  ref_logp=dev(ref), weights=dev(w))
    s, rw, l, g, slope = R.preference(host(x), y, starts, ref, w, kind, 0.3, 0.1, 0.2, average,
                                      float(np.float32(0.9)), 0.5)
    check_logp(lp, l, vocab)
    each = 1.5 * max(lengths) * tol(vocab)  # of a sequence's sum
    if average:
        each = 3 * tol(vocab)
    assert (np.abs(host(rewards) - rw) <= 0.3 * each + 2.0**-23 * np.abs(rw)).all()
    big = 2 * np.abs(rw).max() / 0.3 + 2
    assert (np.abs(host(stats) - s) <= 4 * each * big + 2.0**-22 * np.abs(s)).all(), (stats, s)
    # the slope moves with both sums: by 2 d h (squared), at most beta^2 / 4 d h (sigmoid)
    row = np.array([0 if a is None else abs(a) for a in slope]) * 0.9
    moved = 0.5 / pairs * 1.5 * (4 if average else 1) * 2 * each
    check_grad(grad, g, dtype, vocab, row + moved / (8 * tol(vocab)) * (row > 0))
    assert op.device_error() == 0


def test_no_reference_no_weights():
    from fsdp_buffer_layout_gb300.objectives import PreferenceLoss
    rng = np.random.default_rng(5)
    x, y = make_logits(rng, 9, 700, FP32), rng.integers(0, 700, 9)
    op = PreferenceLoss(1, 9, 700, dtype=FP32, beta=0.5)
    stats, rewards, lp, grad = op(x, dev(y, torch.int64), dev([0, 4, 9], torch.int64))
    s, rw, _, g, slope = R.preference(host(x), y, [0, 4, 9], None, None, "sigmoid", 0.5, 0.0, 0.0,
                                      False, 1.0, 1.0)
    assert np.abs(host(rewards) - rw).max() <= 10 * tol(700) + 2.0**-22 * np.abs(rw).max()
    assert np.abs(host(stats) - s).max() <= 20 * tol(700) + 2.0**-22 * np.abs(s).max()
    assert np.abs(host(grad) - g).max() <= 20 * tol(700)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_masked_words(dtype):
    """-inf and the type's lowest value in runs, at the start, at the end, at
    the target; the gradient of a masked word is 0."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    vocab = 9000
    rng = np.random.default_rng(1)
    x = make_logits(rng, 6, vocab, dtype)
    x[0, :8000] = -math.inf
    x[1, 100:] = torch.finfo(dtype).min
    x[2, 1:] = -math.inf
    x[3, ::2] = -math.inf
    x[4, :] = torch.finfo(dtype).min
    y = np.array([8500, 50, 0, 33, 7, 11])
    old, adv = np.full(6, -2.0, np.float32), np.array([1, -1, 1, -1, 0.5, 1], np.float32)
    op = PolicyLoss(6, vocab, dtype=dtype, clip_low=0.2, clip_high=1e6, mean=False)
    stats, lp, grad = op(x, dev(y, torch.int64), dev(old), dev(adv))
    s, l, g, _ = R.policy(host(x), y, old, adv, old, None, 0.2, 1e6, 0.0, 1.0, 1.0, False)
    check_logp(lp, l, vocab)
    assert lp[2].item() == 0.0
    check_grad(grad, g, dtype, vocab, policy_scale(l, old, adv, old, np.ones(6), 0.0, 1.0, 1.0))
    assert (grad[0, :8000] == 0).all() and (grad[3, ::2] == 0).all()


def test_rows_without_a_distribution_give_nan_and_stay_alone():
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, TokenLogprobs
    rng = np.random.default_rng(2)
    x = make_logits(rng, 5, 5000, FP32)
    x[1, 17], x[2, 400], x[3, :] = math.nan, math.inf, -math.inf
    y = np.array([1, 2, 3, 4, 5])
    lp = TokenLogprobs(5, 5000, dtype=FP32)(x, dev(y, torch.int64))
    assert torch.isnan(lp).tolist() == [False, True, True, True, False]
    one = dev(np.ones(5, np.float32))
    grad = PolicyLoss(5, 5000, dtype=FP32)(x, dev(y, torch.int64), lp.clone(), one)[2]
    assert torch.isnan(grad).any(1).tolist() == [False, True, True, True, False]
    check_logp(lp[[0, 4]], R.logprobs(host(x[[0, 4]]), y[[0, 4]]), 5000)


@pytest.mark.parametrize("vocab,dtype", [(3000, BF16), (40001, FP32)])
def test_masked_rows_are_not_read(vocab, dtype):
    """Rows of masked tokens hold NaN; rows whose mask leaves nothing at all
    give a loss of 0 and zero gradients."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss
    x, y, w, old, ref, adv = policy_case(8, vocab, dtype, masked=False)
    w[[1, 6]] = 0.0
    y[4] = -1
    x[[1, 4, 6]] = math.nan
    old[1] = ref[4] = adv[6] = np.nan
    op = PolicyLoss(8, vocab, dtype=dtype, kl_beta=0.1)
    stats, lp, grad = op(x, dev(y, torch.int64), dev(old), dev(adv), ref_logp=dev(ref),
                         weights=dev(w))
    assert torch.isfinite(stats).all() and torch.isfinite(grad).all()
    assert (grad[[1, 4, 6]] == 0).all() and (lp[[1, 4, 6]] == 0).all()
    nothing = torch.full((8,), -1, dtype=torch.int64, device="cuda")
    stats, lp, grad = op(x, nothing, dev(old), dev(adv), ref_logp=dev(ref), weights=dev(w))
    assert (stats == 0).all() and (lp == 0).all() and (grad == 0).all()
    pref = PreferenceLoss(1, 8, vocab, dtype=dtype, average=True)
    stats, rewards, lp, grad = pref(x, nothing, dev([0, 4, 8], torch.int64))
    assert abs(stats[0].item() - math.log(2)) < 1e-6 and (rewards == 0).all() and (grad == 0).all()


def test_target_out_of_range_sets_the_error_word():
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    x, y, w, old, ref, adv = policy_case(4, 500, BF16, masked=False)
    y[2] = 500
    op = PolicyLoss(4, 500)
    stats, lp, grad = op(x, dev(y, torch.int64), dev(old), dev(adv), weights=dev(w))
    assert op.device_error() == 16
    assert lp[2].item() == 0 and (grad[2] == 0).all() and grad[1].any()


def test_no_tokens():
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss, TokenLogprobs
    x, none = torch.empty(0, 100, dtype=BF16, device="cuda"), torch.empty(0, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    assert TokenLogprobs(4, 100)(x, y).numel() == 0
    stats, lp, grad = PolicyLoss(4, 100)(x, y, none, none)
    assert (stats == 0).all() and grad.shape == (0, 100)
    stats, rewards, _, _ = PreferenceLoss(2, 4, 100)(x, y, dev([0] * 5, torch.int64))
    assert abs(stats[0].item() - math.log(2)) < 1e-6 and (rewards == 0).all()


def test_offsets_past_32_bits():
    """Rows at element offsets above 2^32, in the logits and in the gradient,
    against the same rows close together (at the same places modulo 16 bytes,
    which set the order of a row's sum)."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    ld, vocab = (1 << 30) + 8, 1003
    x = torch.empty(4 * ld + vocab, dtype=BF16, device="cuda").as_strided((5, vocab), (ld, 1))
    g = torch.empty(4 * ld + vocab, dtype=BF16, device="cuda").as_strided((5, vocab), (ld, 1))
    small, y, w, old, ref, adv = policy_case(5, vocab, BF16, pad=5, masked=False)
    x.copy_(small)
    op = PolicyLoss(5, vocab, kl_beta=0.1)
    args = (dev(y, torch.int64), dev(old), dev(adv), dev(ref), dev(w))
    want = [t.clone() for t in op(small, *args)]
    got = op(x, *args, grad=g)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_bits_again_on_another_stream_and_in_a_graph():
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss
    x, y, w, old, ref, adv = policy_case(300, 8200, BF16)
    args = (x, dev(y, torch.int64), dev(old), dev(adv), dev(ref), dev(w))
    want = [t.clone() for t in PolicyLoss(300, 8200, kl_beta=0.1)(*args)]
    starts = dev([0, 100, 150, 290, 300], torch.int64)
    pref = (x, args[1], starts, args[4], args[5])
    want += [t.clone() for t in PreferenceLoss(2, 300, 8200)(*pref)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    op, pop = PolicyLoss(300, 8200, kl_beta=0.1, stream=side), PreferenceLoss(2, 300, 8200, stream=side)
    for _ in range(3):
        got = list(op(*args)) + list(pop(*pref))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t in got:
        t.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        op(*args)
        pop(*pref)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_against_differences_of_the_loss():
    """The kernel's gradient of fp32 logits against central differences of the
    64-bit losses (step 1e-5: their error is below 1e-8)."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss
    x, y, w, old, ref, adv = policy_case(5, 40, FP32)
    got = PolicyLoss(5, 40, dtype=FP32, clip_low=0.2, clip_high=0.25, kl_beta=0.2)(
        x, dev(y, torch.int64), dev(old), dev(adv), dev(ref), dev(w))[2]
    base = host(x)

    def difference(f, at, h=1e-5):
        up, down = base.copy(), base.copy()
        up[at] += h
        down[at] -= h
        return (f(up) - f(down)) / (2 * h)

    def loss(v):
        return R.policy(v, y, old, adv, ref, w, 0.2, 0.25, 0.2, 1.0, 1.0, True)[0][0]

    pref = PreferenceLoss(1, 5, 40, dtype=FP32, beta=0.4)(
        x, dev(y, torch.int64), dev([0, 2, 5], torch.int64), dev(ref), dev(w))[3]

    def pair_loss(v):
        return R.preference(v, y, [0, 2, 5], ref, w, "sigmoid", 0.4, 0.0, 0.0, False, 1.0, 1.0)[0][0]

    for t in range(5):
        for v in [0, 1, 39] + ([int(y[t])] if y[t] >= 0 else []):
            assert abs(got[t, v].item() - difference(loss, (t, v))) < 4e-6
            assert abs(pref[t, v].item() - difference(pair_loss, (t, v))) < 4e-6


def test_python_refusals():
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss, TokenLogprobs
    x, y, w, old, ref, adv = policy_case(4, 64, BF16)
    yt, o, a = dev(y, torch.int64), dev(old), dev(adv)
    op = PolicyLoss(4, 64)
    for bad in [(x.float(), yt, o, a), (x.cpu(), yt, o, a), (x[:, :63], yt, o, a), (x, yt.int(), o, a),
                (x, yt[:3], o, a), (x, yt, o.double(), a), (x, yt, o, a.cpu()),
                (x.t().contiguous().t(), yt, o, a), (x[:1].expand(4, 64), yt, o, a),
                (torch.cat([x, x]), yt, o, a)]:
        with pytest.raises(ValueError):
            op(*bad)
    with pytest.raises(ValueError):
        op(x, yt, o, a, grad=x[:3])
    with pytest.raises(ValueError):
        PolicyLoss(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        PreferenceLoss(1, 4, 64, kind="other")
    with pytest.raises(ValueError):
        PreferenceLoss(1, 4, 64)(x, yt, dev([0, 4], torch.int64))
    with pytest.raises(ValueError):
        TokenLogprobs(-1, 64)


@pytest.mark.parametrize("vocab,dtype,pad,lengths,lead", [
    (16500, BF16, 0, (60, 0, 100, 55, 40, 90), 0),
    (16511, BF16, 3, (400, 300, 1, 0, 500, 299), 7),
    (70001, FP32, 0, (200, 50, 0, 120, 0, 130, 30, 1), 0),
    (33000, FP32, 0, (2,) * 300, 3),
    (32000, BF16, 0, (3, 900), 100),
])
@pytest.mark.parametrize("kind,average", [("sigmoid", False), ("squared", True)])
def test_preference_loss_of_many_long_rows(vocab, dtype, pad, lengths, lead, kind, average):
    """More rows than SMs, beyond the short ones; sequences of very different
    lengths; many small pairs."""
    test_preference_loss(vocab, dtype, pad, lengths, lead, kind, average)


def test_preference_long_rows_in_place_and_same_bits():
    from fsdp_buffer_layout_gb300.objectives import PreferenceLoss
    rng = np.random.default_rng(8)
    x = make_logits(rng, 1600, 16500, BF16)
    y = rng.integers(0, 16500, 1600)
    y[rng.random(1600) < 0.3] = -1
    starts = dev([0, 300, 500, 900, 1000, 1300, 1590], torch.int64)
    ref = dev(rng.normal(size=1600))
    op = PreferenceLoss(3, 1600, 16500)
    args = (dev(y, torch.int64), starts, ref)
    want = [t.clone() for t in op(x, *args)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(op(x, *args), want))
    got = op(x, *args, grad=x)  # over the logits
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert op.device_error() == 0


@pytest.mark.parametrize("dtype,vocab", [(BF16, 32000), (FP32, 50021), (BF16, 5000)])
def test_policy_many_rows_masked_in_runs(dtype, vocab):
    """Several rows a cluster, masked in runs and at random: against the same
    rows in calls of their own."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    rng = np.random.default_rng(11)
    n = 1300
    x = make_logits(rng, n, vocab, dtype)
    y = rng.integers(0, vocab, n)
    y[(np.arange(n) % 100 < 30) | (rng.random(n) < 0.2)] = -1
    old, adv = dev(rng.normal(size=n) - 10), dev(rng.normal(size=n))
    yt = dev(y, torch.int64)
    op = PolicyLoss(n, vocab, dtype=dtype, kl_beta=0.1, mean=False)
    stats, lp, grad = (t.clone() for t in op(x, yt, old, adv, ref_logp=old))
    assert stats[3].item() == (y >= 0).sum()
    part = PolicyLoss(n, vocab, dtype=dtype, kl_beta=0.1, mean=False)
    for i in (0, 31, 299, 1299):
        s1, l1, g1 = part(x[i:i + 1], yt[i:i + 1], old[i:i + 1], adv[i:i + 1], ref_logp=old[i:i + 1])
        # (split over more CTAs, so summed in another order)
        assert abs(l1.item() - lp[i].item()) <= 2 * tol(vocab) + 2.0**-23 * abs(lp[i].item())
        a, b = host(g1[0]), host(grad[i])
        assert np.abs(a - b).max() <= 2.0**-7 * np.abs(b).max() if dtype == BF16 else \
            np.abs(a - b).max() <= 16 * tol(vocab) * np.abs(b).max()
    assert not grad[torch.from_numpy(y < 0).cuda()].any()


def test_rows_longer_than_a_cluster_holds():
    """800000 words: the policy loss in three passes."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    for vocab, masked in ((800000, False), (790003, True)):
        x, y, w, old, ref, adv = policy_case(5, vocab, BF16, masked=masked)
        op = PolicyLoss(5, vocab, clip_low=0.2, clip_high=0.25, kl_beta=0.1, scale=0.5)
        stats, lp, grad = op(x, dev(y, torch.int64), dev(old), dev(adv), ref_logp=dev(ref),
                             weights=dev(w))
        s, l, g, _ = R.policy(host(x), y, old, adv, ref, w, 0.2, 0.25, 0.1, 1.0, 0.5, True)
        check_logp(lp, l, vocab)
        big = policy_scale(l, old, adv, ref, w, 0.1, 0.5 / s[3], 1.0)
        check_grad(grad, g, BF16, vocab, big)
        assert (np.abs(host(stats) - s) <= big.sum() * 4 * tol(vocab) + 2.0**-22 * np.abs(s)).all()


def test_no_tokens_of_long_rows():
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss, TokenLogprobs
    x, none = torch.empty(0, 40000, dtype=BF16, device="cuda"), torch.empty(0, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    assert TokenLogprobs(4, 40000)(x, y).numel() == 0
    for mean in (True, False):
        stats, _, grad = PolicyLoss(4, 40000, mean=mean)(x, y, none, none)
        assert (stats == 0).all() and grad.shape == (0, 40000)
    stats, rewards, _, _ = PreferenceLoss(1, 4, 40000)(x, y, dev([0] * 3, torch.int64))
    assert abs(stats[0].item() - math.log(2)) < 1e-6 and (rewards == 0).all()


@pytest.mark.parametrize("vocab", [1000, 16500, 32000])
def test_calls_on_one_workspace_do_not_disturb_each_other(vocab):
    """Different sizes in turn on one object, as a ragged batch gives them."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss
    rng = np.random.default_rng(12)
    x = make_logits(rng, 2500, vocab, BF16)
    y = dev(rng.integers(0, vocab, 2500), torch.int64)
    old, adv = dev(rng.normal(size=2500) - 9), dev(rng.normal(size=2500))
    op, pop = PolicyLoss(2500, vocab, kl_beta=0.1), PreferenceLoss(2, 2500, vocab)
    sizes = (2500, 1, 160, 2100, 7, 900)
    starts = {n: dev([0, n // 4, n // 2, n // 2, n], torch.int64) for n in sizes}

    def calls(n):
        a = op(x[:n], y[:n], old[:n], adv[:n], ref_logp=old[:n])
        b = pop(x[:n], y[:n], starts[n], ref_logp=old[:n])
        return [t.clone() for t in a + b]

    want = {n: calls(n) for n in sizes}
    torch.cuda.synchronize()
    for n in sizes[::-1] + sizes:
        assert all(torch.equal(a, b) for a, b in zip(calls(n), want[n])), n


@pytest.mark.parametrize("vocab", [257, 20000])
def test_preference_of_impossible_tokens(vocab):
    """A target of probability 0 (a -inf logit): the pair's log ratio is
    infinite, the loss 0 or inf, the gradient what the saturated slope gives."""
    from fsdp_buffer_layout_gb300.objectives import PreferenceLoss
    rng = np.random.default_rng(13)
    x = make_logits(rng, 12, vocab, BF16)
    y = rng.integers(0, vocab, 12)
    starts = dev([0, 3, 6, 9, 12], torch.int64)
    op = PreferenceLoss(2, 12, vocab, beta=0.25)
    for row, first_loss, reward in ((7, 0.0, 2), (1, math.inf, 0)):
        z = x.clone()
        z[row, y[row]] = -math.inf
        stats, rewards, logp, grad = op(z, dev(y, torch.int64), starts)
        assert logp[row].item() == -math.inf and rewards[reward].item() == -math.inf
        assert op.device_error() == 0
        g = host(grad)
        assert np.isfinite(g).all()
        p = np.exp(R.log_softmax(host(z)))
        a = 0.0 if first_loss == 0.0 else 0.25 / 2
        for t in (0, 1, 2, 6, 7, 8):  # the first pair: chosen up, rejected down
            want = (1 if t < 3 else -1) * a * (p[t] - (np.arange(vocab) == y[t]))
            assert np.abs(g[t] - want).max() <= 2.0**-8 * max(a, 1e-30)
        pair = op.stats[0].item()
        if first_loss == 0.0:  # the second pair's alone, over two
            h = (host(logp)[3:6].sum() - host(logp)[9:12].sum()) * 0.25
            want = (math.log1p(math.exp(-abs(h))) + max(-h, 0.0)) / 2
            assert abs(pair - want) <= 1e-5 * max(1.0, abs(want))
        else:
            assert pair == math.inf
