"""The losses where rounding, size and place go wrong: rows far from zero, small
and large temperatures, long rows and long calls, and the elements of a
gradient that a loose tolerance would not see.

Tolerances, from the arithmetic. With t = (x - m) log2(e) / temperature, a term
2^t of a row's sum is within 2^-22 (ex2.approx) and |t| 2^-22 of its value (the
difference, c and the product are rounded once each: 3 |t| 2^-24); a thread adds
at most V / 256 + 40 of them in fp32. That bounds the relative error of the sum
and the absolute one of ln p (tol). Away from the target a gradient element is
-a p: its error is relative, a's share (coef_error) plus the sum's, the term's
and the output's rounding (bf16, 8 significant bits: 2^-8). A row of bf16 may
have the term 2^(x c - m c) with m c rounded once, where |m c| < 2^11: 2^-14 in
the exponent. At the target a (1 - p) cancels: a's error and p's, absolutely.
"""
import math

import numpy as np
import pytest
import torch

import objective_reference as R

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
LN2 = math.log(2)


def host(x):
    return x.double().cpu().numpy()


def dev(a, dtype=torch.float32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def tol(vocab):
    return 2.0**-22 + (math.log2(vocab) + 1) * 2.0**-22 + (vocab / 256 + 40) * 2.0**-24


def logp_error(vocab, logp):
    return tol(vocab) + 2.0**-23 * np.abs(logp) + 1e-9


def nan_rows(tokens, vocab, dtype, pad, shift=0):
    """A gradient buffer of NaN: (buffer, rows of stride vocab + pad in it)."""
    ld = vocab + pad
    buf = torch.full((shift + tokens * ld + 64,), math.nan, dtype=dtype, device="cuda")
    return buf, buf.as_strided((tokens, vocab), (ld, 1), shift)


def check_gradient(got, x, targets, slope, slope_error, inv_t, dtype):
    """got against slope_t inv_t (1[v = y] - p): slope in 64 bits (None: a masked
    row, zeros), slope_error its relative error."""
    vocab = x.shape[1]
    for t, a in enumerate(slope):
        row = got[t]
        if a is None or a == 0:
            assert not row.any(), t
            continue
        z = torch.from_numpy(x[t]).cuda() * inv_t
        z = z - z.max()
        p = torch.softmax(z, 0)
        y = int(targets[t])
        want = -a * inv_t * p
        rounding = 2.0**-8 if dtype == BF16 else 2.0**-23
        term = 2.0**-22 + z.clamp(min=-110.0).abs() / LN2 * 2.0**-22 * LN2
        if dtype == BF16:
            term = term + 2.0**-14 * LN2
        rel = slope_error[t] + 2 * tol(vocab) + term + rounding
        full = abs(a * inv_t)
        lim = rel * want.abs() + 2.0**-126 * (1 + full)  # (terms below 2^-126 are flushed)
        py = float(p[y])
        want[y] += a * inv_t
        lim[y] = full * (slope_error[t] + rounding * abs(1 - py) + py * (2 * tol(vocab) + float(term[y])) + 2.0**-22)
        err = (row.double() - want).abs()
        assert bool((err <= lim).all()), (t, float((err / lim).max()), int((err / lim).argmax()))


def policy_slope_error(lp, old, adv, ref, w, beta, f, slope, vocab):
    """Relative error of slope = f w (-r A - beta (exp u - 1)): r's and exp(u)'s
    is ln p's error and a few roundings."""
    out = []
    for t, a in enumerate(slope):
        if not a:
            out.append(0.0)
            continue
        e = logp_error(vocab, lp[t]) + 2.0**-23 * (abs(old[t]) + abs(ref[t])) + 2.0**-20
        out.append(abs(f * w[t]) * (abs(np.exp(lp[t] - old[t]) * adv[t]) + beta * (1 + np.exp(ref[t] - lp[t]))) * e / abs(a))
    return out


def policy_stats_error(w, adv, f, slope, err):
    """Of a sum of terms: what ln p's error moves, and each term's own rounding
    (a clipped one, too, is w times a bound times A)."""
    return sum(abs(a or 0) * e for a, e in zip(slope, err)) + abs(f) * float(np.abs(w * adv).sum()) * 2.0**-21


def policy_inputs(rng, lp, beta):
    """old, ref, advantages around log probabilities, away from the clipping
    range's ends."""
    n = len(lp)
    ratio = np.exp(0.3 * rng.normal(size=n))
    for end in (0.8, 1.25):
        ratio = np.where(np.abs(ratio - end) < 0.02, ratio + 0.05, ratio)
    old = (lp - np.log(ratio)).astype(np.float32)
    ref = (lp + 0.3 * rng.normal(size=n)).astype(np.float32)
    adv = rng.normal(size=n).astype(np.float32)
    return old, ref, np.where(np.abs(adv) < 0.1, np.float32(0.5), adv)


def check_policy(x, y, w, beta=0.1, mean=True, inv_t=1.0, pad=0, shift=0, in_place=False, seed=0):
    """One call on device logits x against the 64-bit form: stats, logp, every
    element of the gradient, and nothing written beside its rows."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    tokens, vocab = x.shape
    dtype, rng = x.dtype, np.random.default_rng(seed)
    t64 = float(np.float32(inv_t))
    live, _ = R.live_tokens(y, w, vocab)
    clean = host(torch.where(dev(live, torch.bool)[:, None], x, torch.zeros_like(x)))
    lp = R.logprobs(clean, y, t64, w)
    old, ref, adv = policy_inputs(rng, lp, beta)
    stats, lp, _, slope = R.policy(clean, y, old, adv, ref, w, 0.2, 0.25, beta, t64, 0.5, mean)
    op = PolicyLoss(tokens, vocab, dtype=dtype, clip_low=0.2, clip_high=0.25, kl_beta=beta,
                    inv_temperature=inv_t, scale=0.5, mean=mean)
    buf, g = (None, x) if in_place else nan_rows(tokens, vocab, dtype, pad, shift)
    out = op(x, dev(y, torch.int64), dev(old), dev(adv), ref_logp=dev(ref) if beta else None,
             weights=dev(w), grad=g)
    assert (np.abs(host(out[1]) - lp) <= logp_error(vocab, lp)).all()
    f = 0.5 / stats[3] if mean else 0.5
    err = policy_slope_error(lp, old, adv, ref, w, beta, f, slope, vocab)
    lim = policy_stats_error(w * live, adv, f, slope, err) + np.abs(stats) * 2.0**-20
    assert (np.abs(host(out[0]) - stats) <= lim).all()
    check_gradient(out[2], clean, y, slope, err, t64, dtype)
    if buf is not None:
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside.as_strided((tokens, vocab), g.stride(), shift)[:] = False
        assert bool(torch.isnan(buf[outside]).all())
    assert op.device_error() == 0


FAR = [-1e9, -1e6, 3e5, -1.3e5, 1.5e7, 1e8, 2.7e9, -1e20, 2000.0, -1400.0, 1500.0]


def far_rows(vocab, seed):
    """bf16 rows whose maximum is far from 0: every third word at the maximum,
    the others a step or more below it (a row of one value at the end)."""
    rng = np.random.default_rng(seed)
    x = np.empty((len(FAR) + 1, vocab), np.float32)
    for r, m in enumerate(FAR):
        x[r] = m - abs(m) * 2.0**-6 * rng.integers(0, 3, vocab)
        x[r, ::3] = m
    x[-1] = -1e9
    return torch.from_numpy(x).to("cuda", BF16)


# words: rows held by registers of 1 and 8 warps, the pipelined kernel, its ring
# with one row's share, and the gradient as a pass of its own
@pytest.mark.parametrize("vocab", [700, 9000, 32000, 420000, 800000])
def test_policy_gradient_of_rows_far_from_zero(vocab):
    x = far_rows(vocab, vocab)
    y = np.random.default_rng(1).integers(0, vocab, len(x))
    y[0] = 0  # (at the maximum)
    lp = R.logprobs(host(x), y)
    y = np.where(lp < -80, 3 * (y // 3), y)  # a probability that fp32 holds
    check_policy(x, y, np.linspace(0.5, 1.5, len(x)).astype(np.float32), pad=8)


@pytest.mark.parametrize("vocab", [700, 9000, 32000, 420000, 800000])
@pytest.mark.parametrize("inv_t", [1e3, 1e5])
def test_policy_gradient_at_small_temperatures(vocab, inv_t):
    """Ordinary logits near temperature 0: the words tied at the maximum (bf16
    has many) share the probability."""
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy((2.5 * rng.normal(size=(6, vocab))).astype(np.float32)).to("cuda", BF16)
    top = x.float().amax(1)
    for r, k in enumerate((1, 2, 3, 7, 64, 500)):
        x[r, torch.from_numpy(rng.choice(vocab, k, replace=False)).cuda()] = top[r].to(BF16)
    y = x.float().argmax(1).cpu().numpy()
    check_policy(x, y, np.ones(6, np.float32), inv_t=inv_t, pad=8)


@pytest.mark.parametrize("vocab", [700, 32000])
@pytest.mark.parametrize("inv_t", [1.0, 1e3])
def test_preference_gradient_of_rows_far_from_zero(vocab, inv_t):
    from fsdp_buffer_layout_gb300.objectives import PreferenceLoss
    x = far_rows(vocab, 5)
    if inv_t != 1.0:
        x[:] = torch.from_numpy(2.5 * np.random.default_rng(3).normal(size=tuple(x.shape)))
        x[:, ::3] = x.float().amax(1, keepdim=True).to(BF16)
    n = len(x)
    y = 3 * np.random.default_rng(2).integers(0, vocab // 3, n)  # at the maximum
    starts, t64 = [0, n // 2, n], float(np.float32(inv_t))
    buf, g = nan_rows(n, vocab, BF16, 8)
    out = PreferenceLoss(1, n, vocab, beta=0.1, inv_temperature=inv_t)(
        x, dev(y, torch.int64), dev(starts, torch.int64), grad=g)
    lp, slope = (R.preference(host(x), y, starts, None, None, "sigmoid", 0.1, 0.0, 0.0, False, t64, 1.0)[i] for i in (2, 4))
    assert (np.abs(host(out[2]) - lp) <= logp_error(vocab, lp)).all()
    # s(z) moves by at most beta d h relatively
    check_gradient(out[3], host(x), y, slope, [2.0**-20 + 0.1 * n * logp_error(vocab, lp).max()] * n,
                   t64, BF16)


@pytest.mark.parametrize("dtype,vocab", [(FP32, 50), (FP32, 1003), (BF16, 1003)])
def test_grad_attribute_is_the_last_calls_gradient(dtype, vocab):
    """The object's `grad` shows the rows of the last call whatever the logits'
    stride was."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss
    rng = np.random.default_rng(1)
    y = dev(rng.integers(0, vocab, 6), torch.int64)
    old, adv = dev(np.full(6, -5.0)), dev(rng.normal(size=6))
    starts = dev([0, 3, 6], torch.int64)
    op, pref = PolicyLoss(6, vocab, dtype=dtype), PreferenceLoss(1, 6, vocab, dtype=dtype)
    for pad in (0, 1, 2, 0, 5):
        x = torch.from_numpy(rng.normal(size=(6, vocab + pad)).astype(np.float32)).to("cuda", dtype)[:, :vocab]
        got = op(x, y, old, adv)[2]
        assert torch.equal(op.grad, got) and op.grad.data_ptr() == got.data_ptr()
        got = pref(x, y, starts)[3]
        assert torch.equal(pref.grad, got)


def test_buffers_belong_to_the_objects_stream():
    """Workspace and outputs come from the memory of the object's own stream, on
    which they are prepared, written and, at the end, given back: memory of the
    caller's stream could still be in use there."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss, Router, TokenLogprobs
    side = torch.cuda.Stream()
    ops = [TokenLogprobs(5, 100, stream=side), PolicyLoss(5, 100, stream=side),
           PreferenceLoss(1, 5, 100, stream=side), Router(5, 16, 2, stream=side)]
    x = torch.randn(5, 16, device="cuda", dtype=BF16)
    torch.cuda.synchronize()
    ops[3].forward(x)
    ops[3].backward(x)
    side.synchronize()
    segments = torch.cuda.memory_snapshot()
    for op in ops:
        held = [v for v in vars(op).values() if isinstance(v, torch.Tensor)]
        assert len(held) >= 2
        for v in held:
            at = v.untyped_storage().data_ptr()
            home = [s["stream"] for s in segments if s["address"] <= at < s["address"] + s["total_size"]]
            assert home == [side.cuda_stream], (type(op).__name__, tuple(v.shape))


def test_router_refuses_a_workspace_that_a_loss_has_used():
    """The losses leave their rows' sums where the router counts: a router call
    there says so in the error word and gives a loss of NaN; a fresh one does not,
    and losses may follow a router."""
    from fsdp_buffer_layout_gb300 import vsf as V
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss, Router
    rng = np.random.default_rng(3)
    x = dev(rng.normal(size=(64, 32)))
    lg = dev(rng.normal(size=(64, 700)))
    long = torch.full((2, 800000), -1.0, device="cuda", dtype=BF16)  # (the policy loss in three passes)
    y, zero = dev(rng.integers(0, 700, 64), torch.int64), dev(np.zeros(64))
    starts = dev([0, 32, 64], torch.int64)
    losses = [lambda: PolicyLoss(64, 700, dtype=FP32), lambda: PreferenceLoss(1, 64, 700, dtype=FP32),
              lambda: PolicyLoss(2, 800000)]

    def call(op):
        if op.tokens == 2:
            return op(long, y[:2], zero[:2], zero[:2])
        return op(lg, y, starts) if isinstance(op, PreferenceLoss) else op(lg, y, zero, zero)

    for sequences in (1, 80):  # (finished by the last CTA; by a launch of its own)
        cuts = dev([0] * sequences + [64], torch.int64)

        def route(r):
            return [t.clone() for t in r.forward(x, seq_starts=cuts)]

        fresh = Router(64, 32, 4, dtype=FP32, balance=0.1, sequences=sequences)
        want = route(fresh)
        assert all(torch.equal(a, b) for a, b in zip(route(fresh), want)) and fresh.device_error() == 0
        for make in losses:
            loss, router = make(), Router(64, 32, 4, dtype=FP32, balance=0.1, sequences=sequences)
            size = max(loss._ws_bytes, router._ws_bytes)
            both = torch.empty(size, dtype=torch.uint8, device="cuda")
            V.vsf_objective_workspace_init(both.data_ptr(), size, loss._st)
            for o in (loss, router):
                o.workspace, o._ws, o._ws_bytes = both, both.data_ptr(), size
            first = route(router)
            assert all(torch.equal(a, b) for a, b in zip(first, want)) and router.device_error() == 0
            got = [t.clone() for t in call(loss) if t is not None]
            alone = [t.clone() for t in call(make()) if t is not None]
            assert all(torch.equal(a, b) for a, b in zip(got, alone)) and loss.device_error() == 0
            assert math.isnan(route(router)[3].item()) and router.device_error() == 32
            V.vsf_objective_workspace_init(both.data_ptr(), size, loss._st)
            assert all(torch.equal(a, b) for a, b in zip(route(router), want)) and router.device_error() == 0


def test_router_backward_of_another_call():
    """The gradient is that of the last forward call: without one, for another
    number of tokens, or for a call that another has followed, it is refused."""
    from fsdp_buffer_layout_gb300.objectives import Router
    rng = np.random.default_rng(4)
    a, b = dev(rng.normal(size=(9, 12))), dev(rng.normal(size=(9, 12)))
    dg = dev(rng.normal(size=(9, 2)))
    op = Router(9, 12, 2, dtype=FP32, balance=0.1)
    with pytest.raises(ValueError):
        op.backward(a, dg)
    op.forward(a)
    first = op.calls
    want = op.backward(a, dg, call=first).clone()
    op.forward(b)
    assert op.calls != first
    with pytest.raises(ValueError):
        op.backward(a, dg, call=first)
    with pytest.raises(ValueError):
        op.backward(a[:5], dg[:5])
    op.backward(b, dg, call=op.calls)
    op.forward(a)  # computed again
    assert torch.equal(op.backward(a, dg, call=op.calls), want)
    with pytest.raises(ValueError):
        op.forward(a.bfloat16())
    assert torch.equal(op.backward(a, dg, call=op.calls), want)  # a refused call leaves the last one


def test_longest_row():
    """Rows of 2^31 - 1 words, the most: a few likely words at both ends and in
    between, the others -inf; a masked row."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, TokenLogprobs
    vocab, ld = (1 << 31) - 1, 1 << 31
    buf = torch.full((3 + 2 * ld,), -math.inf, dtype=BF16, device="cuda")
    x = buf.as_strided((2, vocab), (ld, 1), 3)
    words = [0, 1, 4, 5, 1 << 20, (1 << 30) + 7, vocab - 9, vocab - 8, vocab - 2, vocab - 1]
    at = dev(words, torch.int64)
    z = np.arange(10) * 0.25
    x[1, at] = dev(z).to(BF16)
    p = np.exp(z) / np.exp(z).sum()
    y = dev([-1, vocab - 1], torch.int64)
    logp = TokenLogprobs(2, vocab)(x, y)
    assert logp[0].item() == 0 and abs(logp[1].item() - math.log(p[-1])) <= 2.0**-20
    out = torch.full((3 + 2 * ld,), math.nan, dtype=BF16, device="cuda")
    g = out.as_strided((2, vocab), (ld, 1), 3)
    op = PolicyLoss(2, vocab, with_grad=False)
    op(x, y, logp, dev([1.0, 1.0]), grad=g)
    assert op.device_error() == 0
    want = p.copy()
    want[-1] -= 1.0  # d loss / d x = p - 1[v = y]
    assert (np.abs(host(g[1, at]) - want) <= 2.0**-8 * np.abs(want)).all()
    assert torch.count_nonzero(g[0]).item() == 0
    assert torch.count_nonzero(g[1]).item() == 10  # (NaN would count)
    assert torch.isnan(out[:3]).all() and torch.isnan(out[3 + vocab:3 + ld]).all() and torch.isnan(out[3 + ld + vocab:]).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [700, 33000, 800000])
@pytest.mark.parametrize("inv_t", [2.0**127, 1e30, 1e-30, 2.0**-126, 3e-39, 2e-45])
def test_temperatures_at_the_ends_of_their_range(dtype, vocab, inv_t):
    """Near temperature 0 the probability lies on the largest logits, at a very
    large one on all but the -inf words alike."""
    from fsdp_buffer_layout_gb300.objectives import TokenLogprobs
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.integers(-9, 3, (4, vocab)).astype(np.float32)).to("cuda", dtype)
    x[:, 1::2] = -math.inf
    x[:, 0::64] = 4.0
    y = np.full(4, 64)
    lp = TokenLogprobs(4, vocab, dtype=dtype, inv_temperature=inv_t)(x, dev(y, torch.int64))
    want = R.logprobs(host(x), y, float(np.float32(inv_t)))
    assert (np.abs(host(lp) - want) <= logp_error(vocab, want)).all()
    # (a gradient of 2^-30 / temperature, so that it fits; far below fp32 it is 0)
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    op = PolicyLoss(4, vocab, dtype=dtype, inv_temperature=inv_t, scale=2.0**-30 if inv_t > 1 else 1.0, mean=False)
    g = op(x, dev(y, torch.int64), lp.clone(), dev(np.ones(4)))[2]
    assert torch.isfinite(g).all() and not g[:, 1::2].any()
    if inv_t >= 1e-30:
        t64 = float(np.float32(inv_t))
        scale = 2.0**-30 if inv_t > 1 else 1.0
        check_gradient(g, host(x), y, [-scale] * 4, [2.0**-19 + tol(vocab)] * 4, t64, dtype)


@pytest.mark.parametrize("vocab", [700, 33000, 800000])
def test_advantage_zero_where_the_ratio_overflows(vocab):
    """r A is 0 for A = 0 however far the policy has moved (exp(logp - old) is
    past fp32 above 88); an advantage above 0 is clipped there."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.normal(size=(3, vocab)).astype(np.float32)).to("cuda", BF16)
    y = rng.integers(0, vocab, 3)
    old = np.array([-200, -5, -120], np.float32)
    adv = np.array([0, 0.5, 2], np.float32)
    stats, lp, grad = PolicyLoss(3, vocab, mean=False)(x, dev(y, torch.int64), dev(old), dev(adv))
    s, l, g, _ = R.policy(host(x), y, old, adv, old, None, 0.2, 0.2, 0.0, 1.0, 1.0, False)
    assert (np.abs(host(stats) - s) <= 1e-4 * np.abs(s)).all()
    assert not grad[0].any() and not grad[2].any() and torch.isfinite(grad).all()


@pytest.mark.parametrize("device", ["cpu", "cuda:1", torch.device("meta")])
def test_objects_are_made_on_the_current_device(device):
    """Their calls launch on it; another one is refused when the object is made,
    not at its first call."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, PreferenceLoss, Router, TokenLogprobs
    for make in (lambda d: TokenLogprobs(4, 64, device=d), lambda d: PolicyLoss(4, 64, device=d),
                 lambda d: PreferenceLoss(1, 4, 64, device=d), lambda d: Router(4, 8, 2, device=d)):
        with pytest.raises(ValueError):
            make(device)
        assert make("cuda").device == make(torch.device("cuda", 0)).device == torch.device("cuda", 0)


def likely(rng, tokens, vocab, dtype, pad=0, shift=0):
    """Rows whose ends hold likely words, so that a word left out shows."""
    ld = vocab + pad
    buf = torch.empty(shift + tokens * ld + 16, dtype=dtype, device="cuda")
    buf.copy_(torch.from_numpy((2.5 * rng.normal(size=buf.numel())).astype(np.float32)))
    x = buf.as_strided((tokens, vocab), (ld, 1), shift)
    ends = sorted({v % vocab for v in (*range(9), *range(-9, 0), vocab // 2, vocab // 3)})
    x[:, ends] += 6.0
    return x


STRICT = [  # tokens, vocab, dtype, logits' pad and shift, gradient's pad and shift
    (3, 2, FP32, 0, 0, 3, 1), (5, 31, BF16, 2, 1, 2, 1), (9, 257, BF16, 0, 0, 3, 5),
    (6, 1003, FP32, 1, 1, 1, 1), (9, 2048, BF16, 0, 0, 8, 0), (7, 4099, BF16, 0, 3, 5, 2),
    (5, 9001, FP32, 0, 0, 0, 0), (6, 16384, BF16, 8, 0, 0, 0), (5, 16391, BF16, 1, 7, 1, 7),
    (170, 20000, BF16, 0, 0, 8, 0), (5, 50021, FP32, 3, 2, 3, 2), (5, 65537, BF16, 0, 0, 7, 0),
    (4, 131075, FP32, 5, 2, 5, 2), (5, 300001, BF16, 0, 1, 0, 1),
    # one row's share in the ring: few rows; more rows than clusters; odd places
    (5, 500000, BF16, 0, 0, 8, 0), (45, 400003, BF16, 5, 3, 5, 3), (5, 200000, FP32, 0, 0, 4, 0),
    (41, 201089, FP32, 0, 0, 1, 1),
    # gradient as a pass of its own
    (5, 800000, BF16, 0, 0, 8, 0), (5, 790003, BF16, 1, 3, 2, 5), (4, 400009, FP32, 3, 1, 3, 1),
]


@pytest.mark.parametrize("tokens,vocab,dtype,pad,shift,gpad,gshift", STRICT)
@pytest.mark.parametrize("beta,mean", [(0.1, True), (0.0, False)])
def test_every_element_of_the_policy_gradient(tokens, vocab, dtype, pad, shift, gpad, gshift, beta, mean):
    rng = np.random.default_rng(vocab)
    x = likely(rng, tokens, vocab, dtype, pad, shift)
    y = rng.integers(0, vocab, tokens)
    w = rng.uniform(0.5, 1.5, tokens).astype(np.float32)
    y[0], y[1] = 0, vocab - 1
    if tokens > 3:
        y[2], w[3] = -1, 0.0
        x[2:4] = math.nan
    check_policy(x, y, w, beta, mean, 1.0 if mean else 1.25, gpad, gshift, seed=vocab)
    check_policy(x, y, w, beta, mean, 1.0, in_place=True, seed=vocab)


@pytest.mark.parametrize("tokens", [2049, 8192, 8193, 70000])
@pytest.mark.parametrize("mean", [True, False])
def test_policy_loss_of_many_short_rows(tokens, mean):
    """The sum of the weights by one CTA, by several (the last adds up), by the
    most there are."""
    rng = np.random.default_rng(tokens)
    x = likely(rng, tokens, 40, BF16)
    y = rng.integers(0, 40, tokens)
    w = rng.uniform(0.5, 1.5, tokens).astype(np.float32)
    y[rng.random(tokens) < 0.2], w[rng.random(tokens) < 0.2] = -1, 0.0
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss
    lp = R.logprobs(host(x), y, 1.0, w)
    old, ref, adv = policy_inputs(rng, lp, 0.1)
    s, _, g, slope = R.policy(host(x), y, old, adv, ref, w, 0.2, 0.25, 0.1, 1.0, 0.5, mean)
    err = policy_slope_error(lp, old, adv, ref, w, 0.1, 0.5 / (s[3] if mean else 1), slope, 40)
    op = PolicyLoss(tokens, 40, clip_low=0.2, clip_high=0.25, kl_beta=0.1, scale=0.5, mean=mean)
    args = (x, dev(y, torch.int64), dev(old), dev(adv), dev(ref), dev(w))
    for _ in range(2):
        stats, _, grad = op(*args)
        lim = policy_stats_error(w * (y >= 0), adv, 0.5 / (s[3] if mean else 1), slope, err)
        assert (np.abs(host(stats) - s) <= lim + 2.0**-20 * np.abs(s)).all()
        a = np.array([v or 0.0 for v in slope])
        p = np.exp(R.log_softmax(host(x)))
        one = np.arange(40) == y[:, None]
        lim = np.abs(a[:, None]) * ((np.array(err)[:, None] + 2 * tol(40) + 2.0**-14 + 2.0**-8) * np.where(one, 1 - p, p)
                                    + one * (np.array(err)[:, None] + 2.0**-14 * p)) + 1e-30
        assert (np.abs(host(grad) - g) <= lim).all()


@pytest.mark.parametrize("keep", [400, 0])
def test_many_more_long_rows_than_a_list_holds(keep):
    """157,000 rows of 16,400 words, nearly all of them masked (NaN): clusters
    take rows as they come."""
    from fsdp_buffer_layout_gb300.objectives import PolicyLoss, TokenLogprobs
    tokens, vocab = 157000, 16400
    rng = np.random.default_rng(6)
    at = np.sort(rng.choice(tokens, keep, replace=False)) if keep else np.arange(0)
    x = torch.full((tokens, vocab), math.nan, dtype=BF16, device="cuda")
    rows = dev(at, torch.int64)
    part = likely(rng, max(keep, 1), vocab, BF16)[:keep]
    x[rows] = part
    y, old, adv = np.full(tokens, -1), np.zeros(tokens, np.float32), np.zeros(tokens, np.float32)
    yk = rng.integers(0, vocab, keep)
    y[at] = yk
    lp = R.logprobs(host(part), yk)
    ok, _, ak = policy_inputs(rng, lp, 0.0)
    old[at], adv[at] = ok, ak
    yt = dev(y, torch.int64)
    got = TokenLogprobs(tokens, vocab)(x, yt)
    assert (np.abs(host(got[rows]) - lp) <= logp_error(vocab, lp)).all()
    assert torch.count_nonzero(got).item() == np.count_nonzero(lp)
    op = PolicyLoss(tokens, vocab, clip_low=0.2, clip_high=0.25)
    stats, logp, grad = op(x, yt, dev(old), dev(adv))
    if not keep:
        assert not stats.any() and not logp.any() and torch.count_nonzero(grad).item() == 0
        return
    s, _, _, slope = R.policy(host(part), yk, ok, ak, ok, None, 0.2, 0.25, 0.0, 1.0, 1.0, True)
    err = policy_slope_error(lp, ok, ak, ok, np.ones(keep), 0.0, 1 / keep, slope, vocab)
    lim = policy_stats_error(1.0, ak, 1 / keep, slope, err) + 2.0**-20 * abs(s[0])
    assert abs(stats[0].item() - s[0]) <= lim
    assert stats[3].item() == keep
    check_gradient(grad[rows], host(part), yk, slope, err, 1.0, BF16)
    grad[rows] = 0
    assert torch.count_nonzero(grad).item() == 0
    assert op.device_error() == 0


@pytest.mark.parametrize("vocab,dtype,pad,lengths", [
    (90, BF16, 0, (4100, 3999)), (301, FP32, 1, (1030, 0, 5, 2500)), (16500, BF16, 3, (30, 41, 0, 77)),
    (70001, FP32, 0, (3, 4)), (200000, BF16, 8, (2, 1)),
])
def test_every_element_of_the_preference_gradient(vocab, dtype, pad, lengths):
    """Sequences of some thousand tokens among them."""
    from fsdp_buffer_layout_gb300.objectives import PreferenceLoss
    rng = np.random.default_rng(vocab)
    starts = np.cumsum([0] + list(lengths)) + 2
    n = int(starts[-1]) + 3
    x = likely(rng, n, vocab, dtype, pad)
    y = rng.integers(0, vocab, n)
    y[5::7] = -1
    live = y >= 0
    lp = R.logprobs(host(x), y)
    ref = (lp + rng.normal(size=n) * 0.2 / math.sqrt(n)).astype(np.float32)
    out = R.preference(host(x), y, starts, ref, None, "sigmoid", 0.3, 0.1, 0.2, False, 1.0, 0.5)
    buf, g = nan_rows(n, vocab, dtype, 5)
    op = PreferenceLoss(len(lengths) // 2, n, vocab, dtype=dtype, beta=0.3, smoothing=0.1, margin=0.2, scale=0.5)
    stats, rewards, logp, grad = op(x, dev(y, torch.int64), dev(starts, torch.int64), ref_logp=dev(ref), grad=g)
    assert (np.abs(host(logp) - lp) <= logp_error(vocab, lp)).all()
    # a pair's sum: each token's ln p, and fp32 additions of small differences
    each = np.array([live[a:b].sum() for a, b in zip(starts, starts[1:])]) * (tol(vocab) + 2.0**-20)
    assert (np.abs(host(rewards) - out[1]) <= 0.3 * each + 2.0**-22 * np.abs(out[1])).all()
    dh = each[:len(each) // 2] + each[len(each) // 2:]
    assert (np.abs(host(stats) - out[0]) <= 0.3 * dh.max() + 2.0**-20 * np.abs(out[0])).all()
    slope = out[4]
    # d loss / d h moves by at most beta^2 / 4 d h
    err = [0.0] * n
    for s in range(len(lengths)):
        for t in range(starts[s], starts[s + 1]):
            if slope[t]:
                err[t] = 2.0**-20 + 0.5 / (len(lengths) // 2) * 0.09 / 4 * dh[s % len(dh)] / abs(slope[t])
    check_gradient(grad, host(x), y, slope, err, 1.0, dtype)
    outside = torch.ones_like(buf, dtype=torch.bool)
    outside.as_strided((n, vocab), g.stride(), 0)[:] = False
    assert bool(torch.isnan(buf[outside]).all()) and op.device_error() == 0


def route_gate_error(x, idx, score, renorm, experts):
    """Relative error of each gate. A softmax term 2^t, t = (x - m) log2(e), is
    within 2^-22 (ex2.approx) plus 3 |t| 2^-24 ln 2 (difference, constant and
    product) of its value, a sigmoid within e / (1 + e) of the same for e =
    exp(-x), plus 2^-23 each for its sum and its reciprocal (rcp.approx). Sums
    have at most 21 additions (16 in a lane, 5 by shuffles); one division."""
    t = (x - x.max(1, keepdims=True) if score == "softmax" else -x) / LN2
    term = 2.0**-22 + 3 * np.abs(t) * 2.0**-24 * LN2
    if score == "sigmoid":
        e = np.exp(np.minimum(-x, 700))
        term = term * (e / (1 + e)) + 2.0**-22
    own = np.take_along_axis(term, idx, 1)
    if renorm:
        return own + own.max(1, keepdims=True) + 21 * 2.0**-24 + 2.0**-21
    if score == "sigmoid":
        return own + 2.0**-23
    # the sum's error is its terms', weighted: |t| is at most log2 E there
    return own + 2.0**-22 + 3 * math.log2(2 * experts) * 2.0**-24 + 21 * 2.0**-24 + 2.0**-22


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("experts,k", [(8, 2), (64, 8), (100, 6), (256, 8), (512, 32)])
@pytest.mark.parametrize("offset,spread", [(0.0, 12.0), (1e4, 8.0), (-60.0, 4.0)])
def test_gates_of_spread_and_shifted_logits(experts, k, dtype, score, renorm, offset, spread):
    """Logits of a wide spread, and all of them far from 0."""
    from fsdp_buffer_layout_gb300.objectives import Router
    rng = np.random.default_rng(experts + k)
    x = dev((offset + spread * rng.normal(size=(200, experts))), dtype)
    idx, gates, _, _ = Router(200, experts, k, dtype=dtype, score=score, renorm=renorm).forward(x)
    i, g, *_ = R.route(host(x), k, score, renorm, 1.0, 0.0)
    assert np.array_equal(idx.cpu().numpy(), i)
    lim = route_gate_error(host(x), i, score, renorm, experts) * np.abs(g) + 2.0**-125
    assert (np.abs(host(gates) - g) <= lim).all(), (np.abs(host(gates) - g) / lim).max()
