"""Token scores on the GPU against the 64-bit reference.

Tolerances. A term e = exp(z) is within 2^-22 (ex2.approx) plus |z| 2^-22 (its
argument: three roundings) of its value; a thread adds at most V / 256 + 40 of
them, 2^-24 each, and joins keep that. So a row's sum is within `tol`, relative,
and u / s, the mean of z, within (tol + 2^-22) E|z| + 2^-22 E z^2. ln p and the
entropy add their own roundings, 2^-23 of what they are made of. A gradient
element is a sum of p times pulls and of pulls of its own; each product is
within the error of p (2 tol, 2^-21 and |z| 2^-22) and of its factors; half a step
of the output's type comes on top. Indexes are exact.
"""
import math

import numpy as np
import pytest
import torch

import score_reference as R

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0**-8, FP32: 2.0**-24}


def host(x):
    return x.double().cpu().numpy()


def dev(a, dtype=torch.float32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def tol(vocab):
    return 2.0**-21 + (math.log2(vocab) + 1) * 2.0**-22 + (vocab / 256 + 40) * 2.0**-24


def moments(row, inv_t):
    z, p, lp = R.parts(row, inv_t)
    z = np.where(p > 0, z, 0.0)
    return z, p, np.abs(p * z).sum(), (p * z * z).sum()


def strided(values, dtype, pad=0, shift=0):
    t, v = values.shape
    buf = torch.full((shift + t * (v + pad) + 8,), math.nan, dtype=dtype, device="cuda")
    x = buf.as_strided((t, v), (v + pad, 1), shift)
    x.copy_(torch.from_numpy(values.astype(np.float32)))
    return x


def check(x, y, inv_t, k, got):
    """The four outputs of a forward call on rows without NaN."""
    xs, vocab = host(x), x.shape[1]
    y = np.where(y < vocab, y, -1)
    logp, entropy, idx, top_logp = R.scores(xs, y, inv_t, k)
    assert np.array_equal(host(got[2]), idx)
    lim = tol(vocab) + 2.0**-22 * (np.abs(logp) + math.log(vocab) + 1)
    assert (np.abs(host(got[0]) - logp) <= lim).all(), np.abs(host(got[0]) - logp).max()
    lim = tol(vocab) + 2.0**-22 * (np.abs(top_logp) + math.log(vocab) + 1)
    with np.errstate(invalid="ignore"):
        off = np.abs(host(got[3]) - top_logp)
    assert (np.where(np.isinf(top_logp), host(got[3]) == top_logp, off <= lim)).all()
    for i in np.flatnonzero(y >= 0):
        _, _, az, zz = moments(xs[i], inv_t)
        lim = tol(vocab) * (1 + az) + 2.0**-22 * (zz + az + math.log(vocab) + 1)
        assert abs(host(got[1])[i] - entropy[i]) <= lim, (i, host(got[1])[i], entropy[i])
    assert not host(got[1])[y < 0].any()
    return idx


def check_grad(x, y, inv_t, idx, pulls, got, dtype):
    xs, vocab = host(x), x.shape[1]
    d_logp, d_entropy, d_top = pulls
    want = R.gradient(xs, y, inv_t, idx, *pulls)
    got = host(got)
    assert np.isfinite(got).all()
    for i in range(len(y)):
        if y[i] < 0:
            assert not got[i].any()
            continue
        z, p, az, zz = moments(xs[i], inv_t)
        own = np.zeros(vocab)
        own[y[i]] += abs(d_logp[i])
        for j, v in enumerate(idx[i]):
            if 0 <= v < vocab:
                own[v] += abs(d_top[i, j])
        pull = abs(d_logp[i]) + np.abs(d_top[i]).sum()
        h = abs(d_entropy[i])
        rel = 2 * tol(vocab) + 2.0**-20 + np.abs(z) * 2.0**-21
        mean = tol(vocab) * (1 + az) + 2.0**-22 * (zz + az + 1)
        lim = p * (rel * (pull + h * (np.abs(z) + az)) + h * mean) + 2.0**-22 * own
        lim = inv_t * lim * 1.01 + HALF[dtype] * np.abs(want[i]) + 1e-37
        off = np.abs(got[i] - want[i])
        assert (off <= lim).all(), (i, (off / lim).max(), int((off / lim).argmax()))


SHAPES = [  # tokens, vocab, dtype, k, pad, shift
    (1, 1, BF16, 1, 0, 0), (3, 2, FP32, 2, 0, 0), (5, 31, BF16, 31, 2, 1), (1, 1000, FP32, 4, 0, 3),
    (7, 257, BF16, 0, 0, 0), (17, 4096, BF16, 5, 0, 0), (9, 5003, FP32, 32, 1, 1),
    (4, 32000, BF16, 20, 0, 0), (3, 32000, FP32, 8, 0, 0), (6, 50021, BF16, 7, 3, 5),
    (3, 65537, FP32, 32, 2, 1), (2, 131072, BF16, 20, 0, 0), (2, 131075, FP32, 3, 5, 2),
    (2, 300001, BF16, 9, 0, 0), (2, 1200003, FP32, 5, 1, 0), (200, 640, BF16, 3, 0, 0),
    (700, 96, FP32, 2, 0, 0), (40, 20000, BF16, 6, 1, 0),
]


def make(rng, tokens, vocab, dtype, pad, shift):
    x = strided(rng.normal(size=(tokens, vocab)) * 2.5, dtype, pad, shift)
    ends = sorted({v % vocab for v in (0, 1, 7, 8, -1, -2, -9, vocab // 2)})
    x[:, ends] += 5.0  # likely words where vectors begin and end
    y = rng.integers(0, vocab, tokens)
    if tokens > 2:
        y[1] = -100
    return x, y


@pytest.mark.parametrize("tokens,vocab,dtype,k,pad,shift", SHAPES)
@pytest.mark.parametrize("inv_t,in_place", [(1.0, False), (1.25, True)])
def test_scores_and_gradient(tokens, vocab, dtype, k, pad, shift, inv_t, in_place):
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    rng = np.random.default_rng(vocab + k)
    x, y = make(rng, tokens, vocab, dtype, pad, shift)
    op = TokenScores(tokens, vocab, top_k=k, dtype=dtype, inv_temperature=inv_t)
    got = op.forward(x, dev(y, torch.int64))
    inv_t = float(np.float32(inv_t))
    idx = check(x, y, inv_t, k, got)
    assert op.device_error() == 0
    if tokens > 3 and k > 1:
        y[3] = idx[3, 1]  # a target that is one of the alternatives
    pulls = [rng.normal(size=s).astype(np.float32) for s in (tokens, tokens, (tokens, k))]
    args = [dev(p) for p in pulls]
    before = x.clone()
    out = op.backward(x, dev(y, torch.int64), *args, grad=x if in_place else None)
    check_grad(before, y, inv_t, idx, [p.astype(np.float64) for p in pulls], out, dtype)
    # each pull alone, the others not given
    if not in_place:
        for which in range(3):
            one = [p if i == which else None for i, p in enumerate(args)]
            zero = [p if i == which else np.zeros_like(p) for i, p in enumerate(pulls)]
            out = op.backward(x, dev(y, torch.int64), *one)
            check_grad(before, y, inv_t, idx, [p.astype(np.float64) for p in zero], out, dtype)
        assert not op.backward(x, dev(y, torch.int64)).any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [40, 3000, 70003])
def test_ties(dtype, vocab):
    """Equal logits, in long runs and all over: the lowest indexes; -0 and 0 are equal."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    rng = np.random.default_rng(vocab)
    v = np.stack([np.zeros(vocab), np.where(np.arange(vocab) % 2, 0.0, -0.0), rng.integers(0, 3, vocab),
                  np.arange(vocab)[::-1] // 9, -np.arange(vocab) // 300 * 1.0,
                  np.where(np.arange(vocab) < vocab - 3, 1.0, 1.0), rng.integers(-2, 2, vocab) * 1e-38])
    v[1, ::7] = 1.0
    v = np.concatenate([v, np.arange(vocab)[None] % 250 * 0.5, np.arange(vocab)[None] // 300 * 0.25])
    x = strided(v, dtype, pad=1, shift=3)
    y = np.zeros(len(v), np.int64)
    for k in (1, 5, 32):
        check(x, y, 1.0, k, TokenScores(len(v), vocab, top_k=k, dtype=dtype).forward(x, dev(y, torch.int64)))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [50, 5000, 140001])
def test_masked_words(dtype, vocab):
    """Words masked with -inf or the type's lowest value: fewer finite ones than
    alternatives, runs at the row's start, a row of the lowest value alone."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    rng = np.random.default_rng(vocab)
    low = torch.finfo(dtype).min
    v = rng.normal(size=(6, vocab)) * 2
    v[0, 3:] = -np.inf
    v[1, : vocab - 2] = -np.inf
    v[2, 1::2] = -np.inf
    v[3, 5:] = low
    v[4, :] = low
    v[5, : vocab // 2] = low
    v[5, vocab // 2 + 1:: 3] = -np.inf
    x = strided(v, dtype)
    y = np.array([1, vocab - 1, 2, 0, vocab // 3, vocab - 1])
    y[5] = vocab // 2  # (finite)
    k = 8
    op = TokenScores(6, vocab, top_k=k, dtype=dtype)
    got = op.forward(x, dev(y, torch.int64))
    idx = check(x, y, 1.0, k, got)
    pulls = [rng.normal(size=s) for s in (6, 6, (6, k))]
    pulls[2][~np.isfinite(np.take_along_axis(v, idx, 1))] = 0.0
    pulls = [p.astype(np.float32) for p in pulls]
    out = op.backward(x, dev(y, torch.int64), *[dev(p) for p in pulls])
    check_grad(x, y, 1.0, idx, [p.astype(np.float64) for p in pulls], out, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("inv_t", [1.0, 100.0])
@pytest.mark.parametrize("vocab", [60, 9000])
def test_logits_at_the_ends_of_their_range(vocab, inv_t, dtype):
    """The lowest value beside -inf and nothing else; neighbours of a large value;
    both ends of the range in one row; ones next to a far smaller maximum."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    top, rng = torch.finfo(dtype).max, np.random.default_rng(vocab)
    half = np.arange(vocab) % 2 == 0
    v = np.stack([np.where(half, -top, -np.inf), np.where(half, 2.0**30, 2.0**30 * (1 - 2.0**-8)),
                  np.where(half, top, -top), np.where(np.arange(vocab) < vocab - 1, -np.inf, -top),
                  rng.normal(size=vocab) - 2.0**100, np.where(half, -200.0, -330.0)])
    x = strided(v, dtype)
    y = np.array([0, 2, 2, vocab - 1, 4, 6])
    got = TokenScores(6, vocab, top_k=3, dtype=dtype, inv_temperature=inv_t).forward(x, dev(y, torch.int64))
    check(x, y, inv_t, 3, got)


@pytest.mark.parametrize("vocab", [30, 6001])
def test_rows_that_give_nan(vocab):
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    x = torch.randn(5, vocab, device="cuda")
    x[0, vocab // 2] = math.nan
    x[1, 3] = math.inf
    x[2] = -math.inf
    x[3] = math.nan  # (masked)
    y = dev([1, 2, 3, -1, 4], torch.int64)
    op = TokenScores(5, vocab, top_k=3, dtype=FP32)
    logp, entropy, idx, top_logp = op.forward(x, y)
    for out in (logp, entropy, top_logp):
        assert torch.isnan(out[:3]).all() and torch.isfinite(out[3:]).all()
    assert (idx[:4] == -1).all() and (idx[4] >= 0).all() and not logp[3] and not top_logp[3].any()
    one = torch.ones(5, device="cuda")
    g = op.backward(x, y, one, one, torch.ones(5, 3, device="cuda"))
    assert torch.isnan(g[:3]).any(1).all() and not g[3].any() and torch.isfinite(g[4]).all()


@pytest.mark.parametrize("inv_t", [2.0**127, 1e30, 1e-30, 2.0**-126, 2e-45])
@pytest.mark.parametrize("vocab", [700, 33000])
def test_temperatures_at_the_ends_of_their_range(vocab, inv_t):
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    rng = np.random.default_rng(vocab)
    v = rng.integers(-9, 3, (3, vocab)).astype(float)
    v[:, 1::2] = -np.inf
    v[:, 0::64] = 4.0
    x, y = strided(v, BF16), np.full(3, 64)
    t32 = float(np.float32(inv_t))
    op = TokenScores(3, vocab, top_k=4, inv_temperature=inv_t)
    check(x, y, t32, 4, op.forward(x, dev(y, torch.int64)))
    if 1e-30 <= inv_t <= 1e30:
        pulls = [np.full(s, 2.0**-40 if inv_t > 1 else 1.0) for s in (3, 3, (3, 4))]
        idx = R.scores(v, y, t32, 4)[2]
        out = op.backward(x, dev(y, torch.int64), *[dev(p) for p in pulls])
        want = R.gradient(v, y, t32, idx, *pulls)
        assert torch.isfinite(out).all()
        assert (np.abs(host(out) - want) <= (2.0**-7) * np.abs(want) + 2.0**-18 * t32 * pulls[0][0]).all()


@pytest.mark.parametrize("vocab", [40000, 131076])
def test_reference_of_the_exponents(vocab):
    """The exponents' reference lies at most 16 units of ln 2 below the row's maximum,
    also where 16 units are no number of the logits' type: next to 2^27, whose neighbours
    are 16 apart, 30 units at this temperature. Every lane begins at the lower one."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    inv_t, n = 1.3, np.arange(vocab)
    v = np.where(n // 128 % 16 < 4, 2.0**27, 2.0**27 + 16)[None].repeat(3, 0)
    v[1, -1] = 2.0**27 - 8
    v[2, n // 128 % 16 == 5] = 2.0**27 + 32
    x, y = strided(v, FP32), np.array([5, vocab - 1, vocab // 2])
    op = TokenScores(3, vocab, top_k=2, dtype=FP32, inv_temperature=inv_t)
    check(x, y, float(np.float32(inv_t)), 2, op.forward(x, dev(y, torch.int64)))
    norm = host(op.norm)
    above = (v.max(1) - norm[:, 0]) * inv_t / math.log(2)
    # (0.08 and 200 / c are within 2^-23 of what they stand for)
    assert (above >= 0).all() and (above <= 16 * (1 + 2.0**-20)).all(), above
    assert (norm[:, 1] <= vocab * 2.0**16 * (1 + 2.0**-10)).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [9000, 40000, 131075])
def test_far_logits_at_a_high_temperature(vocab, dtype):
    """Logits whose difference is out of range, low ones first in every lane, at a
    temperature that leaves them 60 apart."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    n = np.arange(vocab)
    span = 32 * 16 // dtype.itemsize
    v = np.where(n // span % 16 < 4, -3e38, 3e38)[None].repeat(2, 0)
    v[1] *= -1
    x = strided(v, dtype)
    y = np.array([5 * span, 1])
    for inv_t in (1e-37, 3e-37):
        op = TokenScores(2, vocab, top_k=3, dtype=dtype, inv_temperature=inv_t)
        got = op.forward(x, dev(y, torch.int64))
        check(x, y, float(np.float32(inv_t)), 3, got)
        pulls = [np.ones(s, np.float32) for s in (2, 2, (2, 3))]
        out = op.backward(x, dev(y, torch.int64), *[dev(p) for p in pulls])
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tokens,vocab", [(120, 70003), (220, 5000), (220, 300), (400, 5000), (400, 70003), (600, 5000),
                                          (500, 30001), (1000, 900), (3, 150001)])
@pytest.mark.parametrize("inv_t,k", [(1.0, 8), (1e30, 3), (1.0, 32)])
def test_edge_rows_in_calls_of_any_size(tokens, vocab, dtype, inv_t, k):
    """Ties, masked words and rows that give NaN, some of each left out, however a
    call's rows are shared out."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    rng = np.random.default_rng(vocab)
    low, n = torch.finfo(dtype).min, np.arange(vocab)
    v = np.stack([np.zeros(vocab), rng.integers(0, 3, vocab), n[::-1] // 99, np.where(n % 250 == 249, 4.0, -np.inf),
                  np.where(n < 5, 2.0, -np.inf), np.where(n < 5, 2.0, low), np.where(n == vocab - 1, -1.0, -np.inf),
                  np.full(vocab, low), n % 128 * 0.5, n // 300 % 4 * 0.25, np.full(vocab, -np.inf)])
    sound = len(v) - 1
    which = np.arange(tokens) % len(v)
    x, y = strided(v[which], dtype, pad=1, shift=2), np.where(which == 6, vocab - 1, np.where(which == 3, 249, 2))
    y[which == 7] = np.where(np.arange(tokens)[which == 7] % 2, -1, 2)
    op = TokenScores(tokens, vocab, top_k=k, dtype=dtype, inv_temperature=inv_t)
    got = op.forward(x, dev(y, torch.int64))
    assert op.device_error() == 0
    inv_t = float(np.float32(inv_t))
    for i in {0, tokens // len(v) // 2 * len(v), (tokens - 1) // len(v) * len(v)}:
        rows = slice(i, min(i + sound, tokens))
        check(x[rows], y[rows], inv_t, k, [o[rows] for o in got])
    same = torch.from_numpy(which + len(v) * (y < 0))
    for w in same.unique():
        idx = got[2].cpu()[same == w]
        assert (idx == idx[0]).all()
    nan = torch.from_numpy(which == sound).cuda()
    for o in (got[0], got[1], got[3]):
        assert torch.isnan(o[nan]).all() and not torch.isnan(o[~nan]).any()
    assert (got[2][nan] == -1).all()


def test_targets_and_words_out_of_range():
    """A target >= V is left out and reported; words out of range, and a word
    twice, in what backward is given."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    rng = np.random.default_rng(1)
    vocab, k = 2000, 4
    x, y = strided(rng.normal(size=(4, vocab)) * 2, FP32), np.array([5, vocab, 7, 1 << 40])
    op = TokenScores(4, vocab, top_k=k, dtype=FP32)
    check(x, y, 1.0, k, op.forward(x, dev(y, torch.int64)))
    assert op.device_error() == 16
    op.top_idx[0] = dev([-1, vocab, 1 << 30, 5], torch.int32)
    op.top_idx[2] = dev([9, 9, 7, 9], torch.int32)
    pulls = [rng.normal(size=s).astype(np.float32) for s in (4, 4, (4, k))]
    out = op.backward(x, dev(y, torch.int64), *[dev(p) for p in pulls])
    check_grad(x, np.where(y < vocab, y, -1), 1.0, host(op.top_idx).astype(np.int64),
               [p.astype(np.float64) for p in pulls], out, FP32)


@pytest.mark.parametrize("dtype,vocab,pad,shift", [
    (BF16, 4099, 0, 3), (BF16, 16384, 8, 0), (FP32, 9001, 0, 0), (BF16, 33, 3, 1), (FP32, 1003, 3, 2)])
def test_gradient_stays_inside_its_rows(dtype, vocab, pad, shift):
    """What lies between and around the gradient's rows keeps its NaN, wherever
    the rows start against the logits'."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    rng = np.random.default_rng(vocab)
    x, y = make(rng, 5, vocab, dtype, pad, shift)
    op = TokenScores(5, vocab, top_k=3, dtype=dtype, with_grad=False)
    idx = host(op.forward(x, dev(y, torch.int64))[2]).astype(np.int64)
    pulls = [rng.normal(size=s).astype(np.float32) for s in (5, 5, (5, 3))]
    for g_pad, g_shift in ((pad, shift), (pad + 1, shift), (5, 1), (16 // dtype.itemsize, 0)):
        buf = torch.full((g_shift + 5 * (vocab + g_pad) + 9,), math.nan, dtype=dtype, device="cuda")
        g = buf.as_strided((5, vocab), (vocab + g_pad, 1), g_shift)
        assert op.backward(x, dev(y, torch.int64), *[dev(p) for p in pulls], grad=g) is g
        check_grad(x, y, 1.0, idx, [p.astype(np.float64) for p in pulls], g, dtype)
        g.fill_(math.nan)
        assert torch.isnan(buf).all()
        op.backward(x, dev(y, torch.int64), *[dev(p) for p in pulls], grad=g)
        assert int(torch.isnan(buf).sum()) == buf.numel() - 5 * vocab


def test_calls_are_independent():
    """Fewer tokens than the object holds; a second stream; a captured pair of
    calls replayed on new inputs; the same bits each time."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    g = torch.Generator(device="cuda").manual_seed(3)
    vocab, k = 9000, 6
    sets = []
    for n in (64, 64, 17):
        sets.append((torch.randn(n, vocab, device="cuda", generator=g).bfloat16() * 2,
                     torch.randint(-1, vocab, (n,), device="cuda", generator=g),
                     torch.randn(n, device="cuda", generator=g), torch.randn(n, device="cuda", generator=g),
                     torch.randn(n, k, device="cuda", generator=g)))

    def run(op, s):
        return (*op.forward(s[0], s[1]), op.backward(*s))

    want = [run(TokenScores(64, vocab, top_k=k), s) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ops = [TokenScores(64, vocab, top_k=k, stream=s) for s in streams]
    torch.cuda.synchronize()
    for i, s in enumerate(sets + sets[:1]):
        both = [run(op, s) for op in ops]
        torch.cuda.synchronize()
        for got in both:
            assert all(torch.equal(p, q) for p, q in zip(got, want[i % 3]))
    stream = streams[0]
    fixed = [t.clone() for t in sets[0]]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = run(ops[0], fixed)
    for s, b in zip(sets[:2], want):
        for t, v in zip(fixed, s):
            t.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, b))


def test_no_tokens():
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    x, y = torch.zeros(0, 50, device="cuda", dtype=BF16), torch.zeros(0, dtype=torch.int64, device="cuda")
    for op in (TokenScores(0, 50, top_k=2), TokenScores(3, 50, top_k=2)):
        got = op.forward(x, y)
        assert [tuple(t.shape) for t in got] == [(0,), (0,), (0, 2), (0, 2)]
        assert op.backward(x, y).shape == (0, 50)


def test_object_refuses():
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    op = TokenScores(8, 100, top_k=2)
    x, y = torch.zeros(8, 100, device="cuda", dtype=BF16), torch.zeros(8, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="last forward"):
        op.backward(x, y)
    for bad in (x.float(), x[:, :50], x.cpu(), torch.zeros(9, 100, device="cuda", dtype=BF16)):
        with pytest.raises(ValueError, match="logits"):
            op.forward(bad, y)
    for bad in (y.int(), y[:4], y.cpu()):
        with pytest.raises(ValueError, match="targets"):
            op.forward(x, bad)
    op.forward(x, y)
    first = op.calls
    op.forward(x, y)
    with pytest.raises(ValueError, match="has followed"):
        op.backward(x, y, call=first)
    with pytest.raises(ValueError, match="d_top"):
        op.backward(x, y, d_top=torch.zeros(8, 3, device="cuda"))
    with pytest.raises(ValueError, match="tokens"):
        op.backward(x[:4], y[:4])
    with pytest.raises(ValueError, match="none given"):
        bare = TokenScores(8, 100, with_grad=False)
        bare.forward(x, y)
        bare.backward(x, y)
    for bad in (dict(top_k=33), dict(top_k=-1), dict(top_k=101)):
        with pytest.raises(ValueError):
            TokenScores(8, 100 if bad["top_k"] != 101 else 3, **bad)


def test_longest_row():
    """Rows of 2^31 - 1 words, the most: a few finite ones at both ends and in
    between, the others -inf; a masked row; the gradient with rows that start
    elsewhere against 16 bytes than the logits'."""
    from fsdp_buffer_layout_gb300.objectives import TokenScores
    vocab, ld = (1 << 31) - 1, 1 << 31
    buf = torch.full((3 + 2 * ld,), -math.inf, dtype=BF16, device="cuda")
    x = buf.as_strided((2, vocab), (ld, 1), 3)
    words = [0, 1, 4, 5, 1 << 20, (1 << 30) + 7, vocab - 9, vocab - 8, vocab - 2, vocab - 1]
    at = dev(words, torch.int64)
    z = np.arange(10) * 0.25
    x[1, at] = dev(z).to(BF16)
    y = dev([-1, vocab - 1], torch.int64)
    op = TokenScores(2, vocab, top_k=4, with_grad=False)
    logp, entropy, idx, top_logp = op.forward(x, y)
    p = np.exp(z) / np.exp(z).sum()
    assert idx[1].tolist() == words[:5:-1] and idx[0].tolist() == [-1] * 4
    assert abs(logp[1].item() - math.log(p[-1])) <= 2.0**-20
    assert abs(entropy[1].item() + (p * np.log(p)).sum()) <= 2.0**-19
    assert np.abs(host(top_logp[1]) - np.log(p[:5:-1])).max() <= 2.0**-20
    h, d_top = -(p * np.log(p)).sum(), np.array([0.5, 0, -1.0, 2.0])
    want = -p * (1.0 + d_top.sum() + 3.0 * (np.log(p) + h))
    want[-1] += 1.0
    want[:5:-1] += d_top
    del logp, entropy, top_logp
    for shift in (3, 4):
        out = torch.full((shift + 2 * ld,), math.nan, dtype=BF16, device="cuda")
        g = out.as_strided((2, vocab), (ld, 1), shift)
        op.backward(x, y, dev([1.0, 1.0]), dev([3.0, 3.0]), dev(np.stack([d_top, d_top])), grad=g)
        assert (np.abs(host(g[1, at]) - want) <= 2.0**-8 * np.abs(want) + 2.0**-18).all()
        assert torch.count_nonzero(g[0]).item() == 0
        assert torch.count_nonzero(g[1]).item() == 10  # (NaN would count)
        assert torch.isnan(out[:shift]).all() and torch.isnan(out[shift + vocab:shift + ld]).all()
        del out, g
    assert op.device_error() == 0
