"""Tokens by expert and the experts' products on the GPU against the 64-bit reference.

Tolerances. The sort and the rows' copy are exact. A sum of n fp32 products, added
in any order, is within n 2^-24 of the sum of their absolute values (n 2^-23 for the
tensor cores, whose additions may cut off instead of rounding); the rounding to
the output's type adds half a step, 2^-8 of the value for bf16 and 2^-24 for fp32.
"""
import numpy as np
import pytest
import torch

import expert_reference as R

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0**-8, FP32: 2.0**-24}


def host(x):
    return x.double().cpu().numpy()


def strided(rows, width, pad, shift, dtype, rng, scale=1.0):
    """A matrix in rows of width + pad elements, `shift` elements into its memory."""
    ld = width + pad
    buf = torch.zeros(shift + max(rows, 1) * ld, dtype=dtype, device="cuda")
    x = torch.as_strided(buf, (rows, width), (ld, 1), shift)
    x.copy_(torch.from_numpy((rng.normal(size=(rows, width)) * scale).astype(np.float32)))
    return x


def choices(rng, tokens, experts, k, masked):
    idx = rng.integers(0, experts, size=(tokens, k)).astype(np.int32)
    if masked:
        idx[rng.random((tokens, k)) < 0.2] = -1
        idx[rng.random(tokens) < 0.2] = -1
        idx[rng.random((tokens, k)) < 0.02] = experts + 5  # no expert of this layer
    return torch.from_numpy(idx).cuda()


DISPATCH = [  # tokens, experts, k, width, dtype, masked, pad, shift
    (0, 3, 2, 16, BF16, False, 0, 0),
    (1, 1, 1, 1, BF16, False, 0, 0),
    (1, 8, 3, 64, FP32, False, 0, 0),
    (7, 5, 2, 8, BF16, True, 0, 0),
    (8, 32, 4, 2880, BF16, False, 0, 0),
    (33, 6, 5, 257, BF16, True, 0, 0),
    (33, 6, 6, 257, FP32, True, 2, 1),
    (40, 4, 2, 1030, BF16, True, 2, 8),    # aligned rows with a tail
    (100, 512, 8, 130, FP32, True, 2, 4),
    (65, 3, 32, 96, BF16, True, 0, 3),     # rows off the 16-byte boundaries
    (300, 7, 7, 40, FP32, True, 1, 0),
    (257, 9, 8, 64, BF16, True, 0, 0),     # eight lanes a token
    (130, 9, 5, 250, BF16, True, 6, 8),
    (90, 9, 8, 61, FP32, True, 0, 1),
    (64, 40, 9, 64, BF16, True, 0, 0),     # as narrow, but nine choices
]


@pytest.mark.parametrize("case", DISPATCH, ids=str)
def test_dispatch(case):
    from fsdp_buffer_layout_gb300.experts import Dispatch
    tokens, experts, k, width, dtype, masked, pad, shift = case
    rng = np.random.default_rng(hash(case[:4]) % 1000 + 1)
    idx = choices(rng, tokens, experts, k, masked)
    x, d_out = (strided(tokens, width, pad, shift, dtype, rng) for _ in range(2))
    y, d_rows = (strided(tokens * k, width, pad, shift, dtype, rng) for _ in range(2))
    gates = torch.from_numpy(rng.normal(size=(tokens, k)).astype(np.float32)).cuda()
    call = Dispatch(tokens, experts, k, width, dtype=dtype)
    want_starts, want_source, want_place = R.sort(host(idx).astype(np.int64).reshape(tokens, k), experts)
    starts, source, place = call.sort(idx)
    assert np.array_equal(host(starts), want_starts)
    assert np.array_equal(host(source), want_source)
    assert np.array_equal(host(place).reshape(tokens, k), want_place)
    # garbage behind the last row must not matter, nor what no choice took
    n = int(want_starts[-1])
    y[n:] = float("nan")
    d_rows[n:] = float("nan")
    gates[torch.from_numpy(want_place < 0).cuda()] = float("nan")
    rows = call.gather(x)
    assert torch.equal(rows.cpu(), torch.from_numpy(
        R.gather(host(x), want_place, np.zeros((tokens * k, width)))).to(dtype))

    def check(got, want, size, terms):
        got = host(got)
        bound = HALF[dtype] * np.abs(want) + 1.01 * terms * 2.0**-24 * size + 1e-38
        assert got.shape == want.shape and np.isfinite(got).all()
        assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / bound)

    g0, p = np.nan_to_num(host(gates)), want_place
    y0 = np.nan_to_num(host(y))
    check(call.combine(y, gates), R.combine(y0, p, g0), R.combine(np.abs(y0), p, np.abs(g0)), k + 1)
    dr = np.nan_to_num(host(d_rows))
    one = np.ones((tokens, k))
    check(call.gather_backward(d_rows), R.combine(dr, p, one), R.combine(np.abs(dr), p, one), k)
    d_y, d_gates = call.combine_backward(d_out, y, gates)
    zero = np.zeros((tokens * k, width))
    want_dy, want_dg = R.combine_grad(host(d_out), y0, p, g0, zero)
    check(d_y, want_dy, np.abs(want_dy), 2)
    size = R.combine_grad(np.abs(host(d_out)), np.abs(y0), p, g0, zero)[1]
    off = np.abs(host(d_gates).reshape(tokens, k) - want_dg)
    assert (off <= 1.01 * (width / 32 + 48) * 2.0**-24 * size + 1e-38).all()
    # the same again, and into y itself
    again = y.clone(memory_format=torch.preserve_format) if pad == 0 and shift == 0 else None
    if again is not None and tokens:
        got = call.combine_backward(d_out, again, gates, d_y=again)[0]
        assert torch.equal(got[:n], d_y[:n]) and torch.isnan(got[n:]).all()


@pytest.mark.parametrize("tokens,experts,k,live", [
    (1025, 8, 8, 1.0), (4096, 3, 2, 0.5), (8193, 1, 1, 1.0), (20000, 512, 8, 0.9), (70001, 33, 3, 0.97),
    (300000, 256, 5, 1.0)])
def test_sort_of_many(tokens, experts, k, live):
    """Against torch's stable sort of whole numbers; more than one run, and more
    choices a run than the least."""
    from fsdp_buffer_layout_gb300.experts import Dispatch
    g = torch.Generator(device="cuda").manual_seed(tokens)
    idx = (torch.rand(tokens, k, device="cuda", generator=g) ** 2 * experts).int().clamp(max=experts - 1)
    idx[torch.rand(tokens, device="cuda", generator=g) >= live] = -1
    call = Dispatch(tokens, experts, k, 8, with_grad=False)
    for _ in range(2):
        starts, source, place = call.sort(idx)
        flat = idx.flatten().long()
        key = torch.where(flat < 0, experts, flat)
        order = torch.sort(key, stable=True).indices
        counts = torch.bincount(key, minlength=experts + 1)[:experts]
        n = int(counts.sum())
        assert torch.equal(starts[1:].long(), counts.cumsum(0)) and int(starts[0]) == 0
        assert torch.equal(source[:n].long(), order[:n]) and bool((source[n:] == -1).all())
        want = torch.full_like(flat, -1)
        want[order[:n]] = torch.arange(n, device="cuda")
        assert torch.equal(place.flatten().long(), want)
        idx = idx.flip(0).contiguous()


@pytest.mark.parametrize("tokens,experts,k,calls", [
    (20000, 32, 4, (20000, 16384, 15000, 3000, 10241, 400, 0, 20000)),
    (10000, 256, 8, (8192, 10000, 8193, 1)), (131073, 5, 1, (65536, 65537, 131072, 131073, 70000))])
def test_sorts_of_fewer_tokens(tokens, experts, k, calls):
    """One object, calls of fewer tokens than it holds, one after the other; and rows
    of as many tokens to their places and back."""
    from fsdp_buffer_layout_gb300.experts import Dispatch
    g = torch.Generator(device="cuda").manual_seed(tokens)
    call = Dispatch(tokens, experts, k, 8, with_grad=False)
    for n in calls:
        idx = torch.randint(-1, experts, (n, k), device="cuda", generator=g).int()
        starts, source, place = call.sort(idx)
        want_starts, want_source, want_place = R.sort(host(idx).astype(np.int64).reshape(n, k), experts)
        assert np.array_equal(host(starts), want_starts) and np.array_equal(host(source), want_source)
        assert np.array_equal(host(place).reshape(n, k), want_place)
        x = torch.randn(n, 8, device="cuda", generator=g).bfloat16()
        rows, here = call.gather(x), source >= 0
        assert torch.equal(rows[here], x[source[here].long() // k])


@pytest.mark.parametrize("dtype,width", [(BF16, 2048), (FP32, 999)])
def test_many_rows(dtype, width):
    """More rows than warps run at a time, in both directions."""
    from fsdp_buffer_layout_gb300.experts import Dispatch
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens, experts, k = 4099, 64, 6
    idx = torch.randint(-1, experts, (tokens, k), device="cuda", generator=g).int()
    call = Dispatch(tokens, experts, k, width, dtype=dtype)
    starts, source, place = call.sort(idx)
    n = int(starts[-1])
    x, d_out = (torch.randn(tokens, width, device="cuda", generator=g).to(dtype) for _ in range(2))
    y = torch.randn(tokens * k, width, device="cuda", generator=g).to(dtype)
    gates = torch.rand(tokens, k, device="cuda", generator=g)
    rows = call.gather(x)
    assert torch.equal(rows[:n], x[source[:n].long() // k]) and not rows[n:].any()
    taken = torch.where((place >= 0)[:, :, None], y[place.long().clamp(min=0)].double(), 0.0)
    want = (taken * gates.double()[:, :, None]).sum(1)
    size = (taken.abs() * gates.double()[:, :, None]).sum(1)
    off = (call.combine(y, gates).double() - want).abs()
    assert bool((off <= HALF[dtype] * want.abs() + 8 * 2.0**-24 * size).all())
    d_y, d_gates = call.combine_backward(d_out, y, gates)
    want = gates.flatten()[source[:n].long()].double()[:, None] * d_out[source[:n].long() // k].double()
    assert bool(((d_y[:n].double() - want).abs() <= (HALF[dtype] + 2.0**-23) * want.abs()).all())
    assert not d_y[n:].any()
    want = (taken * d_out.double()[:, None]).sum(2)
    size = (taken * d_out.double()[:, None]).abs().sum(2)
    assert bool(((d_gates.double() - want).abs() <= (width / 32 + 48) * 2.0**-24 * size).all())


# ------------------------------------------------------------------ products
PRODUCTS = [  # rows of each expert, rows behind, out, in, pads
    ([1], 0, 1, 1, 0),
    ([3], 0, 8, 16, 0),
    ([16], 0, 64, 64, 0),
    ([0, 5, 0], 3, 32, 24, 0),
    ([17, 1, 0, 40], 2, 130, 70, 8),
    ([32, 31, 33, 64, 15], 0, 256, 128, 0),
    ([255, 256, 257], 5, 96, 200, 0),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16], 1, 300, 65, 16),
    ([700, 0, 129, 513], 100, 521, 333, 0),
    ([64] * 40 + [0] * 3 + [65], 0, 257, 129, 0),   # many tiles of one stage
    ([1000], 24, 1000, 520, 0),
    ([90, 300, 10], 0, 2880, 576, 0),
    ([300, 7, 220, 31, 0, 513], 3, 9000, 70, 0),    # more wide tiles than pairs of CTAs
    ([200, 130, 257], 0, 70, 9000, 0),
    ([150, 400], 9, 1030, 1100, 0),                 # tiles of half the width
    ([1200, 1100, 900], 0, 64, 1500, 0),            # of a quarter
]


def product_inputs(counts, behind, n, k, pad, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * n + k)
    rows, experts = sum(counts) + behind, len(counts)

    def made(*shape):
        wide = -(-shape[-1] // 8) * 8 + pad
        return torch.randn(*shape[:-1], wide, device="cuda", generator=g).bfloat16()[..., :shape[-1]]

    starts = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
    return starts, made(rows, k), made(experts, n, k), made(rows, n)


def product_bound(want, size, terms):
    return HALF[BF16] * want.abs() + 1.01 * terms * 2.0**-23 * size + 1e-38


def check_products(call, starts, x, w, d_y):
    """All three products of every expert against 64 bits; rows behind untouched."""
    cuts = starts.tolist()
    y, d_x = call.forward(x, w, starts), call.backward_input(d_y, w, starts)
    d_w = call.backward_weight(d_y, x, starts)
    n, k = w.shape[1:]
    for e, (a, b) in enumerate(zip(cuts, cuts[1:])):
        xe, we, de = x[a:b].double(), w[e].double(), d_y[a:b].double()
        for got, p, q, terms in ((y[a:b], xe, we.t(), k), (d_x[a:b], de, we, n),
                                 (d_w[e], de.t(), xe, b - a)):
            want, size = p @ q, p.abs() @ q.abs()
            off = (got.double() - want).abs()
            assert bool((off <= product_bound(want, size, terms)).all()), (e, float(off.max()))
    assert not y[cuts[-1]:].any() and not d_x[cuts[-1]:].any()
    assert call.device_error() == 0


@pytest.mark.parametrize("case", PRODUCTS, ids=str)
def test_products(case):
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    counts, behind, n, k, pad = case
    starts, x, w, d_y = product_inputs(*case)
    call = ExpertLinear(x.shape[0], len(counts), n, k)
    # rows behind the last one, and the weights of experts without a row, are not read
    x[starts[-1]:] = float("nan")
    d_y[starts[-1]:] = float("nan")
    cuts = starts.tolist()
    call.d_weight.fill_(float("nan"))
    check_products(call, starts, x, w, d_y)
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")
    y = call.forward(x, w, starts)
    assert not y[cuts[-1]:].any() and bool(torch.isfinite(y).all())


def test_an_experts_rows_stay_its_own():
    """NaN and infinities in one expert's rows reach no other expert."""
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    counts = [5, 21, 64, 130, 7]
    starts, x, w, d_y = product_inputs(counts, 0, 200, 136, 0)
    cuts = starts.tolist()
    call = ExpertLinear(x.shape[0], 5, 200, 136)
    for bad in (1, 3):
        x[cuts[bad]:cuts[bad + 1]] = float("nan")
        d_y[cuts[bad]:cuts[bad + 1]] = float("inf")
    y, d_x = call.forward(x, w, starts), call.backward_input(d_y, w, starts)
    d_w = call.backward_weight(d_y, x, starts)
    for e in range(5):
        finite = e not in (1, 3)
        for part in (y[cuts[e]:cuts[e + 1]], d_x[cuts[e]:cuts[e + 1]], d_w[e]):
            assert bool(torch.isfinite(part).all()) == finite, e
    assert call.device_error() == 0


def test_products_without_rows():
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    starts = torch.zeros(4, dtype=torch.int32, device="cuda")
    call = ExpertLinear(50, 3, 40, 24)
    w = torch.randn(3, 40, 24, device="cuda").bfloat16()
    for rows in (0, 50):  # none in the arrays, none of any expert
        x = torch.randn(rows, 24, device="cuda").bfloat16()
        d_y = torch.randn(rows, 40, device="cuda").bfloat16()
        call.d_weight.fill_(3.0)
        assert call.forward(x, w, starts).shape == (rows, 40)
        assert not call.backward_input(d_y, w, starts).any() and not call.y.any()
        assert not call.backward_weight(d_y, x, starts).any()


def test_starts_out_of_range():
    """What starts holds is device memory: whatever it is, no access leaves the
    arrays. Clamped to [0, rows] and to what precedes."""
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    rows, n, k = 70, 48, 40
    _, x, w, d_y = product_inputs([rows, 0, 0], 0, n, k, 0)
    call = ExpertLinear(rows, 3, n, k)
    bad = torch.tensor([-5, 20, 10, 1 << 30], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 20, 20, rows], dtype=torch.int32, device="cuda")
    for run in (lambda s: call.forward(x, w, s), lambda s: call.backward_input(d_y, w, s),
                lambda s: call.backward_weight(d_y, x, s)):
        a = run(bad).clone()
        assert torch.equal(a, run(good))
    assert call.device_error() == 0


def test_offsets_past_32_bits():
    """Rows 2^20 elements apart, 2^31 and more from the first to the last."""
    from fsdp_buffer_layout_gb300.experts import Dispatch, ExpertLinear
    tokens, experts, k, width, ld = 1100, 5, 2, 72, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(2)

    def far(rows):
        x = torch.empty(rows * ld, dtype=BF16, device="cuda").as_strided((rows, width), (ld, 1))
        return x.copy_(torch.randn(rows, width, device="cuda", generator=g))

    idx = torch.randint(-1, experts, (tokens, k), device="cuda", generator=g).int()
    gates = torch.rand(tokens, k, device="cuda", generator=g)
    x, y = far(tokens), far(tokens * k)
    near = [t.contiguous() for t in (x, y)]
    calls = [Dispatch(tokens, experts, k, width) for _ in range(2)]
    starts = [c.sort(idx)[0] for c in calls][0]
    rows = far(tokens * k).zero_()
    assert torch.equal(calls[0].gather(x, out=rows), calls[1].gather(near[0]))
    assert torch.equal(calls[0].combine(y, gates), calls[1].combine(near[1], gates))
    assert torch.equal(calls[0].gather_backward(y), calls[1].gather_backward(near[1]))
    d_y = far(tokens * k).zero_()
    a = calls[0].combine_backward(x, y, gates, d_y=d_y)
    b = calls[1].combine_backward(near[0], near[1], gates)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    del d_y, a, x
    w = torch.randn(experts, 96, width, device="cuda", generator=g).bfloat16()
    d = torch.randn(tokens * k, 96, device="cuda", generator=g).bfloat16()
    layers = [ExpertLinear(tokens * k, experts, 96, width) for _ in range(2)]
    assert torch.equal(layers[0].forward(y, w, starts), layers[1].forward(near[1], w, starts))
    assert torch.equal(layers[0].backward_weight(d, y, starts), layers[1].backward_weight(d, near[1], starts))
    rows.zero_()
    assert torch.equal(layers[0].backward_input(d, w, starts, out=rows),
                       layers[1].backward_input(d, w, starts))


@pytest.mark.parametrize("experts,rows", [(512, 1), (512, 3), (300, 40)])
def test_many_experts(experts, rows):
    """As many as a launch may have, a row or some each, every third without one."""
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    counts = [0 if e % 3 == 1 else rows + e % 2 for e in range(experts)]
    starts, x, w, d_y = product_inputs(counts, 0, 72, 40, 0)
    check_products(ExpertLinear(x.shape[0], experts, 72, 40), starts, x, w, d_y)


def test_products_on_streams_and_in_graphs():
    """Two objects at once on two streams, and a captured call replayed on new
    inputs, give the bits of calls one after the other."""
    from fsdp_buffer_layout_gb300.experts import Dispatch, ExpertLinear
    tokens, experts, k, h, f = 300, 9, 3, 256, 320
    g = torch.Generator(device="cuda").manual_seed(11)
    w = torch.randn(experts, f, h, device="cuda", generator=g).bfloat16()

    def inputs():
        return (torch.randint(-1, experts, (tokens, k), device="cuda", generator=g).int(),
                torch.randn(tokens, h, device="cuda", generator=g).bfloat16(),
                torch.rand(tokens, k, device="cuda", generator=g))

    def made(stream=None):
        return (Dispatch(tokens, experts, k, h, stream=stream),
                ExpertLinear(tokens * k, experts, f, h, stream=stream))

    def run(calls, idx, x, gates):
        to, layer = calls
        starts, _, _ = to.sort(idx)
        rows = to.gather(x)
        y = layer.forward(rows, w, starts)
        d_rows = layer.backward_input(y, w, starts)
        d_w = layer.backward_weight(y, rows, starts)
        return (to.combine(d_rows, gates), *to.combine_backward(x, d_rows, gates), d_w,
                to.gather_backward(d_rows))

    sets = [inputs() for _ in range(3)]
    # (an object each: rows behind the last one keep what another call left there)
    plain = [made() for _ in sets]
    want = [run(p, *s) for p, s in zip(plain, sets)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    pairs = [made(s) for s in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run(p, *s) for p, s in zip(pairs, sets)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for p, q in zip(a, b):
                assert torch.equal(p, q)
    fixed = [t.clone() for t in sets[0]]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    calls = made(stream)
    with torch.cuda.stream(stream):
        run(calls, *fixed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = run(calls, *fixed)
    for s, b in zip(sets, want):
        for t, v in zip(fixed, s):
            t.copy_(v)
        calls[0].d_y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, b):
            assert torch.equal(p, q)
    assert all(layer.device_error() == 0 for _, layer in pairs + [calls] + plain)


@pytest.mark.parametrize("dtype,width,gap", [(BF16, 128, 0), (FP32, 77, 3), (BF16, 200, 8)])
def test_columns_of_shared_rows(dtype, width, gap):
    """Inputs and outputs side by side in the rows of one array."""
    from fsdp_buffer_layout_gb300.experts import Dispatch
    rng = np.random.default_rng(width)
    tokens, experts, k, at = 50, 5, 3, width + gap
    buf = strided(tokens * k, 2 * at, 0, 0, dtype, rng)
    before = host(buf)
    left, right = buf[:, :width], buf[:, at:at + width]
    idx = choices(rng, tokens, experts, k, True)
    gates = torch.from_numpy(rng.normal(size=(tokens, k)).astype(np.float32)).cuda()
    op = Dispatch(tokens, experts, k, width, dtype=dtype)
    starts, _, place = op.sort(idx)
    place, n = host(place).astype(int), int(starts[-1])
    op.gather(left[:tokens], out=right)
    want = before.copy()
    want[:, at:at + width] = R.gather(before[:tokens, :width], place, before[:, at:at + width])
    assert np.array_equal(host(buf), want) and n > 0
    d_out = strided(tokens, width, 0, 0, dtype, rng)
    d_y, d_gates = op.combine_backward(d_out, right, gates, d_y=left)
    want_y, want_gates = R.combine_grad(host(d_out), want[:, at:at + width], place, host(gates), want[:, :width])
    assert d_y is left
    assert (np.abs(host(left) - want_y) <= (HALF[dtype] + 2.0**-24) * np.abs(want_y) * 1.01).all()
    assert np.array_equal(host(right), want[:, at:at + width])
    size = R.combine_grad(np.abs(host(d_out)), np.abs(want[:, at:at + width]), place, host(gates),
                          want[:, :width])[1]
    assert (np.abs(host(d_gates) - want_gates) <= (width + 1) * 2.0**-24 * size * 1.01).all()


@pytest.mark.parametrize("counts,n,k", [
    ([40, 0, 33, 70], 3, 5), ([64, 32, 96], 94, 523), ([100, 32], 1001, 257), ([70, 64], 7, 9),
    ([33, 64, 31], 130, 70), ([300, 257], 263, 1030), ([64], 1, 1), ([32, 64], 8, 16), ([128], 511, 383)])
def test_products_stay_inside_their_rows(counts, n, k):
    """What lies beside and behind the outputs' rows keeps its values, whatever the
    widths are; NaN beside and behind the inputs' rows does not matter."""
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    g = torch.Generator(device="cuda").manual_seed(n)
    rows, experts = sum(counts) + 4, len(counts)
    starts = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")

    def among(rows, width, fill):
        """An array of `width` in rows 16 to 23 elements longer, 8 elements into a buffer."""
        ld = -(-width // 8) * 8 + 16
        buf = fill(8 + rows * ld + 24)
        return buf, buf.as_strided((rows, width), (ld, 1), 8)

    def noise(size):
        return torch.randn(size, device="cuda", generator=g).bfloat16()

    def nan(size):
        return torch.full((size,), float("nan"), dtype=BF16, device="cuda")

    x, d_y, w = (among(r, c, nan)[1] for r, c in ((rows, k), (rows, n), (experts * (n + 1), k)))
    for t in (x[:-4], d_y[:-4], w):
        t.copy_(torch.randn(t.shape, device="cuda", generator=g))
    w = w.as_strided((experts, n, k), ((n + 1) * w.stride(0), w.stride(0), 1), w.storage_offset())
    op = ExpertLinear(rows, experts, n, k)
    want = [t.clone() for t in (op.forward(x, w, starts), op.backward_input(d_y, w, starts),
                                op.backward_weight(d_y, x, starts))]
    assert all(torch.isfinite(t).all() for t in want)
    used = sum(counts)
    for call, args, new, height, width in ((op.forward, (x, w, starts), want[0], rows, n),
                                           (op.backward_input, (d_y, w, starts), want[1], rows, k)):
        buf, out = among(height, width, noise)
        before = buf.clone()
        assert call(*args, out=out) is out
        before.as_strided(out.shape, out.stride(), out.storage_offset())[:used] = new[:used]
        assert torch.equal(buf, before)
    buf, flat = among(experts * (n + 1), k, noise)
    shape, stride = (experts, n, k), ((n + 1) * flat.stride(0), flat.stride(0), 1)
    before, out = buf.clone(), buf.as_strided(shape, stride, 8)
    op.backward_weight(d_y, x, starts, out=out)
    before.as_strided(shape, stride, 8).copy_(want[2])
    assert torch.equal(buf, before)
    assert op.device_error() == 0


def test_rows_of_earlier_calls():
    """A call with fewer choices leaves the rows behind its last one as they were, in
    the object's outputs and in given ones; what `source` marks is the result."""
    from fsdp_buffer_layout_gb300.experts import Dispatch, ExpertLinear
    rng = np.random.default_rng(21)
    tokens, experts, k, width = 90, 5, 3, 72
    x, d_out = (strided(tokens, width, 0, 0, BF16, rng) for _ in range(2))
    y, given = (strided(tokens * k, width, 0, 0, BF16, rng) for _ in range(2))
    w = strided(experts * width, width, 0, 0, BF16, rng).view(experts, width, width)
    gates = torch.from_numpy(rng.random(size=(tokens, k)).astype(np.float32)).cuda()
    idx = [choices(rng, tokens, experts, k, masked) for masked in (False, True)]

    def run(to, layer, idx):
        starts, source, _ = to.sort(idx)
        rows = to.gather(x)
        out = (rows, to.combine_backward(d_out, y, gates)[0], layer.forward(rows, w, starts),
               layer.backward_input(y, w, starts), to.gather(x, out=given))
        return int(starts[-1]), source, out

    made = [(Dispatch(tokens, experts, k, width), ExpertLinear(tokens * k, experts, width, width))
            for _ in range(2)]
    full, _, out = run(*made[0], idx[0])
    before = [t.clone() for t in out]
    n, source, out = run(*made[0], idx[1])
    _, _, want = run(*made[1], idx[1])
    assert full == tokens * k > n
    for got, old, new in zip(out, before, want):
        assert torch.equal(got[n:], old[n:]) and got[n:].any()
        kept = torch.where(source[:, None] >= 0, got, 0)
        assert torch.equal(kept[:n], new[:n]) and not kept[n:].any()
        assert torch.equal(kept.float().sum(0), torch.where(source[:, None] >= 0, new, 0).float().sum(0))


def test_a_single_row_among_others():
    """One token's row in a column block of the array whose other columns are
    written: a single row has no stride, and shares no byte with them."""
    from fsdp_buffer_layout_gb300.experts import Dispatch, ExpertLinear
    rng = np.random.default_rng(8)
    buf = strided(8, 128, 0, 0, BF16, rng)
    left, right = buf[:, :64], buf[:, 64:]
    want = host(left[3])
    idx = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    op = Dispatch(1, 8, 8, 64)
    op.sort(idx)
    op.gather(left[3:4], out=right)
    assert (host(right) == want).all()
    out = op.combine(right, torch.ones(1, 8, device="cuda"), out=left[5:6])
    assert (host(out) == 8 * want).all() and (host(left[3]) == want).all()
    w = strided(64, 64, 0, 0, BF16, rng)[None]
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    before, y = host(buf), ExpertLinear(1, 1, 64, 64).forward(left[2:3], w, starts, out=right[2:3])
    want, size = before[2:3, :64] @ host(w[0]).T, np.abs(before[2:3, :64]) @ np.abs(host(w[0])).T
    assert (np.abs(host(y) - want) <= (HALF[BF16] * np.abs(want) + 64 * 2.0**-23 * size) * 1.01).all()
    before[2, 64:] = host(y)
    assert np.array_equal(host(buf), before)
    from fsdp_buffer_layout_gb300 import vsf as V
    for bad in (buf[:, 63:127], buf[:, 1:65]):  # one column of the row itself
        with pytest.raises(V.VsfError, match="overlaps"):
            op.gather(left[3:4], out=bad)


def test_products_beside_their_rows():
    """Rows and products in the rows of one array; one expert whose matrix has an
    odd stride; a single row of any stride."""
    from fsdp_buffer_layout_gb300.experts import ExpertLinear
    rng = np.random.default_rng(5)
    rows, experts, n_out, n_in = 70, 3, 40, 64
    buf = strided(rows, n_in + n_out, 0, 0, BF16, rng)
    x, y = buf[:, :n_in], buf[:, n_in:]
    w = strided(experts * n_out, n_in, 0, 0, BF16, rng).view(experts, n_out, n_in)
    starts = torch.tensor([0, 20, 20, 61], dtype=torch.int32, device="cuda")
    before = host(buf)
    op = ExpertLinear(rows, experts, n_out, n_in)
    op.forward(x, w, starts, out=y)
    got = host(buf)
    want = R.product(before[:, :n_in], host(w), host(starts).astype(int))
    size = R.product(np.abs(before[:, :n_in]), np.abs(host(w)), host(starts).astype(int))
    lim = HALF[BF16] * np.abs(want[:61]) + n_in * 2.0**-23 * size[:61]
    assert np.array_equal(got[:, :n_in], before[:, :n_in]) and np.array_equal(got[61:], before[61:])
    assert (np.abs(got[:61, n_in:] - want[:61]) <= lim * 1.01).all()
    one = ExpertLinear(1, 1, n_out, n_in)
    w1, starts = w[1].as_strided((1, n_out, n_in), (n_out * n_in - 3, n_in, 1)), starts[:2].clamp(max=1)
    x1 = x[3:4].clone().as_strided((1, n_in), (n_in + 1, 1))
    got = host(one.forward(x1, w1, starts))
    want, size = host(x1) @ host(w1)[0].T, np.abs(host(x1)) @ np.abs(host(w1)[0]).T
    assert (np.abs(got - want) <= (HALF[BF16] * np.abs(want) + n_in * 2.0**-23 * size) * 1.01).all()
    d_w = torch.empty_like(w1[0]).as_strided((1, n_out, n_in), (n_out * n_in + 5, n_in, 1))
    d_y = strided(1, n_out, 0, 0, BF16, rng).as_strided((1, n_out), (n_out + 3, 1))
    assert one.backward_weight(d_y, x1, starts, out=d_w) is d_w
    want = host(d_y).T @ host(x1)
    assert (np.abs(host(d_w)[0] - want) <= HALF[BF16] * np.abs(want) * 1.01).all()


def test_objects_refuse():
    from fsdp_buffer_layout_gb300.experts import Dispatch, ExpertLinear
    call = Dispatch(8, 4, 2, 32)
    x, y = torch.zeros(8, 32, device="cuda", dtype=BF16), torch.zeros(16, 32, device="cuda", dtype=BF16)
    gates = torch.zeros(8, 2, device="cuda")
    with pytest.raises(ValueError, match="sort first"):
        call.gather(x)
    idx = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    for bad in (idx.long(), idx[:, :1], idx.cpu(), torch.zeros(9, 2, dtype=torch.int32, device="cuda"),
                torch.zeros(2, 8, dtype=torch.int32, device="cuda").t()):
        with pytest.raises(ValueError, match="idx"):
            call.sort(bad)
    call.sort(idx)
    first = call.calls
    for bad in (x.float(), x[:4], x[:, :16], x.cpu(), x.t().contiguous().t()):
        with pytest.raises(ValueError, match="x:"):
            call.gather(bad)
    with pytest.raises(ValueError, match="gates"):
        call.combine(y, gates.double())
    with pytest.raises(ValueError, match="gates"):
        call.combine_backward(x, y, None)
    with pytest.raises(ValueError, match="y:"):
        call.combine(x, gates)
    call.sort(idx[:4].contiguous())
    with pytest.raises(ValueError, match="has followed"):
        call.gather_backward(y[:8], call=first)
    bare = Dispatch(8, 4, 2, 32, with_grad=False)
    bare.sort(idx)
    with pytest.raises(ValueError, match="with_grad"):
        bare.gather_backward(y)
    assert bare.gather_backward(y, out=x) is x
    for bad in ((-1, 4, 2, 32), (8, 0, 2, 32), (8, 513, 2, 32), (8, 4, 33, 32), (8, 4, 2, 0)):
        with pytest.raises(ValueError, match="out of range"):
            Dispatch(*bad)
    layer = ExpertLinear(16, 4, 24, 32)
    w = torch.zeros(4, 24, 32, device="cuda", dtype=BF16)
    starts = torch.zeros(5, dtype=torch.int32, device="cuda")
    for args, what in (((y, w.float(), starts), "weight"), ((y, w[:3], starts), "weight"),
                       ((y, w, starts[:4]), "starts"), ((y, w, starts.long()), "starts"),
                       ((y[:, :16], w, starts), "x"),
                       ((torch.zeros(17, 32, device="cuda", dtype=BF16), w, starts), "x")):
        with pytest.raises(ValueError, match=what):
            layer.forward(*args)
    odd = torch.zeros(4, 24, 33, device="cuda", dtype=BF16)[:, :, :32]
    from fsdp_buffer_layout_gb300 import vsf as V
    with pytest.raises(V.VsfError, match="16-byte"):
        layer.forward(y, odd, starts)
