"""The mixture-of-experts calls without a GPU: refusals of the C entry points, and
the 64-bit reference's gradients against central differences."""
import numpy as np
import pytest

import expert_reference as R
from fsdp_buffer_layout_gb300 import vsf as V

A = 1 << 20  # an aligned address that no refused call reads
ARG, ALIGN = V.VSF_ERR_ARG, V.VSF_ERR_ALIGN


def refuse(call, args, change, want):
    with pytest.raises(V.VsfError) as e:
        call(**{**args, **change})
    assert e.value.status == want, change


SORT = dict(idx=A, T=4, top_k=2, E=8, starts=2 * A, source=3 * A, place=4 * A, d_workspace=5 * A,
            ws_bytes=1 << 20, stream=0)
GATHER = dict(x=A, dtype=V.VSF_BF16, T=4, H=64, ld=64, place=2 * A, top_k=2, rows=3 * A, rows_ld=64,
              stream=0)
COMBINE = dict(y=A, dtype=V.VSF_FP32, T=4, H=64, y_ld=64, place=2 * A, gates=3 * A, top_k=2, out=4 * A,
               out_ld=64, stream=0)
GRAD = dict(d_out=A, dtype=V.VSF_BF16, T=4, H=64, d_out_ld=64, y=2 * A, y_ld=64, place=3 * A,
            gates=4 * A, top_k=2, d_y=5 * A, d_y_ld=64, d_gates=6 * A, stream=0)
FORWARD = dict(x=A, rows=16, K=64, x_ld=64, w=2 * A, E=4, N=96, w_ld=64, w_stride=96 * 64, starts=3 * A,
               y=4 * A, y_ld=96, d_err=5 * A, stream=0)
INPUT = dict(d_y=A, rows=16, N=96, d_y_ld=96, w=2 * A, E=4, K=64, w_ld=64, w_stride=96 * 64,
             starts=3 * A, d_x=4 * A, d_x_ld=64, d_err=5 * A, stream=0)
WEIGHT = dict(d_y=A, rows=16, N=96, d_y_ld=96, x=2 * A, K=64, x_ld=64, E=4, starts=3 * A, d_w=4 * A,
              d_w_ld=64, d_w_stride=96 * 64, d_err=5 * A, stream=0)


@pytest.mark.parametrize("change,want", [
    (dict(idx=0), ARG), (dict(place=0), ARG), (dict(starts=0), ARG), (dict(d_workspace=0), ARG),
    (dict(T=-1), ARG), (dict(T=(1 << 23) + 1), ARG), (dict(top_k=0), ARG), (dict(top_k=33), ARG),
    (dict(E=0), ARG), (dict(E=513), ARG), (dict(ws_bytes=8), ARG),
    (dict(T=8192, ws_bytes=16), ARG),  # 16384 choices need counts of four runs
    (dict(place=A), ARG), (dict(starts=4 * A + 4), ARG), (dict(source=4 * A + 28), ARG),  # overlaps
    (dict(idx=A + 2), ALIGN), (dict(source=A + 1), ALIGN), (dict(d_workspace=A + 8), ALIGN)])
def test_sort_refusals(change, want):
    refuse(V.vsf_expert_sort, SORT, change, want)


def test_sort_workspace():
    assert V.vsf_expert_sort_workspace_bytes(4, 2, 8) > 0
    assert V.vsf_expert_sort_workspace_bytes(1 << 23, 32, 512) <= 1 << 20
    for bad in ((-1, 2, 8), (4, 0, 8), (4, 33, 8), (4, 2, 0), (4, 2, 513), ((1 << 23) + 1, 1, 8)):
        assert V.vsf_expert_sort_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("top_k,experts", [(1, 1), (1, 32), (4, 32), (5, 3), (8, 256), (32, 512)])
def test_sort_workspace_holds_every_smaller_call(top_k, experts):
    """The size asked for the most tokens is enough for fewer: it never falls, and a
    call is refused for less than what is asked for its own number only."""
    edges = [m * n // top_k + d for n in (1024, 2048, 65536) for m in range(1, 9) for d in range(-2, 3)]
    sizes = [V.vsf_expert_sort_workspace_bytes(t, top_k, experts)
             for t in sorted({0, 1, 1 << 23, *range(0, 400_000 // top_k, 331), *edges})]
    assert sizes == sorted(sizes) and sizes[0] > 0
    args = dict(SORT, top_k=top_k, E=experts, idx=1 << 40, starts=2 << 40, source=3 << 40, place=4 << 40)
    for t in (3000, 65536 // top_k, 65536 // top_k + 1):
        least = V.vsf_expert_sort_workspace_bytes(t, top_k, experts)
        refuse(V.vsf_expert_sort, args, dict(T=t, ws_bytes=least - 1), ARG)


@pytest.mark.parametrize("call,args,extra", [
    (V.vsf_expert_gather, GATHER, [
        (dict(x=0), ARG), (dict(rows=0), ARG), (dict(ld=63), ARG), (dict(rows_ld=63), ARG),
        (dict(rows=A + 128), ARG), (dict(x=A + 1), ALIGN), (dict(rows=A + 1), ALIGN)]),
    (V.vsf_expert_combine, COMBINE, [
        (dict(y=0), ARG), (dict(out=0), ARG), (dict(y_ld=63), ARG), (dict(out_ld=63), ARG),
        (dict(out=A), ARG), (dict(gates=A + 2), ALIGN), (dict(y=A + 2), ALIGN)]),
    (V.vsf_expert_combine_grad, GRAD, [
        (dict(d_out=0), ARG), (dict(y=0), ARG), (dict(d_y=0), ARG), (dict(gates=0), ARG),
        (dict(d_gates=0), ARG), (dict(d_gates=4 * A), ARG), (dict(d_gates=3 * A + 4), ARG), (dict(d_y=A), ARG), (dict(d_y=2 * A + 2), ARG),
        (dict(d_y=2 * A, d_y_ld=72), ARG), (dict(d_gates=A + 2), ALIGN), (dict(d_y=5 * A + 1), ALIGN)])])
def test_row_refusals(call, args, extra):
    for change, want in extra + [
            (dict(place=0), ARG), (dict(dtype=5), ARG), (dict(T=-1), ARG), (dict(H=0), ARG),
            (dict(H=(1 << 24) + 1), ARG), (dict(top_k=0), ARG), (dict(top_k=33), ARG),
            (dict(place=A + 2), ALIGN)]:
        refuse(call, args, change, want)
    call(**{**args, "T": 0})  # nothing to do, nothing launched


@pytest.mark.parametrize("call,args,extra", [
    (V.vsf_expert_product, FORWARD, [
        (dict(x=0), ARG), (dict(w=0), ARG), (dict(y=0), ARG), (dict(x_ld=56), ARG), (dict(y_ld=88), ARG),
        (dict(w_ld=56), ARG), (dict(w_stride=95 * 64), ARG), (dict(y=A), ARG), (dict(y=2 * A + 64), ARG),
        (dict(x=A + 8), ALIGN), (dict(w=2 * A + 2), ALIGN), (dict(y=4 * A + 4), ALIGN),
        (dict(x_ld=65), ALIGN), (dict(w_ld=65, w_stride=97 * 65), ALIGN), (dict(y_ld=97), ALIGN),
        (dict(w_stride=96 * 64 + 4), ALIGN),
        (dict(starts=4 * A + 16), ARG)]),
    (V.vsf_expert_product_input_grad, INPUT, [
        (dict(d_y=0), ARG), (dict(w=0), ARG), (dict(d_x=0), ARG), (dict(d_y_ld=88), ARG),
        (dict(d_x_ld=56), ARG), (dict(w_stride=95 * 64), ARG), (dict(d_x=A), ARG),
        (dict(d_y=A + 8), ALIGN), (dict(d_x_ld=65), ALIGN)]),
    (V.vsf_expert_product_weight_grad, WEIGHT, [
        (dict(d_y=0), ARG), (dict(x=0), ARG), (dict(d_w=0), ARG), (dict(rows=0, d_w=0), ARG),
        (dict(d_w_ld=56), ARG), (dict(d_w_stride=95 * 64), ARG), (dict(d_w=2 * A), ARG),
        (dict(d_w=4 * A + 8), ALIGN), (dict(d_w_stride=96 * 64 + 4), ALIGN), (dict(x_ld=68), ALIGN)])])
def test_product_refusals(call, args, extra):
    for change, want in extra + [
            (dict(rows=-1), ARG), (dict(rows=(1 << 28) + 1), ARG), (dict(E=0), ARG), (dict(E=513), ARG),
            (dict(N=0), ARG), (dict(K=0), ARG), (dict(K=(1 << 24) + 1), ARG), (dict(starts=0), ARG),
            (dict(d_err=0), ARG), (dict(starts=A + 2), ALIGN)]:
        refuse(call, args, change, want)


@pytest.mark.parametrize("call,args,changes", [
    (V.vsf_expert_gather, GATHER, [
        dict(rows=2 * A), dict(rows=2 * A + 16), dict(ld=1 << 39), dict(ld=1 << 57),
        dict(rows_ld=96, ld=96, rows=A + 62), dict(rows_ld=96, ld=96, rows=A + 66)]),
    (V.vsf_expert_combine, COMBINE, [
        dict(out=2 * A), dict(out=3 * A + 28), dict(y_ld=1 << 39), dict(T=1 << 23, out_ld=1 << 38),
        dict(y_ld=130, out_ld=130, out=A + 4 * 63), dict(y_ld=130, out_ld=130, out=A + 4 * 67)]),
    (V.vsf_expert_combine_grad, GRAD, [
        dict(d_gates=A), dict(d_gates=2 * A + 1020), dict(d_gates=5 * A), dict(d_y=3 * A), dict(d_y=4 * A + 28),
        dict(d_y=6 * A), dict(d_out_ld=1 << 39), dict(y_ld=128, d_y_ld=128, d_y=2 * A + 126)]),
    (V.vsf_expert_product, FORWARD, [
        dict(x_ld=1 << 39), dict(rows=1 << 28, y_ld=1 << 32), dict(w_stride=1 << 39),
        dict(x_ld=160, y_ld=160, y=A + 112), dict(x_ld=152, y_ld=152, y=A + 128)]),
    (V.vsf_expert_product_input_grad, INPUT, [
        dict(d_x=3 * A), dict(d_y_ld=160, d_x_ld=160, d_x=A + 176)]),
    (V.vsf_expert_product_weight_grad, WEIGHT, [
        dict(d_w=3 * A), dict(d_w=A + 64), dict(d_w_ld=1 << 39), dict(d_w_stride=1 << 39)])])
def test_overlaps_and_long_strides(call, args, changes):
    """An output among an input's rows, by one column too many; offsets past 2^58."""
    for change in changes:
        refuse(call, args, change, ARG)


def test_wait_selftest_refuses_a_limit_above_one_second():
    with pytest.raises(V.VsfError) as e:
        V.vsf_selftest_pair_waits(1_000_000_001)
    assert e.value.status == ARG
    V.vsf_selftest_pair_waits()


def test_no_rows_is_no_error():
    V.vsf_expert_product(**{**FORWARD, "rows": 0})
    V.vsf_expert_product_input_grad(**{**INPUT, "rows": 0})


def differences(f, x, step=1e-5):
    """Central differences of the scalar f at x."""
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        at = x[i]
        x[i] = at + step
        up = f()
        x[i] = at - step
        g[i] = (up - f()) / (2 * step)
        x[i] = at
    return g


def test_reference_gradients():
    """Linear and bilinear maps: central differences are exact but for rounding
    (1e-16 of values near 10, divided by the step)."""
    rng = np.random.default_rng(3)
    idx = np.array([[0, 2], [2, -1], [3, 0], [-1, -1], [2, 2]])
    starts, source, place = R.sort(idx, 4)
    assert starts.tolist() == [0, 2, 2, 6, 7] and source.tolist() == [0, 5, 1, 2, 8, 9, 4, -1, -1, -1]
    x, y = rng.normal(size=(5, 3)), rng.normal(size=(10, 3))
    gates, d_out, d_rows = rng.normal(size=(5, 2)), rng.normal(size=(5, 3)), rng.normal(size=(10, 3))
    zero = np.zeros((10, 3))
    got = R.combine(d_rows, place, np.ones((5, 2)))
    want = differences(lambda: (R.gather(x, place, zero) * d_rows).sum(), x)
    np.testing.assert_allclose(got, want, atol=1e-9)
    d_y, d_gates = R.combine_grad(d_out, y, place, gates, zero)

    def loss():
        return (R.combine(y, place, gates) * d_out).sum()

    np.testing.assert_allclose(d_y, differences(loss, y), atol=1e-9)
    np.testing.assert_allclose(d_gates, differences(loss, gates), atol=1e-9)
    w, rows, d_p = rng.normal(size=(4, 2, 3)), rng.normal(size=(7, 3)), rng.normal(size=(7, 2))
    d_x, d_w = R.product_grad(d_p, rows, w, starts)

    def scalar():
        return (R.product(rows, w, starts) * d_p).sum()

    np.testing.assert_allclose(d_x, differences(scalar, rows), atol=1e-9)
    np.testing.assert_allclose(d_w, differences(scalar, w), atol=1e-9)
