"""Token scores without a GPU: refusals, and the reference's gradient against
central differences of the reference's scores."""
import numpy as np
import pytest

import score_reference as R
from fsdp_buffer_layout_gb300 import vsf as V

A = 1 << 20  # an aligned address that no refused call reads
ARG, ALIGN = V.VSF_ERR_ARG, V.VSF_ERR_ALIGN
ROWS = dict(logits=A, dtype=V.VSF_BF16, T=4, V=100, ld=100, targets=2 * A, inv_temperature=1.0, top_k=3,
            stream=0)
SCORES = dict(ROWS, logp=3 * A, entropy=4 * A, top_idx=5 * A, top_logp=6 * A, norm=7 * A,
              d_workspace=8 * A, ws_bytes=1 << 20)
GRAD = dict(ROWS, norm=7 * A, top_idx=5 * A, d_logp=3 * A, d_entropy=4 * A, d_top=6 * A, grad=9 * A,
            grad_ld=100)
BAD_ROWS = [
    (dict(logits=0), ARG), (dict(targets=0), ARG), (dict(dtype=7), ARG), (dict(T=-1), ARG),
    (dict(T=1 << 31), ARG), (dict(V=0), ARG), (dict(V=1 << 31, ld=1 << 31), ARG), (dict(ld=99), ARG),
    (dict(inv_temperature=0.0), ARG), (dict(inv_temperature=float("nan")), ARG),
    (dict(inv_temperature=3e38), ARG), (dict(top_k=-1), ARG), (dict(top_k=33), ARG),
    (dict(V=2, top_k=3), ARG), (dict(norm=0), ARG), (dict(top_idx=0), ARG), (dict(logits=A + 1), ALIGN),
    (dict(targets=2 * A + 4), ALIGN), (dict(norm=7 * A + 8), ALIGN), (dict(top_idx=A + 2), ALIGN),
]


@pytest.mark.parametrize("change,want", BAD_ROWS + [
    (dict(logp=0), ARG), (dict(entropy=0), ARG), (dict(top_logp=0), ARG), (dict(d_workspace=0), ARG),
    (dict(ws_bytes=128), ARG), (dict(d_workspace=8 * A + 4), ALIGN), (dict(logp=A + 2), ALIGN),
    (dict(entropy=A + 1), ALIGN), (dict(top_logp=A + 2), ALIGN)])
def test_scores_refusals(change, want):
    with pytest.raises(V.VsfError) as e:
        V.vsf_token_scores(**{**SCORES, **change})
    assert e.value.status == want


@pytest.mark.parametrize("change,want", BAD_ROWS + [
    (dict(grad=0), ARG), (dict(grad_ld=99), ARG), (dict(grad=A + 2), ARG), (dict(grad=A, grad_ld=101), ARG),
    (dict(grad=9 * A + 1), ALIGN), (dict(d_logp=A + 2), ALIGN), (dict(d_entropy=A + 2), ALIGN),
    (dict(d_top=A + 2), ALIGN)])
def test_gradient_refusals(change, want):
    with pytest.raises(V.VsfError) as e:
        V.vsf_token_scores_grad(**{**GRAD, **change})
    assert e.value.status == want


def test_no_tokens_is_no_error():
    V.vsf_token_scores(**{**SCORES, "T": 0})
    V.vsf_token_scores_grad(**{**GRAD, "T": 0})


def test_workspace_holds_every_smaller_call():
    """Fewer tokens get smaller pieces; the size asked for covers them."""
    for dtype in (V.VSF_BF16, V.VSF_FP32):
        for vocab in (1, 7, 1000, 32000, 131072, 300001, 5_000_000, 2**31 - 1):
            sizes = [V.vsf_token_scores_workspace_bytes(t, vocab, dtype, min(vocab, 4))
                     for t in (0, 1, 7, 100, 4096)]
            assert sizes == sorted(sizes) and sizes[0] > 0
            assert V.vsf_token_scores_workspace_bytes(7, vocab, dtype, 0) <= sizes[2]
    for bad in ((-1, 5, 0, 1), (4, 0, 0, 0), (4, 5, 9, 1), (4, 5, 0, 6), (4, 100, 0, 33), (4, 100, 0, -1)):
        assert V.vsf_token_scores_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("inv_t", [1.0, 0.6, 1.7])
def test_reference_gradient(inv_t):
    """Central differences of step 1e-5: truncation 1e-10 of third derivatives of
    order 10, rounding 1e-16 / 1e-5."""
    rng = np.random.default_rng(2)
    x, y = rng.normal(size=(4, 9)) * 2, np.array([3, -1, 0, 8])
    k = 3
    idx = R.scores(x, y, inv_t, k)[2]
    y[2] = idx[2, 1]  # a target that is one of the alternatives
    d_logp, d_entropy, d_top = rng.normal(size=4), rng.normal(size=4), rng.normal(size=(4, k))

    def loss():
        logp, entropy, now, top_logp = R.scores(x, y, inv_t, k)
        assert (now == idx).all()
        return (d_logp * logp + d_entropy * entropy + (d_top * top_logp).sum(1))[y >= 0].sum()

    got = R.gradient(x, y, inv_t, idx, d_logp, d_entropy, d_top)
    for i in np.ndindex(*x.shape):
        at, step = x[i], 1e-5
        x[i] = at + step
        up = loss()
        x[i] = at - step
        down = loss()
        x[i] = at
        assert abs(got[i] - (up - down) / (2 * step)) <= 1e-8
