"""The training objectives without a GPU: refusals of the C entry points and
of their Python objects, and the 64-bit reference's gradients against central
differences of its own losses."""
import numpy as np
import pytest

import objective_reference as R
from fsdp_buffer_layout_gb300 import vsf as V

A = 1 << 20  # an aligned address that no refused call reads


def policy_args(**kw):
    a = dict(logits=A, dtype=V.VSF_BF16, T=4, V=100, ld=100, targets=A, old_logp=A, ref_logp=A,
             advantages=A, weights=None, hp=V.make_policy_hparams(), stats=A, logp=A, grad=2 * A,
             grad_ld=100, d_workspace=A, ws_bytes=1 << 20, stream=0)
    return {**a, **kw}


BAD_ROWS = [
    (dict(logits=0), V.VSF_ERR_ARG), (dict(targets=0), V.VSF_ERR_ARG),
    (dict(dtype=7), V.VSF_ERR_ARG), (dict(T=-1), V.VSF_ERR_ARG), (dict(T=1 << 31), V.VSF_ERR_ARG),
    (dict(V=0), V.VSF_ERR_ARG), (dict(V=1 << 31, ld=1 << 31), V.VSF_ERR_ARG),
    (dict(ld=99), V.VSF_ERR_ARG), (dict(d_workspace=0), V.VSF_ERR_ARG),
    (dict(ws_bytes=64), V.VSF_ERR_ARG), (dict(d_workspace=A + 8), V.VSF_ERR_ALIGN),
    (dict(logits=A + 1), V.VSF_ERR_ALIGN), (dict(targets=A + 4), V.VSF_ERR_ALIGN),
    (dict(logp=A + 2), V.VSF_ERR_ALIGN),
]
BAD_LOSS = BAD_ROWS + [
    (dict(stats=0), V.VSF_ERR_ARG), (dict(grad_ld=99), V.VSF_ERR_ARG),
    (dict(grad=2 * A + 1), V.VSF_ERR_ALIGN), (dict(grad=A + 2), V.VSF_ERR_ARG),  # overlaps in part
    (dict(grad=A, grad_ld=101), V.VSF_ERR_ARG),
]


def refuse(call, args, want):
    with pytest.raises(V.VsfError) as e:
        call(**args)
    assert e.value.status == want


@pytest.mark.parametrize("change,want", BAD_LOSS + [
    (dict(old_logp=0), V.VSF_ERR_ARG), (dict(advantages=0), V.VSF_ERR_ARG),
    (dict(ref_logp=0, hp=V.make_policy_hparams(kl_beta=0.1)), V.VSF_ERR_ARG),
    (dict(old_logp=A + 2), V.VSF_ERR_ALIGN),
    (dict(hp=V.make_policy_hparams(clip_low=1.5)), V.VSF_ERR_ARG),
    (dict(hp=V.make_policy_hparams(clip_high=-0.1)), V.VSF_ERR_ARG),
    (dict(hp=V.make_policy_hparams(inv_temperature=0.0)), V.VSF_ERR_ARG),
    (dict(hp=V.make_policy_hparams(kl_beta=float("nan"))), V.VSF_ERR_ARG),
])
def test_policy_loss_refusals(change, want):
    refuse(V.vsf_policy_loss, policy_args(**change), want)


@pytest.mark.parametrize("change,want", [b for b in BAD_ROWS] + [
    (dict(inv_temperature=float("inf")), V.VSF_ERR_ARG), (dict(logp=0), V.VSF_ERR_ARG)])
def test_token_logprobs_refusals(change, want):
    a = dict(logits=A, dtype=V.VSF_BF16, T=4, V=100, ld=100, targets=A, inv_temperature=1.0,
             logp=A, d_workspace=A, ws_bytes=1 << 20, stream=0)
    refuse(V.vsf_token_logprobs, {**a, **change}, want)


@pytest.mark.parametrize("change,want", BAD_LOSS + [
    (dict(seq_starts=0), V.VSF_ERR_ARG), (dict(pairs=0), V.VSF_ERR_ARG),
    (dict(seq_starts=A + 4), V.VSF_ERR_ALIGN), (dict(rewards=A + 2), V.VSF_ERR_ALIGN),
    (dict(hp=V.make_preference_hparams(beta=0.0)), V.VSF_ERR_ARG),
    (dict(hp=V.make_preference_hparams(smoothing=0.6)), V.VSF_ERR_ARG),
    (dict(hp=V.make_preference_hparams(kind=9)), V.VSF_ERR_ARG),
])
def test_preference_loss_refusals(change, want):
    a = policy_args(seq_starts=A, pairs=2, rewards=A, hp=V.make_preference_hparams())
    for k in ("old_logp", "advantages"):
        del a[k]
    refuse(V.vsf_preference_loss, {**a, **change}, want)


def route_args(**kw):
    a = dict(logits=A, dtype=V.VSF_BF16, T=4, E=8, ld=8, bias=None, live=None, seq_starts=None,
             sequences=1, hp=V.make_route_hparams(2), idx=A, gates=A, counts=A, loss=A,
             seq_counts=A, seq_coef=A, d_workspace=A, ws_bytes=1 << 20, stream=0)
    return {**a, **kw}


BAD_ROUTE = [
    (dict(logits=0), V.VSF_ERR_ARG), (dict(dtype=3), V.VSF_ERR_ARG), (dict(T=-1), V.VSF_ERR_ARG),
    (dict(T=(1 << 23) + 1), V.VSF_ERR_ARG), (dict(E=0), V.VSF_ERR_ARG),
    (dict(E=513, ld=513), V.VSF_ERR_ARG), (dict(ld=7), V.VSF_ERR_ARG),
    (dict(sequences=2), V.VSF_ERR_ARG), (dict(sequences=0), V.VSF_ERR_ARG),
    (dict(idx=0), V.VSF_ERR_ARG), (dict(seq_counts=0), V.VSF_ERR_ARG),
    (dict(logits=A + 1), V.VSF_ERR_ALIGN), (dict(idx=A + 2), V.VSF_ERR_ALIGN),
    (dict(hp=V.make_route_hparams(0)), V.VSF_ERR_ARG),
    (dict(hp=V.make_route_hparams(9)), V.VSF_ERR_ARG),
    (dict(hp=V.make_route_hparams(2, score=5)), V.VSF_ERR_ARG),
    (dict(hp=V.make_route_hparams(2, balance=float("inf"))), V.VSF_ERR_ARG),
]


@pytest.mark.parametrize("change,want", BAD_ROUTE + [
    (dict(gates=0), V.VSF_ERR_ARG), (dict(loss=0), V.VSF_ERR_ARG),
    (dict(ws_bytes=64), V.VSF_ERR_ARG), (dict(d_workspace=A + 8), V.VSF_ERR_ALIGN)])
def test_route_refusals(change, want):
    refuse(V.vsf_route, route_args(**change), want)


@pytest.mark.parametrize("change,want", BAD_ROUTE + [
    (dict(grad=0), V.VSF_ERR_ARG), (dict(grad_ld=7), V.VSF_ERR_ARG),
    (dict(loss_scale=float("nan")), V.VSF_ERR_ARG), (dict(grad=A + 2), V.VSF_ERR_ARG)])
def test_route_grad_refusals(change, want):
    a = route_args()
    for k in ("bias", "gates", "counts", "loss", "d_workspace", "ws_bytes"):
        del a[k]
    a.update(d_gates=None, loss_scale=1.0, grad=2 * A, grad_ld=8)
    refuse(V.vsf_route_grad, {**a, **change}, want)


def test_workspaces():
    assert V.vsf_objective_workspace_bytes(0, 0) > 0
    assert V.vsf_objective_workspace_bytes(100, 3) > V.vsf_objective_workspace_bytes(100, 0)
    assert V.vsf_objective_workspace_bytes(-1, 0) == 0
    assert V.vsf_route_workspace_bytes(0, 1) == 0 == V.vsf_route_workspace_bytes(513, 1)
    with pytest.raises(V.VsfError):
        V.vsf_objective_workspace_init(0, 64, 0)


# -------------------------------------------- the reference against differences
def differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


@pytest.mark.parametrize("beta,mean", [(0.0, True), (0.3, False)])
def test_reference_policy_gradient(beta, mean):
    r = np.random.default_rng(1)
    x, y = r.normal(size=(5, 7)), np.array([0, 3, -1, 6, 2])
    lp = R.logprobs(x, y)
    old, ref, adv = lp + r.normal(size=5) * 0.4, lp + r.normal(size=5) * 0.3, r.normal(size=5)
    w = np.array([1.0, 0.5, 1.0, 0.0, 2.0])
    a = (y, old, adv, ref, w, 0.2, 0.3, beta, 0.7, 0.5, mean)
    got = R.policy(x, *a)[2]
    # h = 1e-5: h^2 times a third derivative of at most ~10, and 1e-16 / h
    assert np.abs(got - differences(lambda v: R.policy(v, *a)[0][0], x)).max() < 1e-8


@pytest.mark.parametrize("kind,average", [("sigmoid", False), ("squared", True)])
def test_reference_preference_gradient(kind, average):
    r = np.random.default_rng(2)
    x, y = r.normal(size=(9, 6)), r.integers(0, 6, 9)
    y[4] = -1
    a = (y, [0, 3, 3, 5, 8], r.normal(size=9), r.uniform(0.5, 1.5, 9), kind, 0.4, 0.1, 0.2, average,
         1.3, 0.5)
    got = R.preference(x, *a)[3]
    assert np.abs(got - differences(lambda v: R.preference(v, *a)[0][0], x)).max() < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_route_gradient(score, renorm):
    r = np.random.default_rng(3)
    x, dg = r.normal(size=(6, 5)), r.normal(size=(6, 2))
    a = (2, score, renorm, 1.5, 0.7, None, [1, 1, 0, 1, 1, 1], [0, 2, 2, 5])

    def f(v):  # the choice does not change within h
        idx, gates, _, loss, _ = R.route(v, *a)
        return loss + (gates * dg).sum()

    got = R.route(x, *a, d_gates=dg)[4]
    assert np.abs(got - differences(f, x)).max() < 1e-8
