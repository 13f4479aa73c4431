"""The training objectives without a GPU: where their arguments' ranges end."""
import math

import pytest

from fsdp_buffer_layout_gb300 import vsf as V
from test_objectives import A, policy_args


@pytest.mark.parametrize("bad", [0.0, -1.0, 2.0**127 * 1.0000002, 3.0e38, math.inf, math.nan])
def test_inverse_temperature_out_of_range(bad):
    """Above 2^127 its product with log2(e) would not fit fp32."""
    rows = dict(logits=A, dtype=V.VSF_BF16, T=4, V=100, ld=100, targets=A, logp=A, d_workspace=A,
                ws_bytes=1 << 20, stream=0)
    pref = policy_args(seq_starts=A, pairs=2, rewards=A, hp=V.make_preference_hparams(inv_temperature=bad))
    for k in ("old_logp", "advantages"):
        del pref[k]
    for call, args in ((V.vsf_token_logprobs, dict(rows, inv_temperature=bad)),
                       (V.vsf_policy_loss, policy_args(hp=V.make_policy_hparams(inv_temperature=bad))),
                       (V.vsf_preference_loss, pref)):
        with pytest.raises(V.VsfError) as e:
            call(**args)
        assert e.value.status == V.VSF_ERR_ARG and "2^127" in str(e.value)


def test_structs_match_the_header(tmp_path, monkeypatch):
    """The hyper-parameters' ctypes structures against the C header."""
    import test_abi_layout as L
    monkeypatch.setattr(L, "STRUCTS", [V.vsf_policy_hparams, V.vsf_preference_hparams,
                                       V.vsf_route_hparams])
    if L.shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    L.test_ctypes_structs_match_the_header(tmp_path)
