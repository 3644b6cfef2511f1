"""The gated delta rule's final states written over its initial ones (hL is
h0), on sequences that the library cuts into segments: other workgroups then
write hL than read h0.  The same bits as with a buffer of its own, from either
start of the gradients too."""
import pytest
import torch

import selective_state_space_64_amd as ssm
from test_gpu_delta import ARGS, BF16, F32, make, name

pytestmark = pytest.mark.gpu

# the last segment of most is a chunk or less, so that it ends before the others
CASES = [
    (BF16, [2500], False, 1, 1, 128, 64, {}),
    (F32, [1100], False, 1, 2, 64, 40, {}),
    (F32, [1601], False, 1, 1, 100, 130, dict(decay="reset")),
    (BF16, [1500, 1500], False, 1, 2, 40, 200, {}),
    (F32, [1153], False, 1, 1, 200, 10, {}),
    (BF16, [4097], False, 4, 12, 128, 128, {}),
    (BF16, [700, 0, 1, 1500, 64, 900], True, 1, 2, 64, 48, {}),
    (BF16, [4097, 1, 2500, 0, 63, 2945], True, 2, 4, 128, 100, {}),
]


@pytest.mark.parametrize("case", CASES, ids=name)
def test_states_in_place(case):
    dtype, lens, packed, hk, h, K, V, opt = case
    t, _, cu = make(dtype, lens, packed, hk, h, K, V, seed=11, **opt)
    args = [t[n] for n in ARGS]
    y0, h0 = ssm.ssm_delta_fwd(*args, h0=t["h0"], cu_seqlens=cu)
    state = t["h0"].clone()
    y, hL = ssm.ssm_delta_fwd(*args, h0=state, hL=state, cu_seqlens=cu)
    assert hL is state and torch.equal(y, y0) and torch.equal(state, h0)
    state, ws = t["h0"].clone(), ssm.ssm_delta_bwd_workspace(t["q"], t["v"], cu_seqlens=cu)
    y, _ = ssm.ssm_delta_fwd(*args, h0=state, hL=state, cu_seqlens=cu, checkpoints=ws)
    assert torch.equal(y, y0) and torch.equal(state, h0)
    kw = dict(h0=t["h0"], dhL=t["dhL"], cu_seqlens=cu)
    a = ssm.ssm_delta_bwd(*args, t["dy"], workspace=ws, checkpoints_in_workspace=True, **kw)
    b = ssm.ssm_delta_bwd(*args, t["dy"], **kw)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_prefill_in_pieces():
    """A long prompt in pieces, the state handed on in place, against the whole."""
    h, K, V = 2, 64, 64
    t, _, _ = make(BF16, [3 * 1472], False, h, h, K, V, seed=12)
    args = [t[n] for n in ARGS]
    y0, h0 = ssm.ssm_delta_fwd(*args, h0=t["h0"], out_dtype=F32)
    state, ys = t["h0"].clone(), []
    for a in range(0, 3 * 1472, 1472):
        ys.append(ssm.ssm_delta_fwd(*(x[:, a:a + 1472] for x in args), h0=state, hL=state, out_dtype=F32)[0])
    # two runs of 1.2e-4 each (two bf16 terms in the products)
    for got, want in ((torch.cat(ys, 1), y0), (state, h0)):
        assert float(((got - want).abs() / want.abs().clamp_min(want.square().mean().sqrt())).max()) <= 2.4e-4
