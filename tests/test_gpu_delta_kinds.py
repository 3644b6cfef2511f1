"""Every kind of the gated delta rule's kernels against the fp64
recurrence: types of the inputs and of the gradients, padded key sizes, rows
that 16-byte accesses fit and rows that they do not, keys of their own and
shared ones.  Each is compiled by itself, and may go wrong by itself.

Bounds as in test_gpu_delta.py, for gradients of 16 chained or added products:
fp32 inputs 16 x sqrt(256) x 2^-24 / 4 = 4e-6 rms, 5 times that at the largest
element, 2e-5; bf16 inputs (two terms) 5 x 2^-17 / sqrt(3) x sqrt(2 x 16) at the
largest, 1.3e-4, and half as much again where terms cancel, 2e-4; dg four
times; half an ulp for bf16 gradients."""
import pytest
import torch

import selective_state_space_64_amd as ssm
from delta_reference import delta_batch
from test_gpu_delta import ARGS, BF16, F32, error, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hk,h", [(2, 2), (1, 3)], ids=["own", "shared"])
@pytest.mark.parametrize("K,V", [(64, 72), (60, 65), (128, 72), (100, 65), (256, 72), (250, 65), (136, 33)])
@pytest.mark.parametrize("grad", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients(dtype, grad, K, V, hk, h):
    t, r, _ = make(dtype, [150, 150], False, hk, h, K, V, seed=K + h)
    t["dy"] = t["dy"].to(grad)
    r["dy"] = t["dy"].double().cpu().numpy()
    _, _, d0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, r["h0"], r["dy"], r["dhL"])
    d = ssm.ssm_delta_bwd(*(t[n] for n in ARGS), t["dy"], h0=t["h0"], dhL=t["dhL"])
    for n in d0:
        bound = (2e-5 if dtype == F32 else 2e-4) * (4 if n == "dg" else 1)
        if d[n].dtype == BF16:
            bound += torch.finfo(BF16).eps / 2
        assert error(d[n], d0[n]) <= bound, n


@pytest.mark.parametrize("lens", [[150, 150], [1100]], ids=["whole", "cut"])
@pytest.mark.parametrize("K,V", [(64, 72), (64, 33), (60, 65), (128, 136), (128, 33), (100, 65), (256, 72), (250, 65)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(dtype, K, V, lens):
    """The forward's kinds, on whole sequences and on one that is cut into segments; bounds as
    in test_gpu_delta.py (2e-5 for three terms, 1.2e-4 for two)."""
    t, r, _ = make(dtype, lens, False, 1, 2, K, V, seed=K + V)
    args = [t[n] for n in ARGS]
    y0, h0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, r["h0"])
    bound = 2e-5 if dtype == F32 else 1.2e-4
    y, hL = ssm.ssm_delta_fwd(*args, h0=t["h0"], out_dtype=F32)
    assert error(y, y0) <= bound and error(hL, h0) <= bound
    kept = ssm.ssm_delta_bwd_workspace(t["q"], t["v"])
    yc, hc = ssm.ssm_delta_fwd(*args, h0=t["h0"], out_dtype=F32, checkpoints=kept)
    assert torch.equal(yc, y) and torch.equal(hc, hL)
    yb, _ = ssm.ssm_delta_fwd(*args, h0=t["h0"], out_dtype=BF16)
    assert torch.equal(yb, y.to(BF16))
