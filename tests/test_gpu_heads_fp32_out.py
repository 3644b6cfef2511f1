"""An fp32 y of bf16 inputs: the head scan keeps 24 bits of what forms it.

The error is relative in the 2-norm over all of y.  A y is a sum of terms
C S and W x, each off by the rounding of its operands to three bf16 terms
(2^-25), by the fp32 rounding of the products' sums (2^-24, a few of them), by
the hardware's exponential in the decays (an ulp, 2^-23) and by the decay
exponents' own rounding (2^-24 of an exponent of about 1 where a term counts):
2e-7 in the root of the mean square, held to five times that.  Two terms
(up to 2^-17 of an operand) leave 2.4e-6.
"""
import numpy as np
import pytest
import torch

from test_gpu_heads import BF16, F32, call, make, reference

import selective_state_space_64_amd as ssm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,packed,g,h,N,P,opt", [
    ([130, 130], False, 1, 5, 128, 64, {}), ([200], False, 2, 4, 64, 72, dict(steps="small")),
    ([300], False, 1, 2, 100, 36, {}), ([90], False, 1, 2, 217, 7, {}), ([200], False, 1, 2, 256, 64, dict(steps="small")),
    ([1500], False, 1, 2, 32, 16, {}), ([700, 40, 0, 900, 300], True, 1, 2, 64, 64, {}),
    ([1, 0, 63, 64, 65, 128, 7], True, 2, 4, 128, 33, {})], ids=str)
def test_fp32_output_of_bf16_inputs(lens, packed, g, h, N, P, opt):
    t, r, cu = make(BF16, lens, packed, g, h, N, P, seed=N, **opt)
    y0, _ = reference(r, lens if packed else None)
    y, hL = call(t, cu, out_dtype=F32)
    off = y.double().cpu().numpy() - y0
    assert np.sqrt((off * off).sum() / (y0 * y0).sum()) <= 1e-6
    # with states kept for the gradients: the same bits; and the state does not depend on y's type
    ws = ssm.ssm_head_scan_bwd_workspace(t["x"], t["B"], cu_seqlens=cu)
    yc, hc = call(t, cu, out_dtype=F32, checkpoints=ws)
    assert torch.equal(yc, y) and torch.equal(hc, hL) and torch.equal(call(t, cu)[1], hL)
