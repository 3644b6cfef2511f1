"""The gated delta rule on fp32 inputs with keys of more than 128 entries.
Every product of fp32 inputs keeps three bf16 terms (24 bits), whatever K: the
bound is the one of short keys, 4 chained products of up to 256 summands in
fp32, 4 x sqrt(256) x 2^-24 = 4e-6 rms and 5 times that at the largest element,
2e-5; 4 times as much for dg, which sums differences of such terms.  Two terms
in any of the products would leave 2^-17 of an operand, 4e-5 at the largest."""
import pytest

import selective_state_space_64_amd as ssm
from delta_reference import delta_batch
from test_gpu_delta import ARGS, F32, error, make, name

pytestmark = pytest.mark.gpu

CASES = [
    (F32, [129], False, 1, 2, 200, 24, {}),
    (F32, [150], False, 1, 1, 256, 70, dict(state=False)),
    (F32, [257], False, 2, 4, 136, 65, dict(decay="reset")),
    (F32, [100, 0, 37], True, 1, 2, 250, 16, dict(decay="none")),
    # cut into segments
    (F32, [1153], False, 1, 1, 200, 10, {}),
    (F32, [1153], False, 1, 1, 256, 40, dict(decay="none")),
    (F32, [1100, 1, 1300], True, 1, 1, 129, 40, dict(decay="none")),
]


@pytest.mark.parametrize("case", CASES, ids=name)
def test_three_terms(case):
    dtype, lens, packed, hk, h, K, V, opt = case
    t, r, cu = make(dtype, lens, packed, hk, h, K, V, seed=21, **opt)
    y0, h0, d0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, lens if packed else None, r["h0"], r["dy"], r["dhL"])
    args, kw = [t[n] for n in ARGS], dict(h0=t["h0"], cu_seqlens=cu)
    y, hL = ssm.ssm_delta_fwd(*args, **kw)
    assert error(y, y0) <= 2e-5 and error(hL, h0) <= 2e-5
    d = ssm.ssm_delta_bwd(*args, t["dy"], dhL=t["dhL"], **kw)
    for n in d0:
        assert error(d[n], d0[n]) <= (8e-5 if n == "dg" else 2e-5), n
