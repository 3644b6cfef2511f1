"""The decode step of the gated delta rule with either width of its tiles and
every number of rows a thread, with 16-byte accesses to the state and without,
against the fp64 recurrence at the bounds of fp32 arithmetic (2e-5; half an ulp
for a bf16 answer)."""
import pytest

import selective_state_space_64_amd as ssm
from delta_reference import delta_batch
from test_gpu_delta import ARGS, BF16, F32, error, make, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("batch,h,K,V", [
    (2, 3, 30, 40), (2, 3, 33, 41),            # 32 columns for short keys: one and two rows
    (2, 4, 65, 64), (2, 4, 128, 62),           # 16 columns, two rows
    (2, 2, 129, 64), (3, 2, 256, 50),          # 16 columns, four
    (32, 4, 128, 64), (33, 4, 100, 66),        # 32 columns, four
    (32, 8, 256, 64), (33, 8, 200, 62),        # 32 columns, eight
    (31, 4, 128, 64), (32, 4, 129, 64),        # just below the change
])
def test_tiles(dtype, batch, h, K, V):
    t, r, _ = make(dtype, [1] * batch, False, h, h, K, V, seed=K)
    y0, h0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, r["h0"])
    state = t["h0"].clone()
    y = ssm.ssm_delta_update(state, *(t[n][:, 0] for n in ARGS))
    assert error(y, y0[:, 0]) <= tolerance(F32, dtype, 1) and error(state, h0) <= 2e-5
