"""The gated delta rule on slices of one buffer that lie beside each other in
every step: time-major rows ([L][batch][channels]), and the decode step's
answer behind its own inputs.  The same bits as on tensors of their own."""
import pytest
import torch

import selective_state_space_64_amd as ssm
from test_gpu_delta import ARGS, BF16, F32, make

pytestmark = pytest.mark.gpu


def rows(lead, dtype, *parts, fill=float("nan")):
    """A buffer of lead x channels, and its slices [..., heads, width]."""
    widths = [h * w for h, w in parts]
    buf = torch.full((*lead, sum(widths)), fill, dtype=dtype, device="cuda")
    return buf, [x.unflatten(-1, p) for x, p in zip(buf.split(widths, -1), parts)]


@pytest.mark.parametrize("dtype,B,L", [(BF16, 3, 150), (F32, 2, 65), (BF16, 2, 1), (BF16, 1, 70)])
def test_time_major(dtype, B, L):
    hk, h, K, V = 2, 4, 64, 72
    t, _, _ = make(dtype, [L] * B, False, hk, h, K, V, seed=L)
    dense = [t[n] for n in ARGS]
    y0, h0 = ssm.ssm_delta_fwd(*dense, h0=t["h0"])
    d0 = ssm.ssm_delta_bwd(*dense, t["dy"], h0=t["h0"], dhL=t["dhL"])
    parts = (hk, K), (hk, K), (h, V), (h, V)
    buf, views = rows((L, B), dtype, *parts)
    q, k, v, y = (x.transpose(0, 1) for x in views)
    for x, n in ((q, "q"), (k, "k"), (v, "v")):
        x.copy_(t[n])
    g, beta = (t[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("g", "beta"))
    y1, h1 = ssm.ssm_delta_fwd(q, k, v, g, beta, h0=t["h0"], y=y)  # y beside its inputs
    assert torch.equal(y1, y0) and torch.equal(h1, h0)
    out, outs = rows((L, B), dtype, *parts[:3])
    kw = dict(zip(("dq", "dk", "dv"), (x.transpose(0, 1) for x in outs)))
    d1 = ssm.ssm_delta_bwd(q, k, v, g, beta, t["dy"], h0=t["h0"], dhL=t["dhL"], **kw)
    for n in d0:
        assert torch.equal(d1[n], d0[n]), n
    for x, n in ((q, "q"), (k, "k"), (v, "v")):
        assert torch.equal(x, t[n])


def test_overlapping_time_major_slices_are_refused():
    t, _, _ = make(F32, [20, 20], False, 2, 2, 16, 16, seed=1)
    args = [t[n] for n in ARGS]
    buf = torch.zeros(20, 2, 72, device="cuda")
    part = lambda at: buf[..., at:at + 32].unflatten(-1, (2, 16)).transpose(0, 1)  # noqa: E731
    ssm.ssm_delta_bwd(*args, t["dy"], dq=part(0), dk=part(40))
    with pytest.raises(ssm.SSMError, match="ALIAS"):
        ssm.ssm_delta_bwd(*args, t["dy"], dq=part(0), dk=part(31))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_update_answers_into_the_same_rows(dtype):
    B, hk, h, K, V = 3, 2, 4, 64, 48
    t, _, _ = make(dtype, [1] * B, False, hk, h, K, V, seed=2)
    want = t["h0"].clone()
    y0 = ssm.ssm_delta_update(want, *(t[n][:, 0] for n in ARGS))
    buf, (q, k, v, y) = rows((B,), dtype, (hk, K), (hk, K), (h, V), (h, V))
    for x, n in ((q, "q"), (k, "k"), (v, "v")):
        x.copy_(t[n][:, 0])
    state = t["h0"].clone()
    y1 = ssm.ssm_delta_update(state, q, k, v, t["g"][:, 0], t["beta"][:, 0], y=y)
    assert y1 is y and torch.equal(y, y0) and torch.equal(state, want)
    with pytest.raises(ssm.SSMError, match="ALIAS"):
        ssm.ssm_delta_update(state, q, k, v, t["g"][:, 0], t["beta"][:, 0], y=v)
