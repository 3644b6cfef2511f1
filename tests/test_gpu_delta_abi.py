"""Calls of the gated delta rule and of the grouped norm through their C ABI
with strides that the binding does not pass on: of tensors of one step or one
batch entry, where they say nothing."""
import ctypes

import pytest
import torch

import selective_state_space_64_amd as ssm
from test_gpu_delta import ARGS, BF16, F32, make

pytestmark = pytest.mark.gpu

CODE = {F32: ssm.SSM_F32, BF16: ssm.SSM_BF16}


def layout(cls, step):
    """Dense strides but for the step's."""
    lay = cls()
    for i in range(len(lay.step)):
        lay.step[i] = step
    return lay


def batches(lay, sizes):
    for i, n in enumerate(sizes):
        lay.batch[i] = n
    return ctypes.byref(lay)


def run(t, dtype, hk, h, K, V, step):
    B = t["q"].shape[0]
    L = ssm.lib()
    stream = torch.cuda.current_stream().cuda_stream
    out = {"y": torch.full_like(t["v"], float("nan")), "hL": torch.full_like(t["h0"], float("nan"))}
    out.update({"d" + n: torch.full_like(t[n], float("nan")) for n in (*ARGS, "h0")})
    p = {n: x.data_ptr() for n, x in {**t, **out}.items()}
    need = L.ssm_delta_bwd_workspace_bytes(B, 1, hk, h, K, V, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    qk, vy = hk * K, h * V
    fwd = batches(layout(ssm.DeltaLayout, step), (qk, qk, vy, vy, h, h))
    bwd = batches(layout(ssm.DeltaBwdLayout, step), (qk, qk, vy, h, h, vy, qk, qk, vy))
    head = (B, 1, hk, h, K, V, CODE[dtype], 0, None, *(p[n] for n in ARGS), p["h0"], None, 0, CODE[dtype])
    assert L.ssm_delta_fwd(*head, p["y"], p["hL"], ws.data_ptr(), need, fwd, stream) == 0
    assert L.ssm_delta_bwd(*head, p["dy"], p["dhL"], p["dq"], p["dk"], p["dv"], p["dg"], p["dbeta"], p["dh0"],
                           ws.data_ptr(), need, bwd, stream) == 0
    return out


@pytest.mark.parametrize("step", [1, 8, 64])
@pytest.mark.parametrize("dtype,hk,h,K,V", [(BF16, 2, 4, 64, 72), (BF16, 1, 1, 128, 128), (F32, 2, 2, 64, 40),
                                            (BF16, 1, 2, 33, 17)],
                         ids=["copies", "one head", "runs", "elements"])
def test_step_stride_of_one_step(dtype, hk, h, K, V, step):
    t, _, _ = make(dtype, [1, 1, 1], False, hk, h, K, V, seed=step)
    want, got = (run(t, dtype, hk, h, K, V, s) for s in (0, step))
    for n in want:
        assert want[n].isfinite().all() and torch.equal(got[n], want[n]), n


def test_norm_batch_stride_of_one_entry():
    """dx and dz beside each other in the rows of one batch entry, whose batch
    strides lead nowhere and differ."""
    L, dim, groups = 5, 96, 4
    x, z, dy = (torch.randn(1, L, dim, device="cuda") for _ in range(3))
    want = ssm.ssm_group_norm_bwd(x, groups, dy, z=z)
    both = torch.zeros(L, 2 * dim, device="cuda")
    lay = ssm.NormBwdLayout()
    lay.step[3] = lay.step[4] = 2 * dim
    lay.batch[3], lay.batch[4] = 2 * dim * L, 2 * dim * L + 7
    assert ssm.lib().ssm_group_norm_bwd(
        1, L, dim, groups, ssm.SSM_F32, 0, None, x.data_ptr(), None, None, z.data_ptr(), ssm.SSM_F32, dy.data_ptr(),
        both.data_ptr(), both[:, dim:].data_ptr(), None, None, None, 0, ctypes.byref(lay),
        torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(both, torch.cat([want["dx"][0], want["dz"][0]], -1))
    want = ssm.ssm_group_norm_fwd(x, groups)  # and y in place of x
    lay = ssm.NormLayout()
    lay.batch[2] = dim * L + 7
    assert ssm.lib().ssm_group_norm_fwd(
        1, L, dim, groups, ssm.SSM_F32, 0, None, x.data_ptr(), None, None, None, ssm.SSM_F32, x.data_ptr(),
        ctypes.byref(lay), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(x, want)
