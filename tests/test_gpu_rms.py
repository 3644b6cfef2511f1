"""The residual norm on the GPU (ssm_rms_norm_fwd, ssm_rms_norm_bwd) against its
plain fp64 form.

Error of a tensor: max |got - ref| / max(|ref|, rms(ref)).  The kernels work in
fp32: statistics of n <= 2^15 channels (relative error sqrt(n) 2^-24 at most, 1.1e-5, the
sums being trees), about ten operations an element, and for dweight sums of a few
thousand rows: 1.2e-5 covers them at the largest of 1e6 elements.  A bf16 output adds
half an ulp, half of torch.finfo(bfloat16).eps, 2^-8; e4m3 half of its eps, 2^-4,
of a value, and half of its smallest step, 2^-10 of the scale, near zero.
"""
import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from heads_reference import block_scales, rms_norm
from test_gpu_delta import error

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
FP32_ERROR = 1.2e-5


def tolerance(out):
    return FP32_ERROR + (torch.finfo(BF16).eps / 2 if out == BF16 else 0.0)


def make(dtype, shape, stream, weight=True, seed=0):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    t = {"x": torch.tensor(n(shape)).to(dtype), "dy": torch.tensor(n(shape)).to(dtype),
         "residual": torch.tensor(3 * n(shape)).to(stream) if stream else None,
         "dh": torch.tensor(n(shape)).to(stream) if stream else None,
         "weight": torch.tensor(1 + 0.2 * n(shape[-1]), dtype=F32) if weight else None}
    ref = {m: None if v is None else v.double().numpy() for m, v in t.items()}
    return {m: None if v is None else v.cuda() for m, v in t.items()}, ref


def check_8bit(q, scales, y):
    s0 = block_scales(y)
    assert q.dtype == E4M3 and scales.shape == s0.shape and error(scales, s0) <= FP32_ERROR
    s = np.repeat(scales.double().cpu().numpy(), 128, -1)[..., :y.shape[-1]]
    off = np.abs(q.double().cpu().numpy() * s - y)
    # half a step of the value, which may itself be off by FP32_ERROR
    assert (off <= np.maximum(np.abs(y) * (torch.finfo(E4M3).eps / 2 + 2 * FP32_ERROR), s * (2.0 ** -10 + 1e-5))).all()


SHAPES = [(1, 1, 1), (3, 5, 6), (2, 3, 127), (2, 3, 129), (2, 33, 128), (7, 512), (2, 9, 776), (3, 333, 1531), (2, 7, 1536),
          (5, 2560), (1, 300, 2560), (2, 3, 5120), (4, 3, 4099), (3, 8200), (2, 9001), (1, 2, 16392), (2, 20001), (700, 3, 40)]


@pytest.mark.parametrize("out", [F32, BF16, E4M3], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("dtype,stream", [(F32, None), (F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)],
                         ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(dtype, stream, out, shape):
    t, r = make(dtype, shape, stream, weight=shape[-1] != 512, seed=sum(shape))
    y0, h0 = rms_norm(r["x"], r["weight"], r["residual"])
    y, h, scales = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], residual=t["residual"], out_dtype=out)
    if stream:
        assert h.dtype == stream and error(h, h0) <= (2.0 ** -24 if stream == F32 else torch.finfo(BF16).eps / 2)
    else:
        assert h is None
    if out == E4M3:
        check_8bit(y, scales, y0)
    else:
        assert scales is None and y.dtype == out and error(y, y0) <= tolerance(out)


@pytest.mark.parametrize("dtype,stream", [(F32, None), (F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)],
                         ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradients(dtype, stream, shape):
    t, r = make(dtype, shape, stream, weight=shape[-1] != 512, seed=sum(shape))
    h = t["residual"] if stream else t["x"]
    y0, _, d0 = rms_norm(r["residual"] if stream else r["x"], r["weight"], None, dy=r["dy"], dh=r["dh"])
    d = ssm.ssm_rms_norm_bwd(h, t["dy"], weight=t["weight"], dh=t["dh"])
    # where n is small the two parts of a gradient cancel: it is held against their size
    parts = rms_norm(r["residual"] if stream else r["x"], r["weight"], None, dy=r["dy"])[2]["dx"] if shape[-1] > 1 else None
    assert d["dx"].dtype == dtype
    if shape[-1] == 1:
        size = np.abs(r["dy"]).max() + (np.abs(r["dh"]).max() if stream else 0.0)
        hv = (r["residual"] if stream else r["x"])
        size = size * (1 + np.abs(1 / hv).max())
        assert np.abs(d["dx"].double().cpu().numpy() - d0["dx"]).max() <= tolerance(dtype) * size
    else:
        assert parts is not None and error(d["dx"], d0["dx"]) <= tolerance(dtype)
        if stream:
            assert d["dresidual"].dtype == stream and error(d["dresidual"], d0["dx"]) <= tolerance(stream)
        else:
            assert d["dresidual"] is None
    if t["weight"] is None:
        assert d["dweight"] is None
    else:
        assert error(d["dweight"], d0["dweight"]) <= FP32_ERROR
