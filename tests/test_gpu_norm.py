"""The grouped norm on the GPU (ssm_group_norm_fwd, ssm_group_norm_bwd)
against its plain fp64 form.

Error of a tensor: max |got - ref| / max(|ref|, rms(ref)).  The kernels work in
fp32: statistics of n <= 2^13 channels (relative error sqrt(n) 2^-24), about ten
operations an element, and for dweight and dbias sums of a few thousand rows:
1e-5 covers them at the largest of 1e6 elements.  A bf16 output adds half an
ulp: half of torch.finfo(bfloat16).eps, 2^-8.
"""
import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from delta_reference import norm
from test_gpu_delta import error

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def tolerance(out):
    return 1e-5 + (torch.finfo(BF16).eps / 2 if out == BF16 else 0.0)


def make(dtype, shape, act, affine, seed=0, out=None):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    t = {"x": torch.tensor(n(shape) * 0.8 + 0.2).to(dtype), "dy": torch.tensor(n(shape)).to(out or dtype),
         "z": torch.tensor(n(shape)).to(dtype) if act.startswith("gate") else None,
         "weight": torch.tensor(1 + 0.2 * n(shape[-1]), dtype=F32) if affine != "none" else None,
         "bias": torch.tensor(0.2 * n(shape[-1]), dtype=F32) if affine == "both" else None}
    ref = {m: None if v is None else v.double().numpy() for m, v in t.items()}
    return {m: None if v is None else v.cuda() for m, v in t.items()}, ref


#       dtype shape groups act affine rms out
CASES = [
    (F32, (1, 1, 1), 1, "none", "none", True, F32),
    (F32, (1, 1, 2), 1, "none", "both", False, F32),
    (BF16, (3, 5, 6), 3, "silu", "both", False, BF16),
    (BF16, (2, 33, 640), 5, "gate", "weight", True, BF16),
    (F32, (2, 33, 1536), 12, "gate", "weight", True, F32),
    (F32, (2, 7, 1530), 6, "silu", "both", False, F32),
    (BF16, (1, 300, 5120), 40, "gate_first", "weight", True, BF16),
    (BF16, (2, 9, 5120), 1, "none", "weight", True, BF16),
    (F32, (2, 9, 5120), 1, "gate", "both", False, F32),
    (BF16, (4, 3, 4099), 1, "gate_first", "both", False, BF16),
    (F32, (1, 17, 1025), 1, "silu", "weight", False, F32),
    (BF16, (1, 40, 2048), 1, "gate", "both", False, F32),
    (F32, (1, 40, 1024), 1, "none", "none", False, BF16),
    (BF16, (5, 12), 4, "gate", "none", True, BF16),
    (F32, (700, 3, 36), 3, "gate_first", "weight", False, F32),
    (BF16, (1, 4000, 64), 1, "silu", "weight", True, BF16),
]


def name(c):
    return "%s-%s-g%d-%s-%s-%s-%s" % (str(c[0])[6:], "x".join(map(str, c[1])), c[2], c[3], c[4], "rms" if c[5] else "mean",
                                      str(c[6])[6:])


@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward_and_gradients(case):
    dtype, shape, groups, act, affine, rms, out = case
    t, r = make(dtype, shape, act, affine, seed=len(name(case)), out=out)
    opt = dict(rms=rms, silu=act == "silu", gate_first=act == "gate_first")
    kw = dict(weight=t["weight"], bias=t["bias"], z=t["z"], **opt)
    rk = dict(weight=r["weight"], bias=r["bias"], z=r["z"], **opt)
    y = ssm.ssm_group_norm_fwd(t["x"], groups, out_dtype=out, **kw)
    assert y.dtype == out and error(y, norm(r["x"], groups, **rk)) <= tolerance(out)
    d = ssm.ssm_group_norm_bwd(t["x"], groups, t["dy"], **kw)
    d0 = norm(r["x"], groups, dy=r["dy"], **rk)
    # a group of one channel, or a tensor whose true gradient vanishes, is compared with the size of its terms
    for n, want in (("dx", d0["dx"]), ("dz", d0["dz"]), ("dweight", d0["dweight"]), ("dbias", d0["dbias"])):
        given = {"dx": True, "dz": t["z"] is not None, "dweight": t["weight"] is not None,
                 "dbias": t["bias"] is not None}[n]
        if not given:
            assert d[n] is None
        elif n == "dx" and shape[-1] // groups <= 2:  # dx is a small rest of cancelling terms there
            scale = np.abs(r["dy"]).max() * 100
            assert np.max(np.abs(d[n].double().cpu().numpy() - want)) <= tolerance(out) * scale
        else:
            assert error(d[n], want) <= tolerance(d[n].dtype), n
    again = ssm.ssm_group_norm_bwd(t["x"], groups, t["dy"], **kw)
    for n in d:
        assert d[n] is None or torch.equal(d[n], again[n])


@pytest.mark.parametrize("off", [0, 3])
def test_strides(off):
    """x and z as halves of one projection (aligned and not), outputs into parts of wider buffers."""
    B, L, dim, groups = 2, 19, 256, 2
    t, _ = make(BF16, (B, L, dim), "gate", "both", seed=3)
    kw = dict(weight=t["weight"], bias=t["bias"])
    y0 = ssm.ssm_group_norm_fwd(t["x"], groups, z=t["z"], **kw)
    d0 = ssm.ssm_group_norm_bwd(t["x"], groups, t["dy"], z=t["z"], **kw)
    wide = torch.full((B, L, 2 * dim + 8), float("nan"), dtype=BF16, device="cuda")
    out = torch.full_like(wide, float("nan"))
    x, z = wide[..., off:off + dim], wide[..., off + dim:off + 2 * dim]
    x.copy_(t["x"])
    z.copy_(t["z"])
    dx, dz = out[..., off:off + dim], out[..., off + dim:off + 2 * dim]
    y = ssm.ssm_group_norm_fwd(x, groups, z=z, y=dx, **kw)
    d = ssm.ssm_group_norm_bwd(x, groups, t["dy"], z=z, dx=dx, dz=dz, **kw)
    if off == 0:
        assert torch.equal(d["dx"], d0["dx"]) and torch.equal(d["dz"], d0["dz"])
    for n in ("dx", "dz"):
        assert error(d[n], d0[n].double().cpu().numpy()) <= 2.0 ** -8 + 1e-5
    assert d["dx"].data_ptr() == dx.data_ptr()
    y = ssm.ssm_group_norm_fwd(x, groups, z=z, y=x, **kw)  # in place
    assert error(y, y0.double().cpu().numpy()) <= 2.0 ** -8 + 1e-5
    assert torch.equal(z, t["z"]) and wide[..., off + 2 * dim:].isnan().all()


def test_extremes():
    """Rows of zeros, of one value and of large values; a gate far on either side; NaN stays in its group."""
    x = torch.zeros(4, 3, 128, device="cuda")
    x[1], x[2] = 3.0, 1e15
    x[2, :, ::2] = -1e15
    z = torch.full_like(x, -200.0)
    z[..., 64:] = 200.0
    for kw in (dict(), dict(z=z), dict(silu=True), dict(z=z, gate_first=True), dict(rms=True)):
        rk = {n: v.double().cpu().numpy() if n == "z" else v for n, v in kw.items()}
        y = ssm.ssm_group_norm_fwd(x, 2, **kw)
        assert error(y, norm(x.double().cpu().numpy(), 2, **rk)) <= 1e-5
        d = ssm.ssm_group_norm_bwd(x, 2, torch.ones_like(x), **kw)
        assert d["dx"].isfinite().all() and (d["dz"] is None or d["dz"].isfinite().all())
    y0 = ssm.ssm_group_norm_fwd(x, 2)
    x[3, 1, 70] = float("nan")
    y1 = ssm.ssm_group_norm_fwd(x, 2)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[3, 1, 64:] = True
    assert torch.equal(y1[~bad], y0[~bad]) and y1[bad].isnan().all()


def test_stream_and_graph():
    t, _ = make(BF16, (2, 70, 640), "gate", "both", seed=4)
    kw = dict(weight=t["weight"], bias=t["bias"], z=t["z"])

    def step():
        y = ssm.ssm_group_norm_fwd(t["x"], 5, **kw)
        return [y, *ssm.ssm_group_norm_bwd(t["x"], 5, t["dy"], **kw).values()]

    ref = [v.clone() for v in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = ssm.ssm_group_norm_fwd(t["x"], 5, stream=side, **kw)
    side.synchronize()
    assert torch.equal(y, ref[0])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for v in out:
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
        torch.randn(64, 64, device="cuda").sum().item()


def test_far_rows():
    """Rows behind 2^31 elements."""
    L, dim = 6, 128
    far = (1 << 31) + 128
    x = torch.empty(far + L * dim, dtype=BF16, device="cuda").as_strided((2, L, dim), (far, dim, 1))
    t, r = make(BF16, (2, L, dim), "none", "weight", seed=5)
    x.copy_(t["x"])
    assert error(ssm.ssm_group_norm_fwd(x, 2, weight=t["weight"], out_dtype=F32),
                 norm(r["x"], 2, weight=r["weight"])) <= 1e-5
