"""The residual norm on the GPU where it meets its caller: strides, results in
place, scales in any order, special values, far offsets, streams and graphs.
Tolerances are those of test_gpu_rms (derived there)."""
import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from heads_reference import rms_norm
from test_gpu_delta import error
from test_gpu_rms import BF16, E4M3, F32, FP32_ERROR, check_8bit, make, tolerance

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
bits = lambda t: t.view(torch.uint8) if t.dtype == E4M3 else t  # noqa: E731


@pytest.mark.parametrize("out", [F32, BF16, E4M3], ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("dim", [256, 1531, 2560, 9001])
def test_forward_strides(dim, out):
    """Slices of wider rows, also at offsets that no 16-byte access fits: right
    (narrower accesses add a row's squares in another order, so the last bits may
    differ from the dense call's; h, one addition, does not), and nothing is
    written beside them."""
    B, L = 3, 37
    t, r = make(BF16, (B, L, dim), F32, seed=dim)
    _, h0, _ = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], residual=t["residual"], out_dtype=out)
    ref = rms_norm(r["x"], r["weight"], r["residual"])[0]

    def wide(like, dtype, pad):
        w = torch.full((B, L, dim + 2 * pad), 7.0, dtype=F32, device="cuda").to(dtype)
        v = w[..., pad:pad + dim]
        if like is not None:
            v.copy_(like)
        return w, v
    for pad in (1, 8, 64):
        x, res = wide(t["x"], BF16, pad)[1], wide(t["residual"], F32, pad)[1]
        (ho, h), (yo, y) = wide(None, F32, pad), wide(None, out, pad)
        _, _, s = ssm.ssm_rms_norm_fwd(x, weight=t["weight"], residual=res, residual_out=h, y=y)
        assert torch.equal(h, h0)
        if out == E4M3:
            check_8bit(y, s, ref)
        else:
            assert error(y, ref) <= tolerance(out)
        for w in (ho, yo):
            assert (w[..., :pad].float() == 7).all() and (w[..., pad + dim:].float() == 7).all()
    # rows beside each other: x and the residual's slices of one buffer, y over x
    row = torch.cat([t["x"], t["x"]], -1)
    y, _, _ = ssm.ssm_rms_norm_fwd(row[..., :dim], weight=t["weight"], residual=t["residual"], y=row[..., dim:])
    assert torch.equal(row[..., :dim], t["x"]) and error(y, ref) <= tolerance(BF16)


@pytest.mark.parametrize("dim", [128, 776, 2560, 5120, 9001])
def test_scales_in_any_order(dim):
    B, L = 2, 19
    t, r = make(BF16, (B, L, dim), None, seed=dim)
    nb = -(-dim // 128)
    y0, _, s0 = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], out_dtype=E4M3)
    check_8bit(y0, s0, rms_norm(r["x"], r["weight"])[0])
    for order in ((2, 0, 1), (0, 2, 1), (1, 0, 2), (1, 2, 0)):
        s = torch.full([(B, L, nb)[i] for i in order], NAN, device="cuda").permute([order.index(i) for i in range(3)])
        y, _, _ = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], out_dtype=E4M3, scales=s)
        assert torch.equal(s, s0) and torch.equal(bits(y), bits(y0)), order
    padded = torch.full((B, L, nb + 3), 7.0, device="cuda")
    ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], out_dtype=E4M3, scales=padded[..., :nb])
    assert torch.equal(padded[..., :nb], s0) and (padded[..., nb:] == 7).all()


@pytest.mark.parametrize("dim", [100, 2560, 9000, 20001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(dtype, dim):
    t, _ = make(dtype, (2, 9, dim), dtype, seed=dim)
    w = t["weight"]
    y0, h0, _ = ssm.ssm_rms_norm_fwd(t["x"], weight=w, residual=t["residual"])
    y0 = y0.clone()
    for places in ("residual_out=residual", "residual_out=x", "y=x", "y=residual", "residual_out=residual y=x",
                   "residual_out=x y=residual"):
        x, res = t["x"].clone(), t["residual"].clone()
        kw = {a: {"x": x, "residual": res}[b] for a, b in (p.split("=") for p in places.split())}
        y, h, _ = ssm.ssm_rms_norm_fwd(x, weight=w, residual=res, **kw)
        assert torch.equal(y, y0) and torch.equal(h, h0), places
    d0 = ssm.ssm_rms_norm_bwd(h0, t["dy"], weight=w, dh=t["dh"])
    for places in ("dx=dy", "dresidual=dh", "dx=dy dresidual=dh"):
        dy, dh = t["dy"].clone(), t["dh"].clone()
        kw = {a: {"dy": dy, "dh": dh}[b] for a, b in (p.split("=") for p in places.split())}
        d = ssm.ssm_rms_norm_bwd(h0, dy, weight=w, dh=dh, **kw)
        assert all(torch.equal(d[n], d0[n]) for n in d0), places


@pytest.mark.parametrize("dim", [256, 1531, 9001])
@pytest.mark.parametrize("out", [F32, BF16, E4M3], ids=lambda t: str(t)[6:])
def test_special_rows(out, dim):
    """Zero rows, tiny ones, and rows that hold an infinity or a NaN, beside ordinary ones."""
    t, r = make(F32, (9, dim), None, seed=dim)
    x = t["x"]
    y0, _, s0 = ssm.ssm_rms_norm_fwd(x, weight=t["weight"], out_dtype=out)
    x[1], x[3], x[5] = 0.0, x[3] * 1e-30, x[5] * 1e-8
    x[2, dim // 2], x[4, 7], x[6, dim - 1] = NAN, INF, -INF
    y, _, s = ssm.ssm_rms_norm_fwd(x, weight=t["weight"], out_dtype=out)
    for i in (0, 7, 8):
        assert torch.equal(bits(y)[i], bits(y0)[i])
    real = np.asarray(x.double().cpu())[[1, 3, 5]]
    ref = rms_norm(real, r["weight"])[0]
    if out == E4M3:
        assert not y[1].float().any() and (s[1] == 2.0 ** -126).all()
        check_8bit(y[[1, 3, 5]], s[[1, 3, 5]], ref)
        assert s[2].isnan().all()
    else:
        assert not y[1].any() and error(y[3], ref[1]) <= tolerance(out) and error(y[5], ref[2]) <= tolerance(out)
        assert y[2].isnan().all()
        # h / inf is 0, inf / inf NaN: as the formula
        for i, c in ((4, 7), (6, dim - 1)):
            assert y[i, c].isnan() and not y[i, :7].any()


@pytest.mark.parametrize("dim", [256, 9001])
def test_8bit_blocks_with_infinities(dim):
    """An infinite weight: its block alone has an infinite scale."""
    t, _ = make(F32, (3, dim), None, seed=1)
    y0, _, s0 = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], out_dtype=E4M3)
    t["weight"][130] = INF
    y, _, s = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], out_dtype=E4M3)
    assert (s[:, 1] == INF).all()
    keep = [i for i in range(s.shape[1]) if i != 1]
    assert torch.equal(s[:, keep], s0[:, keep])
    rest = [c for c in range(dim) if c // 128 != 1]
    assert torch.equal(bits(y)[:, rest], bits(y0)[:, rest])


@pytest.mark.parametrize("dtype,stream", [(BF16, F32), (F32, BF16), (BF16, BF16)])
def test_stream_type_without_a_residual(dtype, stream):
    t, r = make(dtype, (2, 5, 300), None)
    y, h, _ = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], stream_dtype=stream)
    assert h.dtype == stream and torch.equal(h, t["x"].to(stream))
    assert error(y, rms_norm(r["x"], r["weight"])[0]) <= tolerance(dtype)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_eps(eps):
    t, r = make(F32, (4, 333), None)
    y, _, _ = ssm.ssm_rms_norm_fwd(t["x"], eps=eps)
    d = ssm.ssm_rms_norm_bwd(t["x"], t["dy"], eps=eps)
    y0, _, d0 = rms_norm(r["x"], eps=eps, dy=r["dy"])
    assert error(y, y0) <= FP32_ERROR and error(d["dx"], d0["dx"]) <= FP32_ERROR and d["dweight"] is None


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [96, 2560, 9001])
def test_gradient_strides(dim, dtype):
    B, L = 3, 21
    t, r = make(dtype, (B, L, dim), F32, seed=dim)
    d0 = rms_norm(r["residual"], r["weight"], None, dy=r["dy"], dh=r["dh"])[2]
    for pad in (1, 16):
        def wide(like):
            w = torch.full((B, L, dim + 2 * pad), NAN, dtype=like.dtype, device="cuda")
            w[..., pad:pad + dim].copy_(like)
            return w[..., pad:pad + dim]
        dx, dres = wide(torch.zeros_like(t["dy"])), wide(torch.zeros_like(t["dh"]))
        d = ssm.ssm_rms_norm_bwd(wide(t["residual"]), wide(t["dy"]), weight=t["weight"], dh=wide(t["dh"]), dx=dx,
                                 dresidual=dres)
        assert error(d["dx"], d0["dx"]) <= tolerance(dtype) and error(d["dresidual"], d0["dx"]) <= tolerance(F32)
        assert error(d["dweight"], d0["dweight"]) <= FP32_ERROR
        assert dx._base[..., :pad].isnan().all() and dres._base[..., pad + dim:].isnan().all()


def test_far_offsets():
    """Rows behind 2^31 elements, by the step stride and by the batch stride."""
    dim = 256
    t, _ = make(BF16, (3, dim), BF16)
    y0, h0, _ = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], residual=t["residual"])
    d0 = ssm.ssm_rms_norm_bwd(h0, t["dy"], weight=t["weight"], dh=t["dh"])
    far = (1 << 30) + 200
    for shape in ((3, 1), (1, 3)):
        def away(like=None):
            b = torch.empty(2 * far + dim, dtype=BF16, device="cuda")
            v = b.as_strided((*shape, dim), (far, far, 1) if shape[0] > 1 else (3 * far, far, 1))
            if like is not None:
                v.copy_(like.view(*shape, dim))
            return v
        y, h, _ = ssm.ssm_rms_norm_fwd(away(t["x"]), weight=t["weight"], residual=away(t["residual"]),
                                       residual_out=away(), y=away())
        assert torch.equal(y.reshape(3, dim), y0) and torch.equal(h.reshape(3, dim), h0)
        d = ssm.ssm_rms_norm_bwd(h, away(t["dy"]), weight=t["weight"], dh=away(t["dh"]), dx=away(), dresidual=away())
        assert torch.equal(d["dx"].reshape(3, dim), d0["dx"]) and torch.equal(d["dweight"], d0["dweight"])
        assert torch.equal(d["dresidual"].reshape(3, dim), d0["dresidual"])


def test_largest_row():
    """2^24 channels: the sum of squares in 2^24 terms, a tree of them."""
    dim = 1 << 24
    x = torch.randn(2, dim, device="cuda")
    dy = torch.randn(2, dim, device="cuda")
    y, _, _ = ssm.ssm_rms_norm_fwd(x)
    d = ssm.ssm_rms_norm_bwd(x, dy)
    x, dy = x.double(), dy.double()
    r = (x.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    assert error(y, (x * r).cpu()) <= FP32_ERROR
    assert error(d["dx"], (r * (dy - x * r * r * (x * dy).mean(-1, keepdim=True))).cpu()) <= FP32_ERROR


@pytest.mark.parametrize("dim", [256, 2560])
def test_many_rows(dim):
    """More rows than one sweep of the card takes: dweight in a fixed order, the same bits every time."""
    t, r = make(BF16, (2, 6000, dim), F32, seed=3)
    d = [ssm.ssm_rms_norm_bwd(t["residual"], t["dy"], weight=t["weight"], dh=t["dh"]) for _ in range(3)]
    d0 = rms_norm(r["residual"], r["weight"], None, dy=r["dy"], dh=r["dh"])[2]
    assert error(d[0]["dweight"], d0["dweight"]) <= FP32_ERROR and error(d[0]["dx"], d0["dx"]) <= tolerance(BF16)
    for e in d[1:]:
        assert all(torch.equal(e[n], d[0][n]) for n in e)


def test_stream_and_graph():
    t, _ = make(BF16, (2, 300, 2560), F32, seed=4)
    res = t["residual"].clone()

    def step():
        y, h, _ = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], residual=res, residual_out=res)
        q, _, s = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], out_dtype=E4M3)
        d = ssm.ssm_rms_norm_bwd(h, t["dy"], weight=t["weight"], dh=t["dh"])
        return [y, q.view(torch.uint8), s, *d.values()]

    ref = [x.clone() for x in step()] + [res.clone()]
    res.copy_(t["residual"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, _, _ = ssm.ssm_rms_norm_fwd(t["x"], weight=t["weight"], residual=t["residual"], stream=side)
    side.synchronize()
    assert torch.equal(y, ref[0])
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        res.copy_(t["residual"])
        for x in out:
            x.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip([*out, res], ref):
            assert torch.equal(got, want)
        torch.randn(64, 64, device="cuda").sum().item()


@pytest.mark.parametrize("rows,dim", [(2600, 9001), (1500, 16392), (1100, 20001), (40000, 512), (40000, 99)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_several_rows_a_workgroup(rows, dim, dtype):
    """More rows than are in work at once, for every way that a row is held."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    x, dy, dh, res = (torch.randn(rows, dim, device="cuda", generator=g).to(dtype) for _ in range(4))
    w = 1 + 0.1 * torch.randn(dim, device="cuda", generator=g)
    y, h, _ = ssm.ssm_rms_norm_fwd(x, weight=w, residual=res)
    d = ssm.ssm_rms_norm_bwd(h, dy, weight=w, dh=dh)

    def off(got, ref):
        size = torch.maximum(ref.abs(), ref.square().mean().sqrt())
        return float(((got.double() - ref).abs() / size).max())
    s = x.double() + res.double()
    assert off(y, s * (s.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w) <= tolerance(dtype)
    h, u = h.double(), dy.double() * w
    r = (h.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    assert off(d["dx"], r * (u - h * r * r * (u * h).mean(-1, keepdim=True)) + dh.double()) <= tolerance(dtype)
    # a sum of 4e4 rows in fp32: the threads' own chains of up to 40 rows, then a tree
    assert off(d["dweight"], (dy.double() * h * r).sum(0)) <= FP32_ERROR
