"""The head scan on the GPU where it meets its caller: strides, mixed types,
slots, far offsets, bounds, non-finite values, streams, graphs, states in place.
Tolerances are those of test_gpu_heads (derived there)."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from heads_reference import head_scan_batch
from test_gpu_delta import error
from test_gpu_heads import ARGS, BF16, F32, call, call_bwd, make, reference, tolerance

pytestmark = pytest.mark.gpu

NAN = float("nan")


def steps(t, i):
    return [t[n] if n == "A" else t[n][:, i] for n in ARGS]


@pytest.mark.parametrize("dtype,grad", [(F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("N,P", [(64, 72), (128, 64), (33, 20), (256, 40)])
def test_mixed_types(dtype, grad, N, P):
    """fp32 gradients of bf16 inputs and the other way round, with states kept by the forward call and without."""
    t, r, _ = make(dtype, [150], False, 1, 2, N, P)
    t["dy"], r["dy"] = t["dy"].to(grad), t["dy"].to(grad).double().cpu().numpy()
    y0, h0, d0 = reference(r, grads=True)
    ws = ssm.ssm_head_scan_bwd_workspace(t["x"], t["B"])
    y, _ = call(t, out_dtype=grad, checkpoints=ws)
    assert y.dtype == grad and error(y, y0) <= tolerance(dtype, grad)
    d, e = call_bwd(t, workspace=ws, checkpoints_in_workspace=True), call_bwd(t)
    for n in d0:
        assert torch.equal(d[n], e[n]), n
        assert error(d[n], d0[n]) <= tolerance(dtype, d[n].dtype, n), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("order", ["projection", "heads_first", "time_major", "odd"])
@pytest.mark.parametrize("N,P", [(64, 72), (128, 64)])
def test_strides(order, dtype, N, P):
    """Slices of one conv output, [batch, heads, L, .] and [L, batch, ..] tensors and
    rows that no 16-byte access fits give the dense call's bits."""
    B, L, g, h = 2, 150, 2, 4
    t, _, _ = make(dtype, [L] * B, False, g, h, N, P, seed=5)
    y0, h0 = call(t)
    d0 = call_bwd(t)
    u = dict(t)
    if order in ("heads_first", "time_major"):
        a, b = (1, 2) if order == "heads_first" else (0, 1)
        move = lambda x: x.transpose(a, b).contiguous().transpose(a, b)  # noqa: E731
        for n in ("x", "dt", "B", "C", "dy"):
            u[n] = move(t[n])
        y = move(torch.full_like(t["x"], NAN))
        kw = {n: move(torch.full_like(t[m], NAN)) for n, m in (("dx", "x"), ("ddt", "dt"), ("dBm", "B"), ("dCm", "C"))}
    else:
        pad = 3 if order == "odd" else 0
        sizes = [h * P, g * N, g * N]
        row = torch.full((B, L, sum(sizes) + pad), NAN, dtype=dtype, device="cuda")
        out, at, kw = torch.full_like(row, NAN), pad, {}
        for n, d, size in zip(("x", "B", "C"), ("dx", "dBm", "dCm"), sizes):
            u[n] = row[..., at:at + size].unflatten(-1, t[n].shape[2:])
            u[n].copy_(t[n])
            kw[d] = out[..., at:at + size].unflatten(-1, t[n].shape[2:])
            at += size
        wide = torch.full((B, L, 2 * h + 1), NAN, dtype=dtype, device="cuda")
        u["dt"] = wide[..., 1:h + 1]
        u["dt"].copy_(t["dt"])
        kw["ddt"] = wide[..., h + 1:]
        u["dy"] = torch.full((B, L, h, P + 1), NAN, dtype=dtype, device="cuda")[..., :P] if order == "odd" else t["dy"]
        u["dy"].copy_(t["dy"])
        y = torch.empty(B, L, h, P + 5, dtype=dtype, device="cuda")[..., 5:]
    ws = ssm.ssm_head_scan_bwd_workspace(u["x"], u["B"])
    y1, h1 = call(u, y=y, checkpoints=ws)
    assert torch.equal(y1, y0) and torch.equal(h1, h0)
    d1 = call_bwd(u, workspace=ws, checkpoints_in_workspace=True, **kw)
    for n in d0:
        assert torch.equal(d1[n], d0[n]), n
    if order in ("projection", "odd"):  # nothing between the slices is written
        assert out[..., :pad].isnan().all() and wide[..., 0].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_update_strides(dtype):
    """One token's slices of a projection row, in and out."""
    B, g, h, N, P = 5, 2, 4, 64, 40
    t, _, _ = make(dtype, [1] * B, False, g, h, N, P, seed=2)
    s0, s1 = t["h0"].clone(), t["h0"].clone()
    kw = dict(Dskip=t["D"], dt_bias=t["bias"])
    y0 = ssm.ssm_head_scan_update(s0, *steps(t, 0), **kw)
    row = torch.full((B, 2 * h * P + 2 * g * N + h + 1), NAN, dtype=dtype, device="cuda")
    parts, at = [], 1
    for n, size in (("x", h * P), ("dt", h), ("B", g * N), ("C", g * N)):
        v = row[:, at:at + size]
        v = v if n == "dt" else v.unflatten(-1, t[n].shape[2:])
        v.copy_(t[n][:, 0])
        parts.append(v)
        at += size
    y = row[:, at:].unflatten(-1, (h, P))
    ssm.ssm_head_scan_update(s1, parts[0], parts[1], t["A"], parts[2], parts[3], y=y, **kw)
    assert torch.equal(y, y0) and torch.equal(s1, s0) and row[:, 0].isnan().all()


def test_update_slots():
    """States in a pool; skipped rows leave every state alone and answer zero."""
    batch, g, h, N, P = 6, 2, 4, 64, 48
    t, r, _ = make(BF16, [1] * batch, False, g, h, N, P, seed=1)
    pool = torch.randn(9, h, N, P, device="cuda")
    at = [7, -1, 0, 9, 3, 1 << 30]
    before = pool.clone()
    y = ssm.ssm_head_scan_update(pool, *steps(t, 0), Dskip=t["D"], dt_bias=t["bias"], out_dtype=F32,
                                 slots=torch.tensor(at, dtype=torch.int32, device="cuda"))
    live = [b for b, s in enumerate(at) if 0 <= s < 9]
    r["h0"] = np.stack([before[at[b] if b in live else 0].double().cpu().numpy() for b in range(batch)])
    y0, h1 = reference(r)
    for b in range(batch):
        if b in live:
            assert error(y[b], y0[b, 0]) <= 2e-5 and error(pool[at[b]], h1[b]) <= 2e-5
        else:
            assert not y[b].any()
    rest = [s for s in range(9) if s not in at]
    assert torch.equal(pool[rest], before[rest])


def test_update_far_slot():
    """A state behind 2^31 elements of the pool."""
    h, N, P = 16, 128, 128
    slots = (1 << 31) // (h * N * P) + 3
    pool = torch.empty(slots, h, N, P, device="cuda")
    t, r, _ = make(BF16, [1], False, h, h, N, P)
    pool[-1].copy_(t["h0"][0])
    y = ssm.ssm_head_scan_update(pool, *steps(t, 0), Dskip=t["D"], dt_bias=t["bias"], out_dtype=F32,
                                 slots=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    y0, h0 = reference(r)
    assert error(y, y0[:, 0]) <= 2e-5 and error(pool[-1:], h0) <= 2e-5


@pytest.mark.parametrize("index", ["batch", "step", "head"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_offsets(dtype, index):
    """Elements behind 2^31 of the tensors, by each of the strides."""
    L, h, N, P = 70, 2, 64, 64
    B = 2 if index == "batch" else 1
    t, _, _ = make(dtype, [L] * B, False, h, h, N, P, seed=8)
    strides = {"batch": ((1 << 31) + 64, h * 64, 64, 1), "step": (70 << 25, 1 << 25, 64, 1),
               "head": (1 << 40, 64, (1 << 31) + 64, 1)}[index]
    size = 1 + sum((n - 1) * s for n, s in zip((B, L, h, 64), strides))

    def far():
        return torch.empty(size, dtype=dtype, device="cuda").as_strided((B, L, h, 64), strides)
    u = dict(t)
    for n in ("x", "B", "C"):
        u[n] = far()
        u[n].copy_(t[n])
    y0, h0 = call(t)
    y1, h1 = call(u, y=far())
    assert torch.equal(y1, y0) and torch.equal(h1, h0)
    d0 = call_bwd(t)
    d1 = call_bwd(u, dx=far(), dBm=far(), dCm=far())
    for n in d0:
        assert torch.equal(d1[n], d0[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_clamped_bounds(dtype):
    """Bounds outside the tensors are clamped; covered steps are right, others are not written."""
    t, r, _ = make(dtype, [100], False, 1, 2, 32, 16, seed=4, state=False)
    cu = torch.tensor([-7, 40, 90], dtype=torch.int32, device="cuda")
    y, dx = (torch.full((1, 100, 2, 16), 7.0, device="cuda", dtype=dtype) for _ in "yx")
    ddt = torch.full((1, 100, 2), 7.0, device="cuda", dtype=dtype)
    dB, dC = (torch.full((1, 100, 1, 32), 7.0, device="cuda", dtype=dtype) for _ in "BC")
    _, hL = call(t, cu, y=y)
    d = call_bwd(t, cu, dx=dx, ddt=ddt, dBm=dB, dCm=dC)
    cut = {n: v[:, :90] if n in ("x", "dt", "B", "C", "dy") else v for n, v in r.items()}
    cut["dhL"] = np.zeros((2, 2, 32, 16))
    y0, h0, d0 = reference(cut, [40, 50], grads=True)
    assert error(y[:, :90], y0) <= tolerance(dtype, dtype) and error(hL, h0) <= tolerance(dtype, F32, "hL")
    assert (y[:, 90:] == 7.0).all()
    for n in d0:
        got = d[n]
        if n in ("dx", "ddt", "dBm", "dCm"):
            assert (got[:, 90:] == 7.0).all(), n
            got = got[:, :90]
        assert error(got, d0[n]) <= tolerance(dtype, got.dtype, n), n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nonfinite_stays_in_its_sequence_and_head(dtype):
    lens = [70, 5, 100, 64]
    t, _, cu = make(dtype, lens, True, 2, 4, 64, 64, seed=6)
    y0, h0 = call(t, cu)
    d0 = call_bwd(t, cu)
    t["x"][0, 71, 1] = NAN
    t["x"][0, 145, 3, 2] = float("inf")
    t["dt"][0, 180, 0] = NAN
    y1, h1 = call(t, cu)
    d1 = call_bwd(t, cu)
    same = torch.ones(239, 4, dtype=torch.bool, device="cuda")
    same[70:75, 1] = False
    same[75:175, 3] = False
    same[175:, 0] = False
    clean = same.clone()
    clean[75:139, 3] = True  # the chunk before the infinity
    assert torch.equal(y1[0][clean], y0[0][clean])
    assert y1[0, 71, 1].isnan().all() and not y1[0, 145, 3, 2].isfinite() and y1[0, 180, 0].isnan().all()
    keep = torch.ones(4, 4, dtype=torch.bool)
    keep[1, 1] = keep[2, 3] = keep[3, 0] = False
    assert torch.equal(h1[keep], h0[keep]) and torch.equal(d1["dh0"][keep], d0["dh0"][keep])
    for n in ("dx", "ddt"):
        assert torch.equal(d1[n][0][same], d0[n][0][same]), n
    for n in ("dBm", "dCm"):  # a group's heads are 0, 1 and 2, 3
        both = same.unflatten(1, (2, 2)).all(2)
        assert torch.equal(d1[n][0][both], d0[n][0][both]), n
    assert torch.equal(d1["dA"][2], d0["dA"][2]) and torch.equal(d1["dDskip"][2], d0["dDskip"][2])
    # a non-finite readout stays in its group too
    t["x"].nan_to_num_(0.0, 0.0, 0.0)
    t["dt"].nan_to_num_(0.0)
    y0, h0 = call(t, cu)
    t["C"][0, 100, 1, 7] = float("-inf")
    y1, h1 = call(t, cu)
    assert torch.equal(y1[0, :, :2], y0[0, :, :2]) and torch.equal(h1[:, :2], h0[:, :2])
    assert torch.equal(h1[2], h0[2]) and not y1[0, 100, 2:].isfinite().any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_growth_and_extreme_steps(dtype):
    """A > 0, steps that forget everything at once, and steps too small to move the state."""
    t, r, _ = make(dtype, [140], False, 1, 4, 32, 24, seed=11)
    A = np.array([0.02, -1e4, -1e-6, -3.0])
    bias = np.array([-3.0, 6.0, -60.0, 0.5])
    for n, v in (("A", A), ("bias", bias)):
        t[n] = torch.tensor(v, dtype=F32, device="cuda")
        r[n] = t[n].double().cpu().numpy()
    dt = r["dt"].copy()
    dt[:, ::17, 3] = 1e4   # softplus(u) = u
    dt[:, 5::31, 3] = -1e4  # softplus(u) = 0
    t["dt"] = torch.tensor(dt, device="cuda").to(dtype)
    r["dt"] = t["dt"].double().cpu().numpy()
    y0, h0, d0 = reference(r, grads=True)
    y, hL = call(t)
    d = call_bwd(t)
    for k in range(4):  # each against its own size
        assert error(y[:, :, k], y0[:, :, k]) <= tolerance(dtype, dtype), k
        assert error(hL[:, k], h0[:, k]) <= tolerance(dtype, F32, "hL"), k
        for n in ("dx", "ddt"):
            assert error(d[n][:, :, k], d0[n][:, :, k]) <= tolerance(dtype, dtype, n), (n, k)
        assert error(d["dh0"][:, k], d0["dh0"][:, k]) <= tolerance(dtype, F32, "dh0"), k
    for n in ("dBm", "dCm"):
        assert error(d[n], d0[n]) <= tolerance(dtype, dtype, n), n


@pytest.mark.parametrize("lens,packed", [([100, 100], False), ([1500], False), ([700, 0, 900, 65], True)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_states_in_place(dtype, lens, packed):
    """hL in h0's place and dh0 in dhL's, whole sequences and cut ones: the bits of separate arrays."""
    t, _, cu = make(dtype, lens, packed, 1, 2, 64, 40, seed=12)
    y0, h0 = call(t, cu)
    d0 = call_bwd(t, cu)
    state = t["h0"].clone()
    y, hL = ssm.ssm_head_scan_fwd(*(t[n] for n in ARGS), Dskip=t["D"], dt_bias=t["bias"], h0=state, hL=state, cu_seqlens=cu)
    assert hL is state and torch.equal(hL, h0) and torch.equal(y, y0)
    ws = ssm.ssm_head_scan_bwd_workspace(t["x"], t["B"], cu_seqlens=cu)
    like = lambda n: torch.full_like(t[n], NAN)  # noqa: E731
    out = {"dx": like("x"), "ddt": like("dt"), "ddt_bias": like("bias"), "dA": like("A"), "dBm": like("B"),
           "dCm": like("C"), "dDskip": like("D"), "dh0": t["dhL"].clone()}
    p = lambda x: 0 if x is None else x.data_ptr()  # noqa: E731
    B, L, h, P = t["x"].shape
    code = ssm.SSM_F32 if dtype == F32 else ssm.SSM_BF16
    status = ssm.lib().ssm_head_scan_bwd(
        B, L, 1, h, 64, P, code, 0, p(t["x"]), p(t["dt"]), p(t["bias"]), p(t["A"]), p(t["B"]), p(t["C"]), p(t["D"]),
        p(t["h0"]), p(cu), len(lens) if packed else 0, code, p(t["dy"]), p(out["dh0"]), *(p(o) for o in out.values()),
        p(ws), ws.numel(), None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0
    for n in d0:
        assert torch.equal(out[n], d0[n]), n


def test_optional_outputs():
    """No final state, no dDskip and no ddt_bias: what is returned keeps its bits."""
    t, _, _ = make(BF16, [200], False, 1, 2, 64, 64, seed=13)
    y0, _ = call(t)
    y1, none = call(t, return_final_state=False)
    assert none is None and torch.equal(y1, y0)
    d0 = call_bwd(t)
    t["dhL"] = None
    d1 = call_bwd(t)
    t["dhL"] = torch.zeros_like(t["h0"])
    d2 = call_bwd(t)
    for n in d0:
        assert torch.equal(d1[n], d2[n]), n


@pytest.mark.parametrize("lens,packed", [([130, 130], False), ([1500], False), ([700, 0, 900, 65], True)])
def test_checkpoints_stay(lens, packed):
    """Two backward calls on one workspace that the forward call filled."""
    t, _, cu = make(BF16, lens, packed, 1, 2, 64, 40, seed=16)
    ws = ssm.ssm_head_scan_bwd_workspace(t["x"], t["B"], cu_seqlens=cu)
    call(t, cu, checkpoints=ws)
    first, second = (call_bwd(t, cu, workspace=ws, checkpoints_in_workspace=True) for _ in range(2))
    for n in first:
        assert torch.equal(first[n], second[n]), n


@pytest.mark.parametrize("batch,N,P", [(3, 20, 64), (2, 64, 128), (3, 100, 64), (2, 256, 64), (1, 200, 192)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_update_tiles_of_64(dtype, batch, N, P):
    """The decode step's wide tiles for every number of state rows, and what lies beside a state."""
    t, r, _ = make(dtype, [1] * batch, False, 2, 4, N, P, seed=N)
    y0, h0 = reference(r)
    pool = torch.full((batch + 2, 4, N, P), 7.0, device="cuda")
    pool[1:-1].copy_(t["h0"])
    y = ssm.ssm_head_scan_update(pool[1:-1], *steps(t, 0), Dskip=t["D"], dt_bias=t["bias"])
    assert error(y, y0[:, 0]) <= tolerance(F32, dtype) and error(pool[1:-1], h0) <= tolerance(F32, F32)
    assert (pool[0] == 7).all() and (pool[-1] == 7).all()


def test_stream_and_graph():
    """On another stream than the inputs', and captured: every replay gives the eager bits."""
    lens = [130, 0, 65, 1, 700]
    t, _, cu = make(BF16, lens, True, 2, 4, 64, 64, seed=9)
    state = t["h0"].clone()
    one = [t[n] if n == "A" else t[n][0, :5] for n in ARGS]

    def step():
        ws = ssm.ssm_head_scan_bwd_workspace(t["x"], t["B"], cu_seqlens=cu)
        y, hL = call(t, cu, checkpoints=ws)
        z, _ = call(t, cu)
        d = call_bwd(t, cu, workspace=ws, checkpoints_in_workspace=True)
        u = ssm.ssm_head_scan_update(state, *one, Dskip=t["D"], dt_bias=t["bias"])
        return [y, hL, z, u, *d.values()]

    ref = [x.clone() for x in step()]
    state.copy_(t["h0"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, hL = call(t, cu, stream=side)
    side.synchronize()
    assert torch.equal(y, ref[0]) and torch.equal(hL, ref[1])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        state.copy_(t["h0"])
        for x in out:
            x.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, ref):
            assert torch.equal(got, want)
        torch.randn(64, 64, device="cuda").sum().item()


def test_two_calls_at_once():
    """Two streams, each with its own workspace: the bits of one call behind the other."""
    t, _, _ = make(BF16, [1500], False, 1, 2, 64, 64, seed=14)
    u, _, _ = make(BF16, [1500], False, 1, 2, 64, 64, seed=15)
    want = [(call(v), call_bwd(v)) for v in (t, u)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(call(v, stream=s), call_bwd(v, stream=s)) for v, s in zip((t, u), sides)]
    torch.cuda.synchronize()
    for (a, d), (b, e) in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert all(torch.equal(d[n], e[n]) for n in d)


def test_layer_in_full():
    """A layer's 80 heads of 128 x 64 with one group over 2048 steps against the
    recurrence, two of its heads (dB and dC, which sum over all 80, against one
    head's with the others' x and dy at zero)."""
    t, r, _ = make(BF16, [2048], False, 1, 80, 128, 64, seed=2, state=False)
    y, hL = call(t, out_dtype=F32)
    d = call_bwd(t)
    for h in (0, 79):
        one = {n: v if v is None or n in ("B", "C") else v[h:h + 1] if n in ("A", "D", "bias") else v[:, :, h:h + 1]
               for n, v in r.items()}
        y0, h0, d0 = head_scan_batch(*(one[n] for n in ARGS), one["D"], one["bias"], None, None, one["dy"])
        assert error(y[:, :, h:h + 1], y0) <= tolerance(BF16, F32)
        assert error(hL[:, h:h + 1], h0) <= tolerance(BF16, F32, "hL")
        for n in ("dx", "ddt"):
            assert error(d[n][:, :, h:h + 1], d0[n]) <= tolerance(BF16, BF16, n), n
        u = dict(t, x=torch.zeros_like(t["x"]), dy=torch.zeros_like(t["dy"]))
        u["x"][:, :, h], u["dy"][:, :, h] = t["x"][:, :, h], t["dy"][:, :, h]
        e = call_bwd(u)
        for n in ("dBm", "dCm"):
            assert error(e[n], d0[n]) <= tolerance(BF16, BF16, n), n
