"""Refusals and size rules of the head scan and the residual norm (CPU: every
call here fails validation, device pointers are never followed), the binding's
own checks, and the plain references' gradients against differences."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from heads_reference import head_scan, rms_norm

F32, BF16, E4M3 = ssm.SSM_F32, ssm.SSM_BF16, ssm.SSM_E4M3
NULL, SHAPE, DTYPE, MISALIGNED, ALIAS, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 6, 7

NAMES = ["x", "dt", "bias", "A", "B", "C", "D", "h0", "cu", "y", "hL", "ws", "dy", "dhL", "dx", "ddt", "dbias", "dA",
         "dB", "dC", "dD", "dh0", "state", "slots", "residual", "weight", "residual_out", "scales", "h", "dh",
         "dresidual", "dweight"]
P = {n: 0x100000000 * (i + 1) for i, n in enumerate(NAMES)}


def scan(which, **over):
    a = dict(P, batch=2, L=100, g=2, heads=4, N=64, P=48, dtype=BF16, flags=0, nseq=0, out=BF16, wsb=1 << 40,
             layout=None, cu=None, num_slots=2)
    a.update(over)
    sizes = (a["batch"], a["L"], a["g"], a["heads"], a["N"], a["P"], a["dtype"])
    inputs = (a["x"], a["dt"], a["bias"], a["A"], a["B"], a["C"], a["D"])
    rest = (a["h0"], a["cu"], a["nseq"], a["out"])
    if which == "fwd":
        return ssm.lib().ssm_head_scan_fwd(*sizes, a["flags"], *inputs, *rest, a["y"], a["hL"], a["ws"], a["wsb"],
                                           a["layout"], None)
    if which == "bwd":
        return ssm.lib().ssm_head_scan_bwd(*sizes, a["flags"], *inputs, *rest, a["dy"], a["dhL"], a["dx"], a["ddt"],
                                           a["dbias"], a["dA"], a["dB"], a["dC"], a["dD"], a["dh0"], a["ws"], a["wsb"],
                                           a["layout"], None)
    return ssm.lib().ssm_head_scan_update(a["batch"], *sizes[2:], a["state"], a["num_slots"], a["slots"], *inputs,
                                          a["out"], a["y"], a["layout"], None)


def layout(cls, **at):
    lay = cls()
    for field, entries in at.items():
        if isinstance(entries, dict):
            for i, v in entries.items():
                getattr(lay, field)[i] = v
        else:
            setattr(lay, field, entries)
    return ctypes.byref(lay)


SHARED = ([({n: None}, NULL) for n in ("x", "dt", "A", "B", "C")] + [
    (dict(dtype=2), DTYPE), (dict(dtype=7), DTYPE), (dict(out=-1), DTYPE), (dict(out=E4M3), DTYPE),
    (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(g=0), SHAPE), (dict(g=3), SHAPE), (dict(heads=1), SHAPE),
    (dict(heads=65536), SHAPE), (dict(N=0), SHAPE), (dict(N=257), SHAPE), (dict(P=0), SHAPE), (dict(P=65537), SHAPE),
    (dict(x=P["x"] + 1), MISALIGNED), (dict(dt=P["dt"] + 1), MISALIGNED), (dict(A=P["A"] + 2), MISALIGNED),
    (dict(bias=P["bias"] + 2), MISALIGNED), (dict(D=P["D"] + 1), MISALIGNED)])
SEQUENCES = [
    (dict(L=0), SHAPE), (dict(L=(1 << 28) - 4095), SHAPE), (dict(cu=P["cu"]), SHAPE), (dict(nseq=3), SHAPE),
    (dict(cu=P["cu"], nseq=3), SHAPE),  # packed sequences lie in one batch row
    (dict(flags=4), UNSUPPORTED), (dict(flags=1), UNSUPPORTED), (dict(h0=P["h0"] + 2), MISALIGNED),
    (dict(batch=1, L=4096, wsb=16), WORKSPACE), (dict(batch=1, L=4096, ws=P["ws"] + 8), MISALIGNED),
    (dict(batch=1, L=4096, ws=P["x"]), ALIAS), (dict(batch=1, L=4096, cu=P["ws"] + 4, nseq=3), ALIAS),
    (dict(batch=65535, L=1 << 27, heads=65535, g=1, N=256, P=65536), SHAPE)]
FWD = SHARED + SEQUENCES + [
    (dict(y=None), NULL), (dict(flags=2, ws=None), NULL), (dict(y=P["y"] + 1), MISALIGNED), (dict(y=P["x"]), ALIAS),
    (dict(y=P["C"] + 64), ALIAS), (dict(y=P["A"] - 8), ALIAS), (dict(hL=P["h0"] + 16), ALIAS), (dict(hL=P["y"]), ALIAS),
    (dict(hL=P["D"]), ALIAS), (dict(batch=1, L=4096, ws=None), WORKSPACE), (dict(flags=2, wsb=16), WORKSPACE),
    (dict(layout=layout(ssm.HeadScanLayout, step={0: -1})), SHAPE),
    (dict(layout=layout(ssm.HeadScanLayout, step={0: 48})), SHAPE),       # two heads of 48 share a place
    (dict(layout=layout(ssm.HeadScanLayout, head={2: 63})), SHAPE),
    (dict(layout=layout(ssm.HeadScanLayout, batch={1: 399})), SHAPE),
    (dict(layout=layout(ssm.HeadScanLayout, batch={4: 1 << 56})), SHAPE)]
BWD = SHARED + SEQUENCES + [({n: None}, NULL) for n in ("dy", "dx", "ddt", "dA", "dB", "dC", "ws")] + [
    (dict(dB=P["dB"] + 1), MISALIGNED), (dict(dA=P["dA"] + 2), MISALIGNED), (dict(dx=P["dB"]), ALIAS),
    (dict(dC=P["x"]), ALIAS), (dict(dh0=P["dhL"] + 4), ALIAS), (dict(ddt=P["dbias"]), ALIAS), (dict(dD=P["dA"]), ALIAS),
    (dict(dh0=P["ws"]), ALIAS), (dict(wsb=16), WORKSPACE),
    (dict(layout=layout(ssm.HeadScanBwdLayout, step={8: 100})), SHAPE)]
UPDATE = SHARED + [
    (dict(state=None), NULL), (dict(y=None), NULL), (dict(num_slots=0), SHAPE), (dict(slots=None, num_slots=3), SHAPE),
    (dict(state=P["state"] + 4), MISALIGNED), (dict(slots=P["slots"] + 2), MISALIGNED), (dict(y=P["state"]), ALIAS),
    (dict(y=P["B"]), ALIAS), (dict(state=P["x"]), ALIAS), (dict(slots=P["state"] + 16), ALIAS),
    (dict(state=P["A"]), ALIAS)]


@pytest.mark.parametrize("which,over,status", [("fwd", *c) for c in FWD] + [("bwd", *c) for c in BWD]
                         + [("update", *c) for c in UPDATE], ids=str)
def test_head_scan_refusals(which, over, status):
    assert scan(which, **over) == status


def test_head_scan_workspace_sizes():
    fwd, bwd = ssm.lib().ssm_head_scan_fwd_workspace_bytes, ssm.lib().ssm_head_scan_bwd_workspace_bytes
    for f in (fwd, bwd):
        for bad in ((0, 64, 1, 1, 64, 64, 0), (1, 64, 2, 3, 64, 64, 0), (1, 64, 1, 1, 257, 64, 0), (2, 64, 1, 1, 64, 64, 1),
                    (1, 64, 1, 1, 64, 65537, 0), (1, 64, 1, 1, 64, 64, -1)):
            assert f(*bad) == 0
    assert fwd(4, 2048, 1, 80, 128, 64, 0) == 0  # the card is full: no split
    assert fwd(1, 65521, 1, 24, 128, 64, 0) > 0
    # the states of every chunk, twice, and the sums
    assert bwd(4, 2048, 1, 80, 128, 64, 0) >= 2 * 4 * 128 * 80 * 128 * 64
    # room for a chunk that every packed sequence may end in
    assert bwd(1, 1000, 1, 2, 64, 64, 40) >= 2 * 4 * (16 + 40) * 2 * 64 * 64


def norm(which, **over):
    a = dict(P, batch=2, L=50, dim=256, dtype=BF16, stream=F32, out=BF16, wsb=1 << 40, layout=None)
    if over.get("out", a["out"]) != E4M3 and "scales" not in over:
        a["scales"] = None
    a.update(over)
    if which == "fwd":
        return ssm.lib().ssm_rms_norm_fwd(a["batch"], a["L"], a["dim"], a["dtype"], a["stream"], None, a["x"],
                                          a["residual"], a["weight"], a["residual_out"], a["out"], a["y"], a["scales"],
                                          a["layout"], None)
    return ssm.lib().ssm_rms_norm_bwd(a["batch"], a["L"], a["dim"], a["stream"], a["dtype"], None, a["h"], a["weight"],
                                      a["dy"], a["dh"], a["dx"], a["dresidual"], a["dweight"], a["ws"], a["wsb"],
                                      a["layout"], None)


BOTH = [(dict(dtype=2), DTYPE), (dict(stream=2), DTYPE), (dict(batch=0), SHAPE), (dict(L=0), SHAPE), (dict(dim=0), SHAPE),
        (dict(dim=(1 << 24) + 1), SHAPE), (dict(batch=1 << 16, L=1 << 15), SHAPE), (dict(weight=P["weight"] + 2), MISALIGNED)]
NORM = BOTH + [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(out=E4M3, scales=None), NULL), (dict(out=3), DTYPE),
    (dict(scales=P["scales"]), UNSUPPORTED), (dict(x=P["x"] + 1), MISALIGNED), (dict(residual=P["residual"] + 2), MISALIGNED),
    (dict(out=E4M3, scales=P["scales"] + 1), MISALIGNED), (dict(y=P["x"] + 16), ALIAS), (dict(y=P["residual"]), ALIAS),
    (dict(y=P["residual_out"]), ALIAS), (dict(residual_out=P["x"]), ALIAS), (dict(residual_out=P["residual"] + 4), ALIAS),
    (dict(out=E4M3, scales=P["y"]), ALIAS), (dict(out=E4M3, scales=P["x"]), ALIAS), (dict(out=E4M3, y=P["x"]), ALIAS),
    (dict(y=P["weight"] + 64), ALIAS),
    (dict(layout=layout(ssm.RmsLayout, step={0: 255})), SHAPE), (dict(layout=layout(ssm.RmsLayout, batch={3: 12799})), SHAPE),
    (dict(layout=layout(ssm.RmsLayout, step={1: -1})), SHAPE),
    (dict(out=E4M3, layout=layout(ssm.RmsLayout, scale_step=1)), SHAPE),          # two blocks share a place
    (dict(out=E4M3, layout=layout(ssm.RmsLayout, scale_block=-1)), SHAPE)]
NORM_BWD = BOTH + [
    (dict(h=None), NULL), (dict(dy=None), NULL), (dict(dx=None, dresidual=None), NULL), (dict(ws=None), WORKSPACE),
    (dict(wsb=16), WORKSPACE), (dict(ws=P["ws"] + 8), MISALIGNED), (dict(dy=P["dy"] + 1), MISALIGNED),
    (dict(dx=P["h"]), ALIAS), (dict(dx=P["dy"] + 16), ALIAS), (dict(dresidual=P["dh"] + 4), ALIAS),
    (dict(dresidual=P["dx"]), ALIAS), (dict(dweight=P["weight"]), ALIAS), (dict(ws=P["dx"]), ALIAS),
    (dict(dresidual=P["h"]), ALIAS), (dict(layout=layout(ssm.RmsBwdLayout, step={4: 10})), SHAPE)]


@pytest.mark.parametrize("which,over,status", [("fwd", *c) for c in NORM] + [("bwd", *c) for c in NORM_BWD], ids=str)
def test_rms_norm_refusals(which, over, status):
    assert norm(which, **over) == status


def test_rms_norm_workspace_sizes():
    f = ssm.lib().ssm_rms_norm_bwd_workspace_bytes
    assert f(0, 1, 8) == f(1, 0, 8) == f(1, 1, 0) == f(1 << 16, 1 << 15, 8) == f(1, 1, (1 << 24) + 1) == 0
    assert f(1, 1, 100) == 400 and f(4, 2048, 2560) >= 4 * 2560


@pytest.mark.parametrize("name,bad,error", [
    ("expanded x", dict(x=torch.empty(1, 1, 2, 8).expand(1, 9, 2, 8)), ValueError),
    ("CPU tensors", {}, TypeError),
    ("another type", dict(Bm=torch.empty(1, 9, 1, 16, dtype=torch.bfloat16)), TypeError),
    ("another shape", dict(Cm=torch.empty(1, 9, 1, 17)), ValueError),
    ("dt of another length", dict(dt=torch.empty(1, 8, 2)), ValueError),
    ("rows apart", dict(x=torch.empty(1, 9, 2, 16)[..., ::2]), ValueError),
    ("no tensor", dict(A=[1.0, 2.0]), TypeError),
    ("three dimensions", dict(x=torch.empty(9, 2, 8)), ValueError)])
def test_head_scan_binding_refusals(name, bad, error):
    a = dict(x=torch.empty(1, 9, 2, 8), dt=torch.empty(1, 9, 2), A=torch.empty(2), Bm=torch.empty(1, 9, 1, 16),
             Cm=torch.empty(1, 9, 1, 16))
    a.update(bad)
    with pytest.raises(error):
        ssm.ssm_head_scan_fwd(**a)
    with pytest.raises(error):
        ssm.ssm_head_scan_bwd(**a, dy=torch.empty(1, 9, 2, 8))


@pytest.mark.parametrize("name,bad,error", [
    ("CPU tensors", {}, TypeError), ("expanded", dict(x=torch.empty(1, 8).expand(3, 8)), ValueError),
    ("another shape", dict(residual=torch.empty(3, 9)), ValueError),
    ("scales of a type without them", dict(scales=torch.empty(3, 1)), ValueError),
    ("another scale shape", dict(out_dtype=torch.float8_e4m3fn, scales=torch.empty(3, 2)), ValueError),
    ("an integer type", dict(out_dtype=torch.int8), TypeError)])
def test_rms_norm_binding_refusals(name, bad, error):
    with pytest.raises(error):
        ssm.ssm_rms_norm_fwd(**{**dict(x=torch.empty(3, 8)), **bad})


def differences(f, args, at, eps=1e-6):
    """df / d args[at[0]][at[1]] by central differences."""
    up, down = [a.copy() for a in args], [a.copy() for a in args]
    up[at[0]][at[1]] += eps
    down[at[0]][at[1]] -= eps
    return (f(*up) - f(*down)) / (2 * eps)


def test_reference_head_scan_gradients_against_differences():
    rng = np.random.default_rng(0)
    n = rng.standard_normal
    L, g, h, N, V = 7, 2, 4, 3, 5
    args = [n((L, h, V)), n((L, h)), -rng.uniform(0.5, 2, h), n((L, g, N)), n((L, g, N)), n(h), n(h), n((h, N, V))]
    dy, dhL = n((L, h, V)), n((h, N, V))

    def loss(x, dt, A, B, C, D, bias, h0):
        y, hL = head_scan(x, dt, A, B, C, D, bias, h0)
        return (dy * y).sum() + (dhL * hL).sum()

    d = head_scan(*args, dy=dy, dhL=dhL)[2]
    for i, name in enumerate(("dx", "ddt", "dA", "dBm", "dCm", "dDskip", "ddt_bias", "dh0")):
        for _ in range(4):
            at = tuple(rng.integers(0, s) for s in args[i].shape)
            # central differences are off by eps^2 of the third derivative and 1e-16 / eps of the sum
            assert abs(differences(loss, args, (i, at)) - d[name][at]) <= 1e-7 * max(1, np.abs(d[name]).max())


def test_reference_rms_norm_gradients_against_differences():
    rng = np.random.default_rng(1)
    args, dy, dh = [rng.standard_normal((3, 9)), rng.standard_normal(9)], rng.standard_normal((3, 9)), rng.standard_normal((3, 9))

    def loss(x, w):
        y, h = rms_norm(x, w)
        return (dy * y).sum() + (dh * h).sum()

    d = rms_norm(*args, dy=dy, dh=dh)[2]
    for i, name in enumerate(("dx", "dweight")):
        for _ in range(6):
            at = tuple(rng.integers(0, s) for s in args[i].shape)
            assert abs(differences(loss, args, (i, at)) - d[name][at]) <= 1e-7 * max(1, np.abs(d[name]).max())
