"""Refusals and size rules of the gated delta rule and the grouped norm (CPU:
every call here fails validation, device pointers are never followed), the
binding's own checks, and the plain references' gradients against
differences."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from delta_reference import delta, norm

F32, BF16 = ssm.SSM_F32, ssm.SSM_BF16
NULL, SHAPE, DTYPE, MISALIGNED, ALIAS, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 6, 7

SCALE = ctypes.byref(ctypes.c_float(0.125))


def fake(k):
    return 0x100000000 * (k + 1)


POINTERS = {n: fake(i) for i, n in enumerate(
    ["q", "k", "v", "g", "beta", "h0", "cu", "y", "hL", "ws", "dy", "dhL", "dq", "dk", "dv", "dg", "dbeta", "dh0",
     "state", "slots", "x", "weight", "bias", "z", "dx", "dz", "dweight", "dbias"])}


def delta_sizes(**over):
    s = dict(batch=2, L=100, hk=2, h=4, K=64, V=48, dtype=BF16, flags=0, nseq=0, out=BF16, wsb=1 << 40, layout=None)
    return {**s, **{n: v for n, v in over.items() if n in s}}, {**POINTERS, "cu": None,
                                                               **{n: v for n, v in over.items() if n not in s}}


def call_fwd(**over):
    s, p = delta_sizes(**over)
    return ssm.lib().ssm_delta_fwd(
        s["batch"], s["L"], s["hk"], s["h"], s["K"], s["V"], s["dtype"], s["flags"], SCALE, p["q"], p["k"], p["v"],
        p["g"], p["beta"], p["h0"], p["cu"], s["nseq"], s["out"], p["y"], p["hL"], p["ws"], s["wsb"], s["layout"], None)


def call_bwd(**over):
    s, p = delta_sizes(**over)
    return ssm.lib().ssm_delta_bwd(
        s["batch"], s["L"], s["hk"], s["h"], s["K"], s["V"], s["dtype"], s["flags"], SCALE, p["q"], p["k"], p["v"],
        p["g"], p["beta"], p["h0"], p["cu"], s["nseq"], s["out"], p["dy"], p["dhL"], p["dq"], p["dk"], p["dv"],
        p["dg"], p["dbeta"], p["dh0"], p["ws"], s["wsb"], s["layout"], None)


def call_update(**over):
    s, p = delta_sizes(**over)
    return ssm.lib().ssm_delta_update(
        s["batch"], s["hk"], s["h"], s["K"], s["V"], s["dtype"], SCALE, p["state"], p.get("num_slots", 2), p["slots"],
        p["q"], p["k"], p["v"], p["g"], p["beta"], s["out"], p["y"], s["layout"], None)


def delta_layout(cls, **at):
    lay = cls()
    for field, entries in at.items():
        for i, v in entries.items():
            getattr(lay, field)[i] = v
    return ctypes.byref(lay)


SHARED = [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(g=None), NULL), (dict(beta=None), NULL),
    (dict(dtype=7), DTYPE), (dict(out=-1), DTYPE),
    (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(hk=0), SHAPE), (dict(hk=3), SHAPE), (dict(h=1), SHAPE),
    (dict(K=0), SHAPE), (dict(K=257), SHAPE), (dict(V=0), SHAPE), (dict(V=65537), SHAPE), (dict(h=65536), SHAPE),
    (dict(q=fake(0) + 1), MISALIGNED), (dict(g=fake(3) + 2), MISALIGNED),
]
SEQUENCES = [
    (dict(L=0), SHAPE), (dict(L=(1 << 28) - 4095), SHAPE), (dict(cu=fake(6)), SHAPE), (dict(nseq=3), SHAPE),
    (dict(cu=fake(6), nseq=3), SHAPE),  # packed sequences lie in one batch row
    (dict(flags=4), UNSUPPORTED), (dict(flags=1), UNSUPPORTED), (dict(wsb=16), WORKSPACE),
    (dict(ws=fake(9) + 8), MISALIGNED), (dict(h0=fake(5) + 2), MISALIGNED),
    (dict(ws=fake(0)), ALIAS), (dict(batch=1, cu=fake(9) + 4, nseq=3), ALIAS),
    (dict(batch=65535, L=1 << 27, h=65535, hk=1, K=256, V=65536), SHAPE),
]
FWD = SHARED + SEQUENCES + [
    (dict(y=None), NULL), (dict(flags=2, ws=None), NULL), (dict(y=fake(7) + 1), MISALIGNED),
    (dict(y=fake(0)), ALIAS), (dict(y=fake(2) + 64), ALIAS), (dict(hL=fake(5) + 16), ALIAS), (dict(hL=fake(7)), ALIAS),
    (dict(ws=None), WORKSPACE),
    (dict(layout=delta_layout(ssm.DeltaLayout, step={0: -1})), SHAPE),
    (dict(layout=delta_layout(ssm.DeltaLayout, step={0: 64})), SHAPE),       # two heads of 64 share a place
    (dict(layout=delta_layout(ssm.DeltaLayout, head={2: 47})), SHAPE),
    (dict(layout=delta_layout(ssm.DeltaLayout, batch={4: 399})), SHAPE),
    (dict(layout=delta_layout(ssm.DeltaLayout, batch={1: 1 << 56})), SHAPE),
]
BWD = SHARED + SEQUENCES + [
    (dict(dy=None), NULL), (dict(dq=None), NULL), (dict(dv=None), NULL), (dict(dg=None), NULL), (dict(ws=None), NULL),
    (dict(dk=fake(13) + 1), MISALIGNED), (dict(dbeta=fake(16) + 2), MISALIGNED), (dict(dq=fake(13)), ALIAS),
    (dict(dv=fake(2)), ALIAS), (dict(dh0=fake(11) + 4), ALIAS), (dict(dg=fake(16)), ALIAS), (dict(dh0=fake(9)), ALIAS),
    (dict(layout=delta_layout(ssm.DeltaBwdLayout, step={8: 100})), SHAPE),
]
UPDATE = SHARED + [
    (dict(state=None), NULL), (dict(y=None), NULL), (dict(num_slots=0), SHAPE), (dict(slots=None, num_slots=3), SHAPE),
    (dict(state=fake(18) + 4), MISALIGNED), (dict(slots=fake(19) + 2), MISALIGNED), (dict(y=fake(18)), ALIAS),
    (dict(y=fake(2)), ALIAS), (dict(state=fake(0)), ALIAS), (dict(slots=fake(18) + 16), ALIAS),
]


@pytest.mark.parametrize("over,status", FWD, ids=str)
def test_delta_fwd_refusals(over, status):
    assert call_fwd(**over) == status


@pytest.mark.parametrize("over,status", BWD, ids=str)
def test_delta_bwd_refusals(over, status):
    assert call_bwd(**over) == status


@pytest.mark.parametrize("over,status", UPDATE, ids=str)
def test_delta_update_refusals(over, status):
    assert call_update(**over) == status


def test_delta_workspace_sizes():
    L = ssm.lib()
    for f in (L.ssm_delta_fwd_workspace_bytes, L.ssm_delta_bwd_workspace_bytes):
        assert f(1, 64, 1, 1, 64, 64, 0) > 0
        assert f(1, 65, 1, 1, 64, 64, 0) > f(1, 64, 1, 1, 64, 64, 0)
        assert f(1, 64, 1, 1, 64, 64, 5) > f(1, 64, 1, 1, 64, 64, 0)  # each packed sequence may end in a chunk
        for bad in ((0, 64, 1, 1, 64, 64, 0), (1, 0, 1, 1, 64, 64, 0), (1, 64, 2, 1, 64, 64, 0),
                    (1, 64, 2, 3, 64, 64, 0), (1, 64, 1, 1, 257, 64, 0), (2, 64, 1, 1, 64, 64, 1),
                    (65535, 1 << 27, 1, 65535, 256, 65536, 0)):
            assert f(*bad) == 0
    assert L.ssm_delta_bwd_workspace_bytes(1, 64, 1, 1, 64, 64, 0) > L.ssm_delta_fwd_workspace_bytes(1, 64, 1, 1, 64, 64, 0)


def call_norm(bwd=False, **over):
    s = dict(batch=2, L=5, dim=96, groups=4, dtype=BF16, flags=0, out=BF16, wsb=1 << 40, layout=None)
    p = {**POINTERS, "z": None, "dz": None, **{n: v for n, v in over.items() if n not in s}}
    s.update({n: v for n, v in over.items() if n in s})
    head = (s["batch"], s["L"], s["dim"], s["groups"], s["dtype"], s["flags"], None, p["x"], p["weight"], p["bias"],
            p["z"], s["out"])
    if not bwd:
        return ssm.lib().ssm_group_norm_fwd(*head, p["y"], s["layout"], None)
    return ssm.lib().ssm_group_norm_bwd(*head, p["dy"], p["dx"], p["dz"], p["dweight"], p["dbias"], p["ws"], s["wsb"],
                                        s["layout"], None)


NORM = [
    (dict(x=None), NULL), (dict(flags=4), NULL), (dict(dtype=5), DTYPE), (dict(out=5), DTYPE), (dict(batch=0), SHAPE),
    (dict(L=0), SHAPE), (dict(dim=0), SHAPE), (dict(groups=0), SHAPE), (dict(groups=5), SHAPE),
    (dict(dim=(1 << 24) + 4), SHAPE), (dict(batch=1 << 20, L=1 << 11), SHAPE), (dict(flags=8), UNSUPPORTED),
    (dict(x=fake(20) + 1), MISALIGNED), (dict(weight=fake(21) + 2), MISALIGNED),
]


@pytest.mark.parametrize("over,status", NORM + [
    (dict(y=None), NULL), (dict(flags=2, z=fake(23)), UNSUPPORTED), (dict(y=fake(20) + 2), ALIAS),
    (dict(y=fake(21)), ALIAS), (dict(y=fake(20), out=F32), ALIAS),
    (dict(layout=delta_layout(ssm.NormLayout, step={0: 95})), SHAPE),
    (dict(layout=delta_layout(ssm.NormLayout, batch={2: 479})), SHAPE)], ids=str)
def test_norm_fwd_refusals(over, status):
    assert call_norm(**over) == status


@pytest.mark.parametrize("over,status", NORM + [
    (dict(dy=None), NULL), (dict(dx=None), NULL), (dict(z=fake(23)), NULL), (dict(dz=fake(25)), UNSUPPORTED),
    (dict(flags=2, z=fake(23), dz=fake(25)), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE),
    (dict(ws=fake(9) + 4), MISALIGNED), (dict(dx=fake(10)), ALIAS), (dict(dweight=fake(27)), ALIAS),
    (dict(dweight=fake(9)), ALIAS), (dict(z=fake(23), dz=fake(24)), ALIAS),
    (dict(layout=delta_layout(ssm.NormBwdLayout, step={3: 95})), SHAPE)], ids=str)
def test_norm_bwd_refusals(over, status):
    assert call_norm(bwd=True, **over) == status


def test_slices_of_one_buffer_do_not_overlap():
    """dx and dz beside each other in every step pass the overlap check (the call
    then stops at the workspace); sharing a channel does not."""
    lay = delta_layout(ssm.NormBwdLayout, step={3: 200, 4: 200})
    base = fake(24)
    assert call_norm(bwd=True, z=fake(23), dx=base, dz=base + 2 * 96, ws=base, layout=lay) == ALIAS
    ok = dict(z=fake(23), dx=base, dz=base + 2 * 96, layout=lay, wsb=0)
    assert call_norm(bwd=True, **ok) == WORKSPACE
    for step in ({3: 200, 4: 208}, {3: 200, 4: 200}):
        bad = delta_layout(ssm.NormBwdLayout, step=step)
        off = 2 * 96 if step[4] == 208 else 2 * 95
        assert call_norm(bwd=True, z=fake(23), dx=base, dz=base + off, layout=bad) == ALIAS


@pytest.mark.parametrize("step", [0, 200])
@pytest.mark.parametrize("at", [0, 1, 95, 105, 199, 200])
def test_slices_of_one_step_that_overlap(step, at):
    """With one step a batch entry the entries lie a batch stride apart."""
    lay = delta_layout(ssm.NormBwdLayout, step={3: step, 4: step}, batch={3: 200, 4: 200})
    assert call_norm(bwd=True, L=1, z=fake(23), dx=fake(24), dz=fake(24) + 2 * at, layout=lay) == ALIAS


# ---------------------------------------------------------------- the binding
def tensors():
    r = torch.randn
    return dict(q=r(2, 10, 2, 16), k=r(2, 10, 2, 16), v=r(2, 10, 4, 8), g=r(2, 10, 4), beta=r(2, 10, 4))


@pytest.mark.parametrize("change,error", [
    (lambda t: t.update(k=t["k"][:, :, :1].expand(2, 10, 2, 16)), "broadcast"),
    (lambda t: t.update(g=t["g"].bfloat16()), "float32"),
    (lambda t: t.update(q=t["q"].bfloat16()), "float32"),
    (lambda t: t.update(k=t["k"][:, :9]), "shape"),
    (lambda t: t.update(v=t["v"].transpose(2, 3).contiguous().transpose(2, 3)), "contiguous"),
    (lambda t: t.update(q=t["q"][0]), "batch"),
    (lambda t: t.update(cu_seqlens=torch.tensor([0, 10])), "int32"),
    (lambda t: None, "CUDA"),
])
def test_binding_refusals_delta(change, error):
    t = tensors()
    change(t)
    kw = {n: t.pop(n) for n in list(t) if n == "cu_seqlens"}
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises((TypeError, ValueError), match=error):
        ssm.ssm_delta_fwd(*args, **kw)
    with pytest.raises((TypeError, ValueError), match=error):
        ssm.ssm_delta_bwd(*args, torch.randn(2, 10, 4, 8), workspace=torch.empty(16), **kw)


def test_binding_refusals_update_and_norm():
    t = {n: x[:, 0] for n, x in tensors().items()}
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    with pytest.raises(ValueError, match="slots"):
        ssm.ssm_delta_update(torch.zeros(3, 4, 16, 8), *args)
    with pytest.raises(TypeError, match="CUDA"):
        ssm.ssm_delta_update(torch.zeros(2, 4, 16, 8), *args)
    x = torch.randn(2, 3, 8)
    with pytest.raises(ValueError, match="broadcast"):
        ssm.ssm_group_norm_fwd(x[:1].expand(2, 3, 8), 2)
    with pytest.raises(ValueError, match="shape"):
        ssm.ssm_group_norm_fwd(x, 2, z=torch.randn(2, 3, 9))
    with pytest.raises(TypeError, match="CUDA"):
        ssm.ssm_group_norm_bwd(x, 2, x)


# ---------------------------------------------------------------- the references
def directional(f, args, grads, rng):
    """Central differences of f along a random direction of every argument against the gradients."""
    for n in grads:
        d = rng.standard_normal(args[n].shape)
        e = 1e-5
        hi, lo = (f({**args, n: args[n] + s * e * d}) for s in (1, -1))
        assert np.isclose((hi - lo) / (2 * e), (grads[n] * d).sum(), rtol=2e-6, atol=1e-7), n


def test_delta_reference_gradients():
    rng = np.random.default_rng(0)
    L, hk, h, K, V = 7, 2, 4, 5, 3
    n = rng.standard_normal
    a = dict(q=n((L, hk, K)), k=n((L, hk, K)) * 0.5, v=n((L, h, V)), g=-rng.random((L, h)), beta=rng.random((L, h)),
             h0=n((h, K, V)))
    dy, dhL = n((L, h, V)), n((h, K, V))

    def loss(x):
        y, hL = delta(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, x["h0"])
        return (y * dy).sum() + (hL * dhL).sum()

    _, _, d = delta(*(a[m] for m in ("q", "k", "v", "g", "beta")), 0.7, a["h0"], dy, dhL)
    directional(loss, a, {m: d["d" + m] for m in a}, rng)


@pytest.mark.parametrize("opt", [dict(), dict(rms=True), dict(silu=True), dict(gate=True),
                                 dict(gate=True, gate_first=True, rms=True)], ids=str)
def test_norm_reference_gradients(opt):
    opt = dict(opt)
    gate = opt.pop("gate", False)
    rng = np.random.default_rng(1)
    n = rng.standard_normal
    a = dict(x=n((2, 3, 12)), weight=n(12), bias=n(12))
    if gate:
        a["z"] = n((2, 3, 12))
    dy = n((2, 3, 12))
    f = lambda x: (norm(groups=3, **x, **opt) * dy).sum()  # noqa: E731
    d = norm(groups=3, dy=dy, **a, **opt)
    directional(f, a, {m: d["d" + m] for m in a}, rng)
