"""The calls together as a layer uses them: residual norm, projection, conv,
head scan, gated norm, projection, and the next residual norm, in one piece,
backwards, and one token at a time; against the same layer in fp64 on the CPU
(gradients by autograd)."""
import pytest
import torch
import torch.nn.functional as F

import selective_state_space_64_amd as ssm
from test_gpu_delta import error

pytestmark = pytest.mark.gpu

G, H, N, P, D, W = 2, 4, 32, 24, 72, 4
INNER, CONV = H * P, H * P + 2 * G * N
# fp32: the calls' own errors of up to 2e-5 each (test_gpu_heads, test_gpu_rms,
# test_gpu_norm), six calls one behind the other
TOL = 1.2e-4


def weights(dtype):
    r = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    w = {"norm": 1 + 0.1 * n(D), "inp": n(INNER + CONV + H, D) * D ** -0.5, "conv": n(CONV, W) / 2, "cbias": n(CONV) / 4,
         "A": -torch.rand(H, generator=r) * 4 - 0.3, "Dskip": n(H), "dt_bias": n(H), "gate": 1 + 0.1 * n(INNER),
         "outp": n(D, INNER) * INNER ** -0.5, "next": 1 + 0.1 * n(D)}
    return {k: v.to(dtype).float() if k in ("inp", "outp") else v for k, v in w.items()}


def norm(h, u):
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-5) * u


def conv(w, xbc):
    return F.silu(F.conv1d(F.pad(xbc.transpose(1, 2), (W - 1, 0)), w["conv"][:, None], w["cbias"], groups=CONV)).transpose(1, 2)


def scan(w, c, dt):
    B, L, _ = c.shape
    v, b, r = c.split([INNER, G * N, G * N], -1)
    v, b, r = v.reshape(B, L, H, P), *(k.reshape(B, L, G, N).repeat_interleave(H // G, 2) for k in (b, r))
    step = F.softplus(dt + w["dt_bias"])
    S, ys = torch.zeros(B, H, N, P, dtype=c.dtype), []
    for t in range(L):
        a = (step[:, t] * w["A"]).exp()[..., None, None]
        S = a * S + (step[:, t, :, None] * b[:, t])[..., None] * v[:, t, :, None]
        ys.append((r[:, t, :, :, None] * S).sum(2) + w["Dskip"][:, None] * v[:, t])
    return torch.stack(ys, 1).reshape(B, L, INNER), S


def gated_norm(w, y, z):
    gated = (y * F.silu(z)).unflatten(-1, (G, -1))
    return (gated / torch.sqrt(gated.square().mean(-1, keepdim=True) + 1e-5)).flatten(-2) * w["gate"]


def plain(w, x, res):
    """Returns the last norm's output, the residual stream, and the tensors between the calls."""
    h = x + res
    p = norm(h, w["norm"]) @ w["inp"].T
    z, xbc, dt = p.split([INNER, CONV, H], -1)
    c = conv(w, xbc)
    o = gated_norm(w, scan(w, c, dt)[0], z) @ w["outp"].T
    return norm(o + h, w["next"]), o + h, {"p": p, "c": c, "o": o}


class Layer:
    def __init__(self, w, dtype):
        self.w = {k: v.cuda() for k, v in w.items()}
        self.inp, self.outp = self.w["inp"].to(dtype), self.w["outp"].to(dtype)
        self.dtype = dtype

    def parts(self, c):
        v, b, r = c.split([INNER, G * N, G * N], -1)
        return v.unflatten(-1, (H, P)), b.unflatten(-1, (G, N)), r.unflatten(-1, (G, N))

    def forward(self, x, res, train=False):
        w = self.w
        u, h, _ = ssm.rms_norm_fwd(x, weight=w["norm"], residual=res)
        p = u @ self.inp.T
        z, xbc, dt = p.split([INNER, CONV, H], -1)
        c, carry = ssm.conv1d_fwd_bld(xbc, w["conv"], bias=w["cbias"])
        v, b, r = self.parts(c)
        ws = ssm.ssm_head_scan_bwd_workspace(v, b) if train else None
        y, state = ssm.head_scan_fwd(v, dt, w["A"], b, r, Dskip=w["Dskip"], dt_bias=w["dt_bias"], checkpoints=ws)
        y = y.flatten(-2)
        m = ssm.group_norm_fwd(y, G, weight=w["gate"], z=z, rms=True, gate_first=True)
        o = m @ self.outp.T
        out, h2, _ = ssm.rms_norm_fwd(o, weight=w["next"], residual=h)
        return out, h2, dict(carry=carry, state=state, h=h, u=u, p=p, c=c, y=y, m=m, o=o, out=out, h2=h2, ws=ws)

    def backward(self, k, h2, dout, dh2):
        """Gradients of the calls' inputs up to the conv's output, and of the weights on the way."""
        w = self.w
        e = ssm.rms_norm_bwd(h2, dout, weight=w["next"], dh=dh2)
        z, _, dt = k["p"].split([INNER, CONV, H], -1)
        dp = torch.zeros_like(k["p"])
        dz, _, ddt = dp.split([INNER, CONV, H], -1)
        n = ssm.group_norm_bwd(k["y"], G, e["dx"] @ self.outp, weight=w["gate"], z=z, rms=True, gate_first=True, dz=dz)
        v, b, r = self.parts(k["c"])
        dc = torch.empty_like(k["c"])
        dv, db, dr = self.parts(dc)
        s = ssm.head_scan_bwd(v, dt, w["A"], b, r, n["dx"].unflatten(-1, (H, P)), Dskip=w["Dskip"], dt_bias=w["dt_bias"],
                              workspace=k["ws"], checkpoints_in_workspace=True, dx=dv, dBm=db, dCm=dr, ddt=ddt)
        return {"next": e["dweight"], "gate": n["dweight"], "A": s["dA"], "Dskip": s["dDskip"], "dt_bias": s["ddt_bias"],
                "z": dz, "dt": ddt, "c": dc, "h": e["dresidual"]}

    def step(self, x, res, carry, state):
        w = self.w
        u, h, _ = ssm.rms_norm_fwd(x, weight=w["norm"], residual=res)
        p = u @ self.inp.T
        z, xbc, dt = p.split([INNER, CONV, H], -1)
        c = ssm.conv1d_update(carry, xbc, w["conv"], bias=w["cbias"])
        v, b, r = self.parts(c)
        y = ssm.head_scan_update(state, v, dt, w["A"], b, r, Dskip=w["Dskip"], dt_bias=w["dt_bias"]).flatten(-2)
        m = ssm.group_norm_fwd(y, G, weight=w["gate"], z=z, rms=True, gate_first=True)
        o = m @ self.outp.T
        out, h2, _ = ssm.rms_norm_fwd(o, weight=w["next"], residual=h)
        return dict(h=h, u=u, p=p, c=c, y=y, m=m, o=o, out=out, h2=h2)


def inputs(B, L, dtype):
    r = torch.Generator().manual_seed(L)
    return [torch.randn(B, L, D, generator=r).to(t) for t in (dtype, torch.float32)]


@pytest.mark.parametrize("B,L", [(2, 1), (2, 5), (1, 70), (2, 130)])
def test_layer_and_its_gradients(B, L):
    w, (x, res) = weights(torch.float32), inputs(B, L, torch.float32)
    layer = Layer(w, torch.float32)
    out, h2, k = layer.forward(x.cuda(), res.cuda(), train=True)
    dout, dh2 = torch.randn(B, L, D), torch.randn(B, L, D)
    got = layer.backward(k, h2, dout.cuda(), dh2.cuda())

    leaves = {n: v.double().requires_grad_() for n, v in w.items()}
    want, h2w, mid = plain(leaves, x.double(), res.double())
    for t in mid.values():
        t.retain_grad()
    assert error(out, want.detach()) <= TOL and error(h2, h2w.detach()) <= TOL
    assert error(k["c"], mid["c"].detach()) <= TOL
    ((want * dout).sum() + (h2w * dh2).sum()).backward()
    dz, _, ddt = mid["p"].grad.split([INNER, CONV, H], -1)
    ref = {"z": dz, "dt": ddt, "c": mid["c"].grad, "h": mid["o"].grad,  # o and h add up: one gradient
           **{n: leaves[n].grad for n in ("next", "gate", "A", "Dskip", "dt_bias")}}
    for n in ref:
        # dt, A and dt_bias: 4 times that, as for the scan's own (their terms cancel)
        assert error(got[n], ref[n]) <= TOL * (4 if n in ("dt", "A", "dt_bias") else 1), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_goes_on(dtype):
    """A prefix in one call and the rest a token at a time, against all of it in
    fp64: in fp32 from end to end, and every call by itself from the inputs that
    it had, where bf16 rounds each call's output by up to half an ulp, 2^-8."""
    B, L, cut = 3, 75, 66
    w, (x, res) = weights(dtype), inputs(B, L, dtype)
    layer = Layer(w, dtype)
    _, _, k = layer.forward(x[:, :cut].cuda(), res[:, :cut].cuda())
    names = ("h", "u", "p", "c", "y", "m", "o", "out", "h2")
    parts = {n: [k[n]] for n in names}
    for t in range(cut, L):
        one = layer.step(x[:, t].cuda(), res[:, t].cuda(), k["carry"], k["state"])
        for n in names:
            parts[n].append(one[n][:, None])
    got = {n: torch.cat(v, 1) for n, v in parts.items()}
    w = {n: v.double() for n, v in w.items()}
    x, res = x.double(), res.double()
    g = {n: v.double().cpu() for n, v in got.items()}
    if dtype == torch.float32:
        want, h2, _ = plain(w, x, res)
        assert error(got["out"], want) <= TOL and error(got["h2"], h2) <= TOL
    z, xbc, dt = g["p"].split([INNER, CONV, H], -1)
    y, S = scan(w, g["c"], dt)
    ref = {"h": x + res, "u": norm(x + res, w["norm"]), "c": conv(w, xbc), "y": y, "m": gated_norm(w, g["y"], z),
           "h2": g["o"] + g["h"], "out": norm(g["o"] + g["h"], w["next"])}
    for n, v in ref.items():
        # one call's own error: a sixth of the six calls' in a row, and of two bf16 terms 6e-5 (test_gpu_heads)
        tol = TOL / 6 if dtype == torch.float32 or n in ("h", "h2") else 6e-5 + 2.0 ** -8
        assert error(got[n], v) <= tol, n
    assert error(k["state"], S) <= TOL / 6 and error(k["carry"], xbc[:, -(W - 1):].transpose(1, 2)) == 0
