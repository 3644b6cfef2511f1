"""The delta-rule layer of examples/gated_delta_layer.py on the GPU: decode
goes on where a prefix stopped, and the gradients agree with the same layer in
float64 on the CPU through autograd."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "gated_delta_layer.py")
_spec = importlib.util.spec_from_file_location("gated_delta_layer", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)

# fp32: the calls' own 2e-5 each, five calls one behind the other
TOL = 1e-4


def plain(layer, x, z, g, beta, conv, norm):
    B, L, _ = x.shape
    hk, h, K, V = layer.hk, layer.h, layer.K, layer.V
    W = conv.shape[1]
    c = F.silu(F.conv1d(F.pad(x.transpose(1, 2), (W - 1, 0)), conv[:, None], groups=layer.dim)).transpose(1, 2)
    c.retain_grad()
    q, k, v = c.split([hk * K, hk * K, h * V], -1)

    def unit(t):
        t = t.reshape(B, L, hk, K)
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * K ** -0.5
        return t.repeat_interleave(h // hk, 2)
    q, k, v = unit(q), unit(k), v.reshape(B, L, h, V)
    S, ys = torch.zeros(B, h, K, V, dtype=x.dtype), []
    for t in range(L):
        S = S * g[:, t, :, None, None].exp()
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        ys.append(K ** -0.5 * torch.einsum("bhkv,bhk->bhv", S, q[:, t]))
    y = torch.stack(ys, 1)
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5)
    return y.reshape(B, L, h * V) * norm * F.silu(z), c


def error(got, ref):
    got, ref = got.double().cpu(), ref.detach()
    rms = ref.square().mean().sqrt()
    if rms == 0:  # dg of a first step without a state
        return float(got.abs().max())
    return float(((got - ref).abs() / ref.abs().clamp_min(rms)).max())


@pytest.mark.parametrize("L", [1, 5, 70, 130])
def test_layer_and_its_gradients(L):
    layer = example.GatedDeltaLayer(2, 4, 16, 24, dtype=torch.float32)
    args = example.inputs(layer, 2, L)
    out, kept = layer.forward(*args, train=True)
    dout = torch.randn(out.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    grads = layer.backward(dout, kept["saved"])
    leaves = [t.double().cpu().requires_grad_() for t in (*args, layer.conv, layer.norm)]
    ref, c = plain(layer, *leaves)
    assert error(out, ref) < TOL
    ref.backward(dout.double().cpu())
    for name, leaf in zip(("conv", "z", "g", "beta", "norm"), (c, *leaves[1:4], leaves[5])):
        # 4 times as much for dg, whose terms cancel (as for the call itself)
        assert error(grads[name], leaf.grad) < TOL * (4 if name == "g" else 1), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_goes_on(dtype):
    layer = example.GatedDeltaLayer(2, 4, 32, 40, dtype=dtype)
    x, z, g, beta = example.inputs(layer, 3, 75)
    whole, last = layer.forward(x, z, g, beta)
    out, carry = layer.forward(x[:, :66], z[:, :66], g[:, :66], beta[:, :66])
    for t in range(66, 75):
        out = layer.step(x[:, t], z[:, t], g[:, t], beta[:, t], carry)
        # bf16: an ulp of difference in the delta rule's output, one more from the norm's own rounding
        tol = TOL if dtype == torch.float32 else 2 * torch.finfo(dtype).eps
        assert error(out, whole[:, t].double().cpu()) < tol
    assert error(carry["state"], last["state"].double().cpu()) < (TOL if dtype == torch.float32 else 2.4e-4)


def test_slices_of_one_step():
    """One step a batch entry: outputs beside each other in one row, as for
    longer sequences."""
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, z, dy, w = r(3, 1, 64), r(3, 1, 64), r(3, 1, 64), r(64)
    want = example.ssm.group_norm_bwd(x, 4, dy, weight=w, z=z)
    both = torch.zeros(3, 1, 128, device="cuda")
    example.ssm.group_norm_bwd(x, 4, dy, weight=w, z=z, dx=both[..., :64], dz=both[..., 64:])
    assert torch.equal(both, torch.cat([want["dx"], want["dz"]], -1))
    q, k, v, dv = r(3, 1, 2, 16), r(3, 1, 2, 16), r(3, 1, 2, 16), r(3, 1, 2, 16)
    g, beta = -torch.rand(3, 1, 2, device="cuda"), torch.rand(3, 1, 2, device="cuda")
    want = example.ssm.delta_bwd(q, k, v, g, beta, dv)
    rows = torch.zeros(3, 1, 3, 2, 16, device="cuda")
    example.ssm.delta_bwd(q, k, v, g, beta, dv, **{n: rows[:, :, i] for i, n in enumerate(("dq", "dk", "dv"))})
    assert torch.equal(rows, torch.stack([want[n] for n in ("dq", "dk", "dv")], 2))
