"""A layer of the gated delta rule, run as a model runs it: a whole sequence
forward and backward (as far as the conv's output), then one token at a time
from the state it left.

    projection -> causal conv -> q, k normalised per head -> delta rule
               -> gated norm per head

The projections around it are the caller's and are plain matrix products here.

    python examples/gated_delta_layer.py --tokens 2048 --decode 8
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import torch  # noqa: E402

import selective_state_space_64_amd as ssm  # noqa: E402


class GatedDeltaLayer:
    """qk_heads heads of K keys serve heads / qk_heads value heads of V each."""

    def __init__(self, qk_heads, heads, K, V, width=4, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.hk, self.h, self.K, self.V, self.dtype = qk_heads, heads, K, V, dtype
        self.qk = qk_heads * K
        self.dim = 2 * self.qk + heads * V  # channels of the conv: q, k, v
        self.conv = torch.randn(self.dim, width, device=device, generator=gen) / width
        # a unit key (and query): the root mean square norm over K, times K ** -0.5
        self.unit = torch.full((2 * self.qk,), K ** -0.5, device=device)
        self.norm = torch.ones(heads * V, device=device)

    def split(self, c):
        """q, k, v as views of the conv's output (and the norm's, for q and k)."""
        lead = c.shape[:-1]
        qk = ssm.group_norm_fwd(c[..., :2 * self.qk], 2 * self.hk, weight=self.unit, rms=True, eps=1e-6)
        q, k = (t.unflatten(-1, (self.hk, self.K)) for t in qk.split(self.qk, -1))
        return q, k, c[..., 2 * self.qk:].view(*lead, self.h, self.V)

    def forward(self, x, z, g, beta, train=False):
        """x [batch, L, dim] and the gate z [batch, L, heads V] in, g and beta
        [batch, L, heads] fp32; returns the output and what decode (or
        backward) goes on from."""
        c, conv_state = ssm.conv1d_fwd_bld(x, self.conv, silu=True)
        q, k, v = self.split(c)
        kept = ssm.ssm_delta_bwd_workspace(q, v) if train else None
        y, state = ssm.delta_fwd(q, k, v, g, beta, checkpoints=kept)
        y = y.flatten(-2)
        out = ssm.group_norm_fwd(y, self.h, weight=self.norm, z=z, rms=True)
        return out, dict(conv=conv_state, state=state, saved=(c, q, k, v, y, z, g, beta, kept))

    def backward(self, dout, saved):
        """Gradients down to the conv's output ("conv": silu(conv(x)), whose own
        gradient is the caller's)."""
        c, q, k, v, y, z, g, beta, kept = saved
        n = ssm.group_norm_bwd(y, self.h, dout, weight=self.norm, z=z, rms=True)
        dc = torch.empty_like(c)  # the three gradients land in one row
        dqk = torch.empty_like(c[..., :2 * self.qk])
        dq, dk = (t.unflatten(-1, (self.hk, self.K)) for t in dqk.split(self.qk, -1))
        dv = dc[..., 2 * self.qk:].view(v.shape)
        d = ssm.delta_bwd(q, k, v, g, beta, n["dx"].view(v.shape), workspace=kept,
                          checkpoints_in_workspace=True, dq=dq, dk=dk, dv=dv)
        ssm.group_norm_bwd(c[..., :2 * self.qk], 2 * self.hk, dqk, weight=self.unit, rms=True, eps=1e-6,
                           dx=dc[..., :2 * self.qk])
        return dict(conv=dc, z=n["dz"], g=d["dg"], beta=d["dbeta"], norm=n["dweight"])

    def step(self, x, z, g, beta, carry):
        """One token: x [batch, dim], z [batch, heads V], g and beta [batch,
        heads]; the states in `carry` move on in place."""
        c = ssm.conv1d_update(carry["conv"], x, self.conv, silu=True)
        y = ssm.delta_update(carry["state"], *self.split(c), g, beta)
        return ssm.group_norm_fwd(y.flatten(-2), self.h, weight=self.norm, z=z, rms=True)


def inputs(layer, batch, L, seed=1, device="cuda"):
    gen = torch.Generator(device=device).manual_seed(seed)
    n = lambda *s: torch.randn(*s, device=device, generator=gen)  # noqa: E731
    return (n(batch, L, layer.dim).to(layer.dtype), n(batch, L, layer.h * layer.V).to(layer.dtype),
            -torch.rand(batch, L, layer.h, device=device, generator=gen), torch.sigmoid(n(batch, L, layer.h)))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--decode", type=int, default=8)
    ap.add_argument("--qk-heads", type=int, default=8)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--dim", type=int, default=128, help="keys and values a head")
    a = ap.parse_args()
    layer = GatedDeltaLayer(a.qk_heads, a.heads, a.dim, a.dim)
    x, z, g, beta = inputs(layer, a.batch, a.tokens + a.decode)
    whole, kept = layer.forward(x, z, g, beta, train=True)
    grads = layer.backward(torch.randn_like(whole), kept["saved"])
    print("trained on %d tokens; gradient norms: %s" % (
        a.batch * x.shape[1], ", ".join("%s %.3g" % (m, t.float().norm()) for m, t in grads.items())))
    n = a.tokens
    _, carry = layer.forward(x[:, :n], z[:, :n], g[:, :n], beta[:, :n])
    worst = 0.0
    for t in range(n, n + a.decode):
        out = layer.step(x[:, t], z[:, t], g[:, t], beta[:, t], carry)
        worst = max(worst, float((out.float() - whole[:, t].float()).abs().max()))
    print("decoded %d tokens from the state of %d; largest difference from the whole sequence %.3g"
          % (a.decode, n, worst))


if __name__ == "__main__":
    main()
