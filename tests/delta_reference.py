"""Plain fp64 (numpy) forms of the gated delta rule and the grouped norm, one
step and one row at a time, with their adjoints by the chain rule."""
import numpy as np


def delta(q, k, v, g, beta, scale, h0=None, dy=None, dhL=None):
    """One sequence: q, k [L, hk, K], v [L, h, V], g, beta [L, h], h0 [h, K, V].
    Returns y, hL and, with dy, a dict of gradients."""
    q, k, v, g, beta = (np.asarray(a, np.float64) for a in (q, k, v, g, beta))
    L, h, V = v.shape
    hk, K = q.shape[1:]
    rep = h // hk
    S = np.zeros((h, K, V)) if h0 is None else np.asarray(h0, np.float64).copy()
    y, kept = np.zeros((L, h, V)), []
    for t in range(L):
        qt, kt = np.repeat(q[t], rep, 0), np.repeat(k[t], rep, 0)
        before, a = S, np.exp(g[t])
        D = a[:, None, None] * S
        r = v[t] - np.matmul(kt[:, None, :], D)[:, 0]
        u = beta[t][:, None] * r
        S = D + kt[:, :, None] * u[:, None, :]
        y[t] = scale * np.matmul(qt[:, None, :], S)[:, 0]
        kept.append((before, a, D, r, u, S, qt, kt))
    if dy is None:
        return y, S
    hL, dS = S, np.zeros((h, K, V)) if dhL is None else np.asarray(dhL, np.float64).copy()
    d = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dg": np.zeros_like(g),
         "dbeta": np.zeros_like(beta)}
    fold = lambda x: x.reshape(hk, rep, K).sum(1)  # noqa: E731
    for t in reversed(range(L)):
        before, a, D, r, u, S, qt, kt = kept[t]
        do = scale * np.asarray(dy[t], np.float64)
        d["dq"][t] = fold(np.matmul(S, do[:, :, None])[:, :, 0])
        dS = dS + qt[:, :, None] * do[:, None, :]
        du = np.matmul(kt[:, None, :], dS)[:, 0]
        dr = beta[t][:, None] * du
        d["dbeta"][t] = (du * r).sum(-1)
        d["dv"][t] = dr
        d["dk"][t] = fold(np.matmul(dS, u[:, :, None])[:, :, 0] - np.matmul(D, dr[:, :, None])[:, :, 0])
        dD = dS - kt[:, :, None] * dr[:, None, :]
        d["dg"][t] = a * (dD * before).sum((1, 2))
        dS = a[:, None, None] * dD
    d["dh0"] = dS
    return y, hL, d


def delta_batch(q, k, v, g, beta, scale, lens=None, h0=None, dy=None, dhL=None):
    """[batch, L, ...] tensors, or with `lens` sequences packed into one row."""
    if lens is None:
        at = [(b, slice(None)) for b in range(q.shape[0])]
    else:
        ends = np.cumsum(lens)
        at = [(0, slice(e - n, e)) for n, e in zip(lens, ends)]
    part = lambda x, i: None if x is None else x[i]  # noqa: E731
    runs = [delta(q[b, s], k[b, s], v[b, s], g[b, s], beta[b, s], scale, part(h0, i),
                  None if dy is None else dy[b, s], part(dhL, i)) for i, (b, s) in enumerate(at)]
    join = (lambda xs: np.stack(xs)) if lens is None else (lambda xs: np.concatenate(xs)[None])
    y, hL = join([r[0] for r in runs]), np.stack([r[1] for r in runs])
    if dy is None:
        return y, hL
    grads = {n: join([r[2][n] for r in runs]) for n in ("dq", "dk", "dv", "dg", "dbeta")}
    grads["dh0"] = np.stack([r[2]["dh0"] for r in runs])
    return y, hL, grads


def sigmoid(z):
    return 1 / (1 + np.exp(-z))


def norm(x, groups, weight=None, bias=None, z=None, eps=1e-5, rms=False, silu=False, gate_first=False, dy=None):
    """[..., dim]; returns y, or with dy the gradients."""
    x = np.asarray(x, np.float64)
    dim = x.shape[-1]
    w = np.ones(dim) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(dim) if bias is None else np.asarray(bias, np.float64)
    z = None if z is None else np.asarray(z, np.float64)
    gate = None if z is None else z * sigmoid(z)
    dgate = None if z is None else sigmoid(z) * (1 + z * (1 - sigmoid(z)))
    xin = x * gate if gate_first else x
    rows = xin.reshape(*x.shape[:-1], groups, dim // groups)
    c = rows - (0 if rms else rows.mean(-1, keepdims=True))
    r = 1 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    h = (c * r).reshape(x.shape)
    a = h * w + b
    if dy is None:
        return a * sigmoid(a) if silu else a * gate if z is not None and not gate_first else a
    dy = np.asarray(dy, np.float64)
    da, dz = dy, None
    if silu:
        s = sigmoid(a)
        da = dy * s * (1 + a * (1 - s))
    elif z is not None and not gate_first:
        da, dz = dy * gate, dy * a * dgate
    lead = tuple(range(x.ndim - 1))
    out = {"dweight": (da * h).sum(lead), "dbias": da.sum(lead)}
    dh, hr = (da * w).reshape(rows.shape), h.reshape(rows.shape)
    dc = dh - hr * (dh * hr).mean(-1, keepdims=True)
    if not rms:
        dc = dc - dh.mean(-1, keepdims=True)
    dx = (r * dc).reshape(x.shape)
    if gate_first:
        dx, dz = dx * gate, dx * x * dgate
    return dict(out, dx=dx, dz=dz)
