"""Plain fp64 (numpy) forms of the selective scan with one decay a head and of
the residual norm, one step and one row at a time, with their adjoints by the
chain rule."""
import numpy as np


def softplus(u):
    return np.logaddexp(0.0, u)


def head_scan(x, dt, A, B, C, D=None, bias=None, h0=None, dy=None, dhL=None):
    """One sequence: x [L, h, P], dt [L, h], A, D, bias [h], B, C [L, g, N],
    h0 [h, N, P].  Returns y, hL and, with dy, a dict of gradients."""
    x, dt, A, B, C = (np.asarray(a, np.float64) for a in (x, dt, A, B, C))
    L, h, P = x.shape
    g, N = B.shape[1:]
    rep = h // g
    D = np.zeros(h) if D is None else np.asarray(D, np.float64)
    u = dt + (0.0 if bias is None else np.asarray(bias, np.float64))
    step = softplus(u)
    S = np.zeros((h, N, P)) if h0 is None else np.asarray(h0, np.float64).copy()
    y, kept = np.zeros((L, h, P)), []
    for t in range(L):
        Bt, Ct = np.repeat(B[t], rep, 0), np.repeat(C[t], rep, 0)
        before, a = S, np.exp(step[t] * A)
        S = a[:, None, None] * S + (step[t][:, None] * Bt)[:, :, None] * x[t][:, None, :]
        y[t] = np.matmul(Ct[:, None, :], S)[:, 0] + D[:, None] * x[t]
        kept.append((before, a, S, Bt, Ct))
    if dy is None:
        return y, S
    hL, dS = S, np.zeros((h, N, P)) if dhL is None else np.asarray(dhL, np.float64).copy()
    dy = np.asarray(dy, np.float64)
    d = {"dx": np.zeros_like(x), "ddt": np.zeros_like(dt), "dBm": np.zeros_like(B), "dCm": np.zeros_like(C),
         "dA": np.zeros(h), "dDskip": (dy * x).sum((0, 2)), "ddt_bias": np.zeros(h)}
    fold = lambda a: a.reshape(g, rep, N).sum(1)  # noqa: E731
    for t in reversed(range(L)):
        before, a, S, Bt, Ct = kept[t]
        dS = dS + Ct[:, :, None] * dy[t][:, None, :]
        d["dCm"][t] = fold(np.matmul(S, dy[t][:, :, None])[:, :, 0])
        dSx = np.matmul(dS, x[t][:, :, None])[:, :, 0]
        d["dBm"][t] = fold(step[t][:, None] * dSx)
        d["dx"][t] = step[t][:, None] * np.matmul(Bt[:, None, :], dS)[:, 0] + D[:, None] * dy[t]
        da = a * (dS * before).sum((1, 2))
        d["dA"] += step[t] * da
        d["ddt"][t] = ((Bt * dSx).sum(-1) + A * da) / (1.0 + np.exp(-u[t]))
        dS = a[:, None, None] * dS
    d["ddt_bias"] = d["ddt"].sum(0)
    d["dh0"] = dS
    return y, hL, d


def head_scan_batch(x, dt, A, B, C, D=None, bias=None, lens=None, h0=None, dy=None, dhL=None):
    """[batch, L, ...] tensors, or with `lens` sequences packed into one row."""
    if lens is None:
        at = [(b, slice(None)) for b in range(x.shape[0])]
    else:
        ends = np.cumsum(lens)
        at = [(0, slice(e - n, e)) for n, e in zip(lens, ends)]
    part = lambda v, i: None if v is None else v[i]  # noqa: E731
    runs = [head_scan(x[b, s], dt[b, s], A, B[b, s], C[b, s], D, bias, part(h0, i), None if dy is None else dy[b, s],
                      part(dhL, i)) for i, (b, s) in enumerate(at)]
    join = (lambda v: np.stack(v)) if lens is None else (lambda v: np.concatenate(v)[None])
    y, hL = join([r[0] for r in runs]), np.stack([r[1] for r in runs])
    if dy is None:
        return y, hL
    summed = ("dA", "dDskip", "ddt_bias")
    d = {n: sum(r[2][n] for r in runs) if n in summed else
         (np.stack if n == "dh0" else join)([r[2][n] for r in runs]) for n in runs[0][2]}
    return y, hL, d


def rms_norm(x, weight=None, residual=None, eps=1e-5, dy=None, dh=None):
    """y, h and, with dy, a dict of the gradients of sum dy . y + sum dh . h."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    y = h * r * w
    if dy is None:
        return y, h
    u = np.asarray(dy, np.float64) * w
    d = r * (u - h * r * r * (u * h).mean(-1, keepdims=True)) + (0.0 if dh is None else np.asarray(dh, np.float64))
    return y, h, {"dx": d, "dweight": (dy * h * r).reshape(-1, h.shape[-1]).sum(0)}


def block_scales(y, block=128):
    """The scale of every `block` neighbours of the last index."""
    n = y.shape[-1]
    m = [np.abs(y[..., i:i + block]).max(-1) for i in range(0, n, block)]
    return np.maximum(np.stack(m, -1) / 448.0, 2.0 ** -126)
