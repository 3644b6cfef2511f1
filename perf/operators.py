"""The gated delta rule and the grouped norm around it: the calls that are
timed, in their plain form and through the package.

Five operators, as a layer of a language model uses them.  Per head, with
keys and queries of K entries, values of V entries and a state S of K x V:

    S_t = e^{g_t} S_{t-1} + beta_t k_t (v_t - e^{g_t} S_{t-1}^T k_t)^T
    y_t = scale S_t^T q_t

  fwd       whole sequences (prompts): y and the last state
  train     the same with its gradients: a training step's forward and backward
  update    one new token per sequence on a persistent state
  norm      y = act(normalise(x) w + b) over groups of channels of one step
  norm_bwd  its gradients

``run`` computes them from elementary torch operations in float32 (``own``
false) or by calling the package (``own`` true).
"""
import torch

own = False

F32, BF16 = "f32", "bf16"
CHUNK = 64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a few tokens of a small model: the launch and the chain of one chunk
        dict(name="fwd short f32", op="fwd", dtype=F32, lens="17", hk=2, h=4, K=32, V=40, h0=True),
        # a prompt batch through a layer of 5120 value channels
        dict(name="fwd layer bf16", op="fwd", dtype=BF16, lens="2048,2048,2048,2048", packed=False, hk=40, h=40,
             K=128, V=128, h0=False),
        # prompts of unequal lengths packed into one batch row, keys shared by three value heads
        dict(name="fwd packed bf16", op="fwd", dtype=BF16, lens="4097,1,2500,0,63,6001,777,2945", packed=True, hk=4,
             h=12, K=128, V=128, h0=True),
        # one long document: few rows, a long recurrence
        dict(name="fwd long bf16", op="fwd", dtype=BF16, lens="65521", packed=False, hk=12, h=12, K=128, V=128,
             h0=False),
        # a training step of the layer
        dict(name="train layer bf16", op="train", dtype=BF16, lens="2048,2048,2048,2048", packed=False, hk=40, h=40,
             K=128, V=128, h0=False),
        # fp32 training of a small model, a length that no tile divides
        dict(name="train odd f32", op="train", dtype=F32, lens="777,777", packed=False, hk=2, h=6, K=64, V=96,
             h0=True),
        # one user's next token
        dict(name="update one bf16", op="update", dtype=BF16, batch=1, slots=0, hk=40, h=40, K=128, V=128),
        # a serving batch whose states sit in a pool of slots
        dict(name="update batch bf16", op="update", dtype=BF16, batch=64, slots=80, hk=40, h=40, K=128, V=128),
        # the layer's output norm: one group a head, gated by silu(z)
        dict(name="norm gate bf16", op="norm", dtype=BF16, batch=4, L=2048, dim=5120, groups=40, rms=True,
             act="gate", affine="weight"),
        # the same for one decoded batch of a small model, in fp32
        dict(name="norm step f32", op="norm", dtype=F32, batch=8, L=1, dim=1536, groups=12, rms=True,
             act="gate", affine="weight"),
        # gradients of the layer's output norm
        dict(name="norm_bwd gate bf16", op="norm_bwd", dtype=BF16, batch=4, L=2048, dim=5120, groups=40, rms=True,
             act="gate", affine="weight"),
        # mean and variance, an affine with bias and silu, groups of 255 channels
        dict(name="norm_bwd odd f32", op="norm_bwd", dtype=F32, batch=3, L=333, dim=1530, groups=6, rms=False,
             act="silu", affine="both"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "train", "update", "norm", "norm_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("fwd", "train", "update"):
        hk, rep = rng.choice([1, 2, 4, 6, 8, 12, 16, 20, 40]), rng.choice([1, 1, 2, 3])
        h = min(40, hk * rep) // hk * hk
        K = rng.choice([128, 128, 64, 32, 96, 100, 256, rng.randint(16, 160)])
        V = rng.choice([128, 128, 64, 256, 96, rng.randint(16, 160)])
        case = dict(op=op, dtype=dtype, hk=hk, h=h, K=K, V=V)
        if op == "update":
            batch = _log(rng, 1, 64)
            while batch * h * K * V > 64 * 40 * 128 * 128:
                batch //= 2
            return dict(case, batch=batch, slots=rng.choice([0, batch + rng.randint(0, 16)]))
        # the listed layer has 4 x 2048 tokens of 40 heads of 128 x 128
        most = 4 * 2048 * 40 * 128 * 128 // (1 if dtype == BF16 else 8)
        tokens = max(1, min(_log(rng, 1, 65521 if op == "fwd" else 16384), most // (h * K * V)))
        n = min(tokens, rng.choice([1, 1, 2, 3, 4, 7, 16]))
        packed = rng.random() < 0.4
        if packed:
            cuts = sorted(rng.randint(0, tokens) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
        else:
            lens = [tokens // n] * n
        return dict(case, lens=",".join(map(str, lens)), packed=packed, h0=rng.random() < 0.5)
    while True:
        groups = rng.choice([1, 2, 6, 12, 16, 40])
        per = rng.choice([128, 64, 256, 96, 255, 1536, 5120, rng.randint(2, 700)])
        if groups * per <= 5120:
            break
    batch = rng.choice([1, 2, 3, 4, 8])
    L = _log(rng, 1, 4 * 2048 * 5120 // (batch * groups * per) // (1 if dtype == BF16 else 2))
    return dict(op=op, dtype=dtype, batch=batch, L=min(L, 65536), dim=groups * per, groups=groups,
                rms=rng.random() < 0.5, act=rng.choice(["none", "silu", "gate", "gate_first"]),
                affine=rng.choice(["none", "weight", "both"]))


# ------------------------------------------------------------------ the inputs
def _t(case):
    return torch.float32 if case["dtype"] == F32 else torch.bfloat16


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _t(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    op = case["op"]
    if op in ("norm", "norm_bwd"):
        shape, dim = (case["batch"], case["L"], case["dim"]), case["dim"]
        s = dict(op=op, groups=case["groups"], rms=case["rms"], act=case["act"], eps=1e-5,
                 x=(normal(*shape) * 0.7 + 0.1).to(dt),
                 z=normal(*shape).to(dt) if case["act"].startswith("gate") else None,
                 w=1 + 0.1 * normal(dim) if case["affine"] != "none" else None,
                 b=0.1 * normal(dim) if case["affine"] == "both" else None)
        if op == "norm_bwd":
            s["dy"] = normal(*shape).to(dt)
        return s

    hk, h, K, V = case["hk"], case["h"], case["K"], case["V"]
    if op == "update":
        shape = (case["batch"],)
    elif case.get("packed"):
        shape = (1, sum(_lens(case)))
    else:
        shape = (len(_lens(case)), _lens(case)[0])
    silu = torch.nn.functional.silu
    # the layer's q, k, v leave a short convolution and a silu; q and k are then normalised to length one
    q, k = (torch.nn.functional.normalize(silu(normal(*shape, hk, K)), dim=-1).to(dt) for _ in range(2))
    v = silu(normal(*shape, h, V)).to(dt)
    # decay rates A in [1, 16] and steps of softplus(dt + bias), bias placed for steps in [1e-3, 1e-1]
    A = 1 + 15 * uniform(h)
    bias = torch.log(torch.expm1(torch.exp(uniform(h) * 4.605 - 6.908)))
    g = -A * torch.nn.functional.softplus(normal(*shape, h) + bias)
    s = dict(op=op, q=q, k=k, v=v, g=g, beta=torch.sigmoid(normal(*shape, h)), scale=K ** -0.5)
    if op == "update":
        n = case["slots"]
        s["state"] = 0.3 * normal(n or case["batch"], h, K, V)
        s["slots"] = torch.randperm(n, generator=gen, device="cuda")[:case["batch"]].int() if n else None
        return s
    lens = _lens(case)
    s["h0"] = 0.3 * normal(len(lens), h, K, V) if case["h0"] else None
    s["lens"] = lens
    s["cu"] = None
    if case.get("packed"):
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    if op == "train":
        s["dy"] = normal(*shape, h, V).to(dt)
        s["dhL"] = 0.3 * normal(len(lens), h, K, V) if case["h0"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _call(s) if own else _plain(s)


def _call(s):
    import selective_state_space_64_amd as ssm

    op = s["op"]
    if op == "norm" or op == "norm_bwd":
        kw = dict(weight=s["w"], bias=s["b"], z=s["z"], eps=s["eps"], rms=s["rms"], silu=s["act"] == "silu",
                  gate_first=s["act"] == "gate_first")
        if op == "norm":
            return ssm.ssm_group_norm_fwd(s["x"], s["groups"], **kw)
        return ssm.ssm_group_norm_bwd(s["x"], s["groups"], s["dy"], **kw)
    if op == "update":
        y = ssm.ssm_delta_update(s["state"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"],
                                 slots=s["slots"])
        return y, s["state"]
    args, kw = (s["q"], s["k"], s["v"], s["g"], s["beta"]), dict(scale=s["scale"], h0=s["h0"], cu_seqlens=s["cu"])
    if op == "fwd":
        return ssm.ssm_delta_fwd(*args, **kw)
    ws = ssm.ssm_delta_bwd_workspace(s["q"], s["v"], cu_seqlens=s["cu"])
    y, hL = ssm.ssm_delta_fwd(*args, checkpoints=ws, **kw)
    grads = ssm.ssm_delta_bwd(*args, s["dy"], dhL=s["dhL"], workspace=ws, checkpoints_in_workspace=True, **kw)
    return y, hL, grads


def _plain(s):
    op = s["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "update":
        return _plain_update(s)
    return _plain_delta(s)


def _plain_update(s):
    h = s["v"].shape[-2]
    rep = h // s["q"].shape[-2]
    q, k = (s[n].float().repeat_interleave(rep, dim=-2) for n in ("q", "k"))
    at = slice(None) if s["slots"] is None else s["slots"].long()
    S = s["state"][at] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    y = s["scale"] * (S * q[..., None]).sum(-2)
    s["state"][at] = S
    return y.to(s["v"].dtype), s["state"]


def _chunks(x, lens, packed):
    """[batch, L, heads, ...] -> [sequences, heads, chunks, 64, ...] in float32, zeros behind each sequence's end."""
    n = max(1, -(-max(lens) // CHUNK))
    at = torch.arange(n * CHUNK, device=x.device)[None, :]
    size = torch.tensor(lens, device=x.device)[:, None]
    if packed:
        flat = x.reshape(-1, *x.shape[2:]).float()
        first = size.cumsum(0) - size
        rows = (first + at).clamp(max=flat.shape[0] - 1)
        out = flat[rows]
    else:
        out = x.float()[:, at[0].clamp(max=x.shape[1] - 1)]
    there = (at < size).reshape(len(lens), n * CHUNK, *[1] * (out.dim() - 2))
    out = torch.where(there, out, 0.0).transpose(1, 2)
    return out.reshape(*out.shape[:2], n, CHUNK, *out.shape[3:])


def _steps(x, like, lens, packed):
    """The way back of _chunks, to [batch, L, heads, ...]."""
    x = x.reshape(*x.shape[:2], -1, *x.shape[4:]).transpose(1, 2)
    if packed:
        at = torch.arange(x.shape[1], device=x.device)[None, :]
        size = torch.tensor(lens, device=x.device)[:, None]
        return x[at < size].reshape(like.shape[0], like.shape[1], *x.shape[2:])
    return x[:, :like.shape[1]]


def _plain_delta(s):
    lens, packed, scale = s["lens"], s["cu"] is not None, s["scale"]
    hk, h = s["q"].shape[-2], s["v"].shape[-2]
    q, k = (_chunks(s[n].repeat_interleave(h // hk, dim=-2), lens, packed) for n in ("q", "k"))
    v, g, beta = (_chunks(s[n], lens, packed) for n in ("v", "g", "beta"))
    n = q.shape[2]
    G = g.cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    strict = low.tril(-1)
    decay = torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf).exp()
    P = scale * decay * (q @ k.transpose(-1, -2))
    M = torch.where(strict, beta[..., None] * decay * (k @ k.transpose(-1, -2)), 0.0)
    # T = (1 + M)^-1 by forward substitution, one row of every chunk at a time
    T = torch.eye(CHUNK, device=G.device).expand_as(M).contiguous()
    for i in range(1, CHUNK):
        T[..., i, :i] = -(M[..., i:i + 1, :i] @ T[..., :i, :i])[..., 0, :]
    eG, tail = G.exp()[..., None], (G[..., -1:] - G).exp()[..., None]
    eC = G[..., -1].exp()[..., None, None]
    W, U0 = T @ (beta[..., None] * eG * k), T @ (beta[..., None] * v)
    kT, qe = (tail * k).transpose(-1, -2), scale * eG * q
    S = s["h0"] if s["h0"] is not None else torch.zeros(len(lens), h, k.shape[-1], v.shape[-1], device=G.device)
    entry, U = [], []
    for c in range(n):
        entry.append(S)
        U.append(U0[:, :, c] - W[:, :, c] @ S)
        S = eC[:, :, c] * S + kT[:, :, c] @ U[c]
    S0, U, hL = torch.stack(entry, 2), torch.stack(U, 2), S
    y = _steps(qe @ S0 + P @ U, s["v"], lens, packed).to(s["v"].dtype)
    if s["op"] == "fwd":
        return y, hL

    dy = _chunks(s["dy"], lens, packed)
    dS = s["dhL"] if s["dhL"] is not None else torch.zeros_like(hL)
    KS = k @ S0
    Tt, Pdy, qTdy = T.transpose(-1, -2), P.transpose(-1, -2) @ dy, qe.transpose(-1, -2) @ dy
    rkT, tk = (beta[..., None] * eG * k).transpose(-1, -2), tail * k
    after, dX = [None] * n, [None] * n
    for c in reversed(range(n)):
        after[c] = dS
        dX[c] = Tt[:, :, c] @ (Pdy[:, :, c] + tk[:, :, c] @ dS)
        dS = eC[:, :, c] * dS + qTdy[:, :, c] - rkT[:, :, c] @ dX[c]
    dS1, dX, dh0 = torch.stack(after, 2), torch.stack(dX, 2), dS
    kk, qk = k @ k.transpose(-1, -2), q @ k.transpose(-1, -2)
    dP = torch.where(low, scale * decay * (dy @ U.transpose(-1, -2)), 0.0)
    dM = torch.where(strict, -decay * (dX @ U.transpose(-1, -2)), 0.0)
    bM = beta[..., None] * dM
    qS, dXS, UdS = qe * (dy @ S0.transpose(-1, -2)), dX @ S0.transpose(-1, -2), U @ dS1.transpose(-1, -2)
    dq = scale * eG * (dy @ S0.transpose(-1, -2)) + dP @ k
    dk = (dP.transpose(-1, -2) @ q + (bM + bM.transpose(-1, -2)) @ k + tail * UdS - beta[..., None] * eG * dXS)
    dv = beta[..., None] * dX
    dbeta = (dX * (v - eG * KS)).sum(-1) + (dM * kk).sum(-1)
    # d/dG of every exponential, then G = cumsum(g)
    inner = dP * qk + bM * kk
    out = (tk * UdS).sum(-1)
    dG = inner.sum(-1) - inner.sum(-2) + qS.sum(-1) - (beta[..., None] * eG * k * dXS).sum(-1) - out
    dG[..., -1] += out.sum(-1) + (eC * S0 * dS1).sum((-1, -2))
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    grads = {}
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv), ("dg", dg), ("dbeta", dbeta)):
        x = _steps(x, s["v"], lens, packed)
        if name in ("dq", "dk"):
            x = x.reshape(*x.shape[:2], hk, h // hk, x.shape[-1]).sum(-2)
        grads[name] = x if name in ("dg", "dbeta") else x.to(s["v"].dtype)
    grads["dh0"] = dh0
    return y, hL, grads


def _norm_parts(s, x, z):
    """The steps of the norm's forward, on x and z of any float type."""
    p = {}
    p["in"] = x * (z * torch.sigmoid(z)) if s["act"] == "gate_first" else x
    rows = p["in"].reshape(*x.shape[:-1], s["groups"], -1)
    if not s["rms"]:
        rows = rows - rows.mean(-1, keepdim=True)
    p["r"] = ((rows * rows).mean(-1, keepdim=True) + s["eps"]).rsqrt()
    p["n"] = (rows * p["r"]).reshape(x.shape)
    a = p["n"] if s["w"] is None else p["n"] * s["w"].to(x.dtype)
    p["a"] = a if s["b"] is None else a + s["b"].to(x.dtype)
    return p


def _plain_norm(s):
    p = _norm_parts(s, s["x"].float(), None if s["z"] is None else s["z"].float())
    y = p["a"]
    if s["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif s["act"] == "gate":
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(s["x"].dtype)


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    z = None if s["z"] is None else s["z"].float()
    p = _norm_parts(s, x, z)
    da, dz = dy, None
    if s["act"] == "silu":
        t = torch.sigmoid(p["a"])
        da = dy * (t * (1 + p["a"] * (1 - t)))
    elif s["act"] == "gate":
        t = torch.sigmoid(z)
        da, dz = dy * (z * t), dy * p["a"] * (t * (1 + z * (1 - t)))
    out = {}
    if s["w"] is not None:
        out["dweight"] = (da * p["n"]).sum((0, 1))
    if s["b"] is not None:
        out["dbias"] = da.sum((0, 1))
    dn = (da if s["w"] is None else da * s["w"]).reshape(*x.shape[:-1], s["groups"], -1)
    n = p["n"].reshape(dn.shape)
    dr = dn - n * (dn * n).mean(-1, keepdim=True)
    if not s["rms"]:
        dr = dr - dn.mean(-1, keepdim=True)
    dx = (p["r"] * dr).reshape(x.shape)
    if s["act"] == "gate_first":
        t = torch.sigmoid(z)
        dx, dz = dx * (z * t), dx * x * (t * (1 + z * (1 - t)))
    out["dx"] = dx.to(s["x"].dtype)
    if dz is not None:
        out["dz"] = dz.to(s["x"].dtype)
    return out


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        return _exact_norm(s)
    rep = case["h"] // case["hk"]
    x = {n: s[n].double() for n in ("q", "k", "v", "g", "beta")}
    if op == "update":
        state = s["state"].double()
        rows = range(case["batch"]) if s["slots"] is None else s["slots"].tolist()
        ys = []
        for b, slot in enumerate(rows):
            S, y, _ = _exact_step(state[slot], *(x[n][b] for n in ("q", "k", "v", "g", "beta")), rep, s["scale"])
            state[slot] = S
            ys.append(y)
        return torch.stack(ys), state
    lens, packed = s["lens"], s["cu"] is not None
    tokens = sum(lens) if packed else lens[0]
    if tokens > (80000 if op == "fwd" else 20000):
        return None
    # unpacked batches go through the recurrence side by side, packed sequences one after another
    if not packed:
        return _exact_sequence(s, x, s["h0"], s.get("dhL"), rep, (slice(None), slice(None)))
    parts, first = [], 0
    for i, n in enumerate(lens):
        h0 = None if s["h0"] is None else s["h0"][i:i + 1]
        dhL = s["dhL"][i:i + 1] if s.get("dhL") is not None else None
        parts.append(_exact_sequence(s, x, h0, dhL, rep, (slice(None), slice(first, first + n))))
        first += n
    y, hL = torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts])
    if op == "fwd":
        return y, hL
    grads = {n: torch.cat([p[2][n] for p in parts], 0 if n == "dh0" else 1) for n in parts[0][2]}
    return y, hL, grads


def _exact_step(S, q, k, v, g, beta, rep, scale):
    q, k = q.repeat_interleave(rep, -2), k.repeat_interleave(rep, -2)
    D = torch.exp(g)[..., None, None] * S
    r = v - torch.einsum("...kv,...k->...v", D, k)
    u = beta[..., None] * r
    S = D + k[..., :, None] * u[..., None, :]
    return S, scale * torch.einsum("...kv,...k->...v", S, q), (D, r, u, q, k)


def _exact_sequence(s, x, h0, dhL, rep, at):
    """The recurrence token by token, and its adjoint token by token with the states of 64 steps kept at a time."""
    t = {n: a[at] for n, a in x.items()}
    B, L, h, V = t["v"].shape
    hk, K = t["q"].shape[-2:]
    S = h0.double() if h0 is not None else torch.zeros(B, h, K, V, dtype=torch.float64, device="cuda")
    step = lambda S, i: _exact_step(S, *(t[n][:, i] for n in ("q", "k", "v", "g", "beta")), rep, s["scale"])  # noqa: E731
    y, kept = torch.zeros_like(t["v"]), []
    for i in range(L):
        if s["op"] == "train" and i % CHUNK == 0:
            kept.append(S)
        S, y[:, i], _ = step(S, i)
    if s["op"] == "fwd":
        return y, S
    hL, dy = S, s["dy"][at].double()
    dS = dhL.double() if dhL is not None else torch.zeros_like(S)
    g = {"d" + n: torch.zeros_like(a) for n, a in t.items()}
    fold = lambda a: a.reshape(B, hk, rep, K).sum(2)  # noqa: E731
    for c in reversed(range(len(kept))):
        S, states = kept[c], []
        for i in range(c * CHUNK, min(L, (c + 1) * CHUNK)):
            before = S
            S, _, parts = step(S, i)
            states.append((i, before, S, parts))
        for i, before, S, (D, r, u, q, k) in reversed(states):
            do = s["scale"] * dy[:, i]
            dS = dS + q[..., :, None] * do[..., None, :]
            dq = torch.einsum("bhkv,bhv->bhk", S, do)
            du = torch.einsum("bhkv,bhk->bhv", dS, k)
            dr = t["beta"][:, i][..., None] * du
            dD = dS - k[..., :, None] * dr[..., None, :]
            dk = torch.einsum("bhkv,bhv->bhk", dS, u) - torch.einsum("bhkv,bhv->bhk", D, dr)
            g["dq"][:, i], g["dk"][:, i], g["dv"][:, i] = fold(dq), fold(dk), dr
            g["dbeta"][:, i] = (du * r).sum(-1)
            decay = torch.exp(t["g"][:, i])
            g["dg"][:, i] = decay * (dD * before).sum((-1, -2))
            dS = decay[..., None, None] * dD
    g["dh0"] = dS
    return y, hL, g


def _exact_norm(s):
    """The definition in 64 bits; its gradients through autograd."""
    given = {n: s[n].double().requires_grad_(s["op"] == "norm_bwd") for n in ("x", "z", "w", "b") if s[n] is not None}
    x, z = given["x"], given.get("z")
    silu = torch.nn.functional.silu
    a = x * silu(z) if s["act"] == "gate_first" else x
    a = a.unflatten(-1, (s["groups"], -1))
    mean = 0 if s["rms"] else a.mean(-1, keepdim=True)
    a = ((a - mean) / torch.sqrt(((a - mean) ** 2).mean(-1, keepdim=True) + s["eps"])).flatten(-2)
    a = a * given["w"] if "w" in given else a
    a = a + given["b"] if "b" in given else a
    y = silu(a) if s["act"] == "silu" else a * silu(z) if s["act"] == "gate" else a
    if s["op"] == "norm":
        return y
    names = {"x": "dx", "z": "dz", "w": "dweight", "b": "dbias"}
    grads = torch.autograd.grad(y, list(given.values()), s["dy"].double())
    return {names[n]: v for n, v in zip(given, grads)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 4 if case["dtype"] == F32 else 2
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n = case["batch"] * case["L"] * case["dim"]
        gate = case["act"].startswith("gate")
        if op == "norm":
            return {"bytes": n * e * (3 if gate else 2) + 4 * case["dim"], "flops": n * (14 if gate else 8)}
        return {"bytes": n * e * (5 if gate else 3) + 8 * case["dim"], "flops": n * (30 if gate else 16)}
    hk, h, K, V = case["hk"], case["h"], case["K"], case["V"]
    if op == "update":
        b = case["batch"]
        return {"bytes": b * (8 * h * K * V + e * (2 * hk * K + 2 * h * V) + 8 * h), "flops": 7 * b * h * K * V}
    lens = _lens(case)
    tokens = sum(lens)
    state = 4 * len(lens) * h * K * V
    fwd = tokens * (e * (2 * hk * K + 2 * h * V) + 8 * h) + state * (2 if case["h0"] else 1)
    if op == "fwd":
        return {"bytes": fwd, "flops": 7 * tokens * h * K * V}
    # q, k, v, dy, g, beta in; dq, dk, dv, dg, dbeta out
    bwd = tokens * (e * (4 * hk * K + 3 * h * V) + 16 * h) + state * (3 if case["h0"] else 1)
    return {"bytes": fwd + bwd, "flops": 27 * tokens * h * K * V}
