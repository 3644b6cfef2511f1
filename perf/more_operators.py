"""The selective scan with one decay a head, and the residual norm in front of
it: the calls that are timed, in their plain form and through the package.

Five operators, as a layer of a language model uses them.  Per head, with
inputs and readouts B, C of N entries that the heads of a group share, a value
x of P entries and a state S of N x P:

    D_t = softplus(dt_t + dt_bias),  S_t = e^{D_t A} S_{t-1} + D_t B_t x_t^T
    y_t = S_t^T C_t + Dskip x_t

  fwd       whole sequences (prompts): y and the last state
  train     the same with its gradients: a training step's forward and backward
  update    one new token per sequence on a persistent state
  norm      h = x + residual, y = h / rms(h) * w, in 8 bits with a scale for
            every 128 channels where the projection behind it takes those
  norm_bwd  its gradients, joined with the one that comes down the residual

``run`` computes them from elementary torch operations in float32 (``own``
false) or by calling the package (``own`` true).
"""
import torch

own = False

F32, BF16, E4M3 = "f32", "bf16", "e4m3"
TYPES = {F32: torch.float32, BF16: torch.bfloat16, E4M3: torch.float8_e4m3fn}
CHUNK, BLOCK = 64, 128


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a few tokens of a small model: the launch and one chunk
        dict(name="fwd short f32", op="fwd", dtype=F32, lens="17", packed=False, groups=2, h=4, N=32, P=40, h0=True),
        # a prompt batch through a layer of 5120 channels
        dict(name="fwd layer bf16", op="fwd", dtype=BF16, lens="2048,2048,2048,2048", packed=False, groups=1, h=80,
             N=128, P=64, h0=False),
        # prompts of unequal lengths packed into one batch row, 1536 channels in two groups
        dict(name="fwd packed bf16", op="fwd", dtype=BF16, lens="4097,1,2500,0,63,6001,777,2945", packed=True,
             groups=2, h=24, N=128, P=64, h0=True),
        # one long document: few heads, a long recurrence
        dict(name="fwd long bf16", op="fwd", dtype=BF16, lens="65521", packed=False, groups=1, h=24, N=128, P=64,
             h0=False),
        # a training step of the layer
        dict(name="train layer bf16", op="train", dtype=BF16, lens="2048,2048,2048,2048", packed=False, groups=1,
             h=80, N=128, P=64, h0=False),
        # fp32 training of a small model, a length that no tile divides
        dict(name="train odd f32", op="train", dtype=F32, lens="777,777", packed=False, groups=2, h=6, N=64, P=96,
             h0=True),
        # one user's next token
        dict(name="update one bf16", op="update", dtype=BF16, batch=1, slots=0, groups=1, h=80, N=128, P=64),
        # a serving batch whose states sit in a pool of slots
        dict(name="update batch bf16", op="update", dtype=BF16, batch=64, slots=80, groups=1, h=80, N=128, P=64),
        # the layer's entrance in a prompt: an fp32 residual stream, the projection behind it in 8 bits
        dict(name="norm layer e4m3", op="norm", dtype=BF16, stream=F32, out=E4M3, rows=8192, dim=2560),
        # the same for one decoded batch, the projection in bf16
        dict(name="norm step bf16", op="norm", dtype=BF16, stream=F32, out=BF16, rows=8, dim=2560),
        # gradients of the layer's entrance
        dict(name="norm_bwd layer bf16", op="norm_bwd", dtype=BF16, stream=F32, rows=8192, dim=2560),
        # rows that no vector access divides, the first norm of a model: nothing comes down a residual
        dict(name="norm_bwd odd f32", op="norm_bwd", dtype=F32, stream="", rows=999, dim=1531),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "train", "update", "norm", "norm_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("fwd", "train", "update"):
        groups = rng.choice([1, 1, 2, 3, 4, 8])
        h = groups * rng.randint(1, 80 // groups)
        N = rng.choice([128, 128, 64, 256, 16, rng.randint(1, 256)])
        P = rng.choice([64, 64, 128, 32, 96, rng.randint(1, 160)])
        case = dict(op=op, dtype=dtype, groups=groups, h=h, N=N, P=P)
        if op == "update":
            batch = _log(rng, 1, 64)
            while batch > 1 and batch * h * N * P > 64 * 80 * 128 * 64:
                batch //= 2
            return dict(case, batch=batch, slots=rng.choice([0, batch + rng.randint(0, 16)]))
        # the listed layer has 4 x 2048 tokens of 80 heads of 128 x 64
        most = 4 * 2048 * 80 * 128 * 64 // (1 if dtype == BF16 else 8)
        tokens = max(1, min(_log(rng, 1, 65521 if op == "fwd" else 16384), most // (h * max(N, 32) * max(P, 32))))
        n = min(tokens, rng.choice([1, 1, 2, 3, 4, 7, 16]))
        packed = rng.random() < 0.4
        if packed:
            cuts = sorted(rng.randint(0, tokens) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
        else:
            lens = [tokens // n] * n
        return dict(case, lens=",".join(map(str, lens)), packed=packed, h0=rng.random() < 0.5)
    dim = rng.choice([2560, 768, 1536, 5120, 8192, rng.randint(1, 6000)])
    rows = _log(rng, 1, min(65536, 8192 * 2560 // dim // (1 if dtype == BF16 else 2)))
    case = dict(op=op, dtype=dtype, stream=rng.choice([F32, F32, BF16, ""]), rows=rows, dim=dim)
    return dict(case, out=rng.choice([E4M3, E4M3, BF16, F32])) if op == "norm" else case


# ------------------------------------------------------------------ the inputs
def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if op in ("norm", "norm_bwd"):
        shape, stream = (case["rows"], case["dim"]), TYPES.get(case["stream"])
        s = dict(op=op, w=1 + 0.1 * normal(case["dim"]), eps=1e-5)
        # a residual stream grows over the layers; a few of its channels are far larger than the rest
        wide = (1 + 30 * (uniform(case["dim"]) < 0.004)) if stream else 1.0
        if op == "norm":
            return dict(s, x=normal(*shape).to(dt), residual=(3 * wide * normal(*shape)).to(stream) if stream else None,
                        out=TYPES[case["out"]])
        return dict(s, h=(3 * wide * normal(*shape)).to(stream or dt), dy=normal(*shape).to(dt),
                    dh=normal(*shape).to(stream) if stream else None)

    groups, h, N, P = case["groups"], case["h"], case["N"], case["P"]
    if op == "update":
        shape = (case["batch"],)
    elif case["packed"]:
        shape = (1, sum(_lens(case)))
    else:
        shape = (len(_lens(case)), _lens(case)[0])
    silu = torch.nn.functional.silu
    # x, B and C leave a short convolution and a silu
    s = dict(op=op, x=silu(normal(*shape, h, P)).to(dt), B=silu(normal(*shape, groups, N)).to(dt),
             C=silu(normal(*shape, groups, N)).to(dt), dt=normal(*shape, h).to(dt), D=1 + 0.1 * normal(h),
             A=-(1 + 15 * uniform(h)),  # decay rates in [1, 16]
             # steps of softplus(dt + bias), the bias placed for steps in [1e-3, 1e-1]
             bias=torch.log(torch.expm1(torch.exp(uniform(h) * 4.605 - 6.908))))
    if op == "update":
        n = case["slots"]
        s["state"] = 0.3 * normal(n or case["batch"], h, N, P)
        s["slots"] = torch.randperm(n, generator=gen, device="cuda")[:case["batch"]].int() if n else None
        return s
    lens = _lens(case)
    s["h0"] = 0.3 * normal(len(lens), h, N, P) if case["h0"] else None
    s["lens"], s["cu"] = lens, None
    if case["packed"]:
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    if op == "train":
        s["dy"] = normal(*shape, h, P).to(dt)
        s["dhL"] = 0.3 * normal(len(lens), h, N, P) if case["h0"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _call(s) if own else _plain(s)


def _call(s):
    import selective_state_space_64_amd as ssm

    op = s["op"]
    if op == "norm":
        return ssm.ssm_rms_norm_fwd(s["x"], weight=s["w"], residual=s["residual"], eps=s["eps"], out_dtype=s["out"])
    if op == "norm_bwd":
        return ssm.ssm_rms_norm_bwd(s["h"], s["dy"], weight=s["w"], dh=s["dh"], eps=s["eps"])
    args, kw = (s["x"], s["dt"], s["A"], s["B"], s["C"]), dict(Dskip=s["D"], dt_bias=s["bias"])
    if op == "update":
        return ssm.ssm_head_scan_update(s["state"], *args, slots=s["slots"], **kw), s["state"]
    kw.update(h0=s["h0"], cu_seqlens=s["cu"])
    if op == "fwd":
        return ssm.ssm_head_scan_fwd(*args, **kw)
    ws = ssm.ssm_head_scan_bwd_workspace(s["x"], s["B"], cu_seqlens=s["cu"])
    y, hL = ssm.ssm_head_scan_fwd(*args, checkpoints=ws, **kw)
    return y, hL, ssm.ssm_head_scan_bwd(*args, s["dy"], dhL=s["dhL"], workspace=ws, checkpoints_in_workspace=True, **kw)


def _plain(s):
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "update": _plain_update}.get(s["op"], _plain_scan)(s)


def _softplus(u):
    return torch.logaddexp(u, torch.zeros_like(u))


def _plain_update(s):
    h, groups = s["x"].shape[-2], s["B"].shape[-2]
    x, B, C = s["x"].float(), *(s[n].float().repeat_interleave(h // groups, dim=-2) for n in ("B", "C"))
    step = _softplus(s["dt"].float() + s["bias"])
    at = slice(None) if s["slots"] is None else s["slots"].long()
    S = s["state"][at] * (step * s["A"]).exp()[..., None, None] + (step[..., None] * B)[..., None] * x[..., None, :]
    y = (S * C[..., None]).sum(-2) + s["D"][:, None] * x
    s["state"][at] = S
    return y.to(s["x"].dtype), s["state"]


def _chunks(x, s):
    """[batch, L, heads, ...] -> [sequences, heads, chunks, 64, ...] in float32, zeros behind each sequence's end."""
    lens = s["lens"]
    n = max(1, -(-max(lens) // CHUNK))
    at = torch.arange(n * CHUNK, device=x.device)[None, :]
    size = torch.tensor(lens, device=x.device)[:, None]
    if s["cu"] is not None:
        flat = x.reshape(-1, *x.shape[2:]).float()
        out = flat[(s["cu"][:-1, None].long() + at).clamp(max=flat.shape[0] - 1)]
    else:
        out = x.float()[:, at[0].clamp(max=x.shape[1] - 1)]
    there = (at < size).reshape(len(lens), n * CHUNK, *[1] * (out.dim() - 2))
    out = torch.where(there, out, 0.0).transpose(1, 2)
    return out.reshape(*out.shape[:2], n, CHUNK, *out.shape[3:])


def _steps(x, s):
    """The way back of _chunks, to [batch, L, heads, ...]."""
    x = x.reshape(*x.shape[:2], -1, *x.shape[4:]).transpose(1, 2)
    if s["cu"] is not None:
        at = torch.arange(x.shape[1], device=x.device)[None, :]
        return x[at < torch.tensor(s["lens"], device=x.device)[:, None]][None]
    return x[:, :s["x"].shape[1]]


def _plain_scan(s):
    """64 steps at a time by matrix products, and the chunks' states by another over the chunks."""
    h, groups = s["x"].shape[-2], s["B"].shape[-2]
    u = s["dt"].float() + s["bias"]
    x, step = _chunks(s["x"], s), _chunks(_softplus(u), s)
    B, C = (_chunks(s[n], s).repeat_interleave(h // groups, dim=1) for n in ("B", "C"))
    t = lambda a: a.transpose(-1, -2)  # noqa: E731
    G = (step.double() * s["A"].double()[:, None, None]).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    decay = torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf).exp().float()
    M = decay * (C @ t(B))
    W = M * step[..., None, :]
    eG, tail = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    # the state entering chunk c (and, as the last of them, the final one) from all chunks before it
    ends = torch.cat([torch.zeros_like(G[..., :1, -1]), G[..., -1].cumsum(-1)], -1)
    n = ends.shape[-1] - 1
    past = torch.ones(n + 1, n, dtype=torch.bool, device=G.device).tril(-1)
    T = torch.where(past, ends[..., :, None] - ends[..., None, 1:], -torch.inf).exp().float()
    Z = t(step[..., None] * tail * B) @ x
    S = (T @ Z.flatten(-2)).unflatten(-1, Z.shape[-2:])
    first = ends.exp().float()[..., None, None]
    if s["h0"] is not None:
        S = S + first * s["h0"][:, :, None]
    S0, hL = S[:, :, :-1], S[:, :, -1]
    skip = s["D"][:, None, None, None]
    y = _steps(eG * (C @ S0) + W @ x + skip * x, s).to(s["x"].dtype)
    if s["op"] == "fwd":
        return y, hL.contiguous()

    dy = _chunks(s["dy"], s)
    Z = t(eG * C) @ dy
    last = s["dhL"][:, :, None] if s["dhL"] is not None else torch.zeros_like(Z[:, :, :1])
    Z = torch.cat([Z, last], 2)
    dS1 = (t(T) @ Z.flatten(-2)).unflatten(-1, Z.shape[-2:])
    dh0 = (first * Z).sum(2)
    dx = t(W) @ dy + step[..., None] * tail * (B @ dS1) + skip * dy
    dM = dy @ t(x)
    Sdy, dSx = eG * (dy @ t(S0)), tail * (x @ t(dS1))
    Q = dM * decay * step[..., None, :]
    dC, dB = Q @ B + Sdy, t(Q) @ C + step[..., None] * dSx
    # d/dG of every exponential, then G = cumsum(step A)
    dstep = (dM * M).sum(-2) + (B * dSx).sum(-1)
    dG = (dM * W).sum(-1) + (C * Sdy).sum(-1) - dstep * step
    dG[..., -1] += ((B * dSx).sum(-1) * step).sum(-1) + G[..., -1].exp().float() * (S0 * dS1).sum((-1, -2))
    da = dG.double().flip(-1).cumsum(-1).flip(-1).float()
    ddt = _steps(dstep + s["A"][:, None, None] * da, s) * torch.sigmoid(u)
    per = lambda a: _steps(a, s).unflatten(2, (groups, h // groups)).sum(3).to(s["x"].dtype)  # noqa: E731
    f32 = dict(dA=(step * da).sum((0, 2, 3)), dDskip=(dy * x).sum((0, 2, 3, 4)), ddt_bias=ddt.sum((0, 1)), dh0=dh0)
    return y, hL.contiguous(), dict(f32, dx=_steps(dx, s).to(s["x"].dtype), ddt=ddt.to(s["x"].dtype), dBm=per(dB),
                                    dCm=per(dC))


def _plain_norm(s):
    x = s["x"].float()
    h = x if s["residual"] is None else x + s["residual"].float()
    y = h * ((h * h).mean(-1, keepdim=True) + s["eps"]).rsqrt() * s["w"]
    stream = None if s["residual"] is None else h.to(s["residual"].dtype)
    if s["out"] != torch.float8_e4m3fn:
        return y.to(s["out"]), stream, None
    rows, dim = y.shape
    blocks = torch.nn.functional.pad(y, (0, -dim % BLOCK)).reshape(rows, -1, BLOCK)
    scales = (blocks.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    q = (blocks / scales[..., None]).reshape(rows, -1)[:, :dim].contiguous()
    return q.to(s["out"]), stream, scales


def _plain_norm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = ((h * h).mean(-1, keepdim=True) + s["eps"]).rsqrt()
    n, u = h * r, dy * s["w"]
    dh = r * (u - n * (u * n).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
    return dict(dx=dh.to(s["dy"].dtype), dresidual=None if s["dh"] is None else dh.to(s["h"].dtype),
                dweight=(dy * n).sum(0))


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_bwd":
        return _exact_norm_bwd(s)
    x = {n: s[n].double() for n in ("x", "dt", "A", "B", "C", "D", "bias")}
    if op == "update":
        state, ys = s["state"].double(), []
        rows = range(case["batch"]) if s["slots"] is None else s["slots"].tolist()
        for b, slot in enumerate(rows):
            state[slot], y = _exact_step(state[slot], x, (b,))
            ys.append(y)
        return torch.stack(ys), state
    lens, packed = s["lens"], s["cu"] is not None
    if (sum(lens) if packed else lens[0]) > (80000 if op == "fwd" else 20000):
        return None
    # unpacked batches go through the recurrence side by side, packed sequences one after another
    if not packed:
        return _exact_sequences(s, x, s["h0"], s.get("dhL"), (slice(None),), 0, lens[0])
    parts, at = [], 0
    for i, n in enumerate(lens):
        one = [None if s.get(k) is None else s[k][i:i + 1] for k in ("h0", "dhL")]
        parts.append(_exact_sequences(s, x, *one, (slice(None),), at, n))
        at += n
    y, hL = torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts])
    if op == "fwd":
        return y, hL
    total = lambda k: sum(p[2][k] for p in parts)  # noqa: E731
    join = lambda k: torch.cat([p[2][k] for p in parts], 0 if k == "dh0" else 1)  # noqa: E731
    return y, hL, {k: (total if k in ("dA", "dDskip", "ddt_bias") else join)(k) for k in parts[0][2]}


def _exact_step(S, x, at):
    """S after the step at index `at`, and the step's output."""
    rep = S.shape[-3] // x["B"].shape[-2]
    v, B, C = x["x"][at], *(x[n][at].repeat_interleave(rep, -2) for n in ("B", "C"))
    step = torch.nn.functional.softplus(x["dt"][at] + x["bias"], threshold=200)
    S = torch.exp(step * x["A"])[..., None, None] * S + step[..., None, None] * B[..., :, None] * v[..., None, :]
    return S, torch.matmul(C[..., None, :], S)[..., 0, :] + x["D"][:, None] * v


def _exact_sequences(s, x, h0, dhL, lead, first, L):
    """The recurrence token by token, and its adjoint token by token with the states of 64 steps kept at a time."""
    Bt, _, h, P = s["x"].shape
    groups, N = s["B"].shape[-2:]
    rep = h // groups
    S = h0.double() if h0 is not None else torch.zeros(Bt, h, N, P, dtype=torch.float64, device="cuda")
    y, kept = torch.zeros(Bt, L, h, P, dtype=torch.float64, device="cuda"), []
    for i in range(L):
        if s["op"] == "train" and i % CHUNK == 0:
            kept.append(S)
        S, y[:, i] = _exact_step(S, x, (*lead, first + i))
    if s["op"] == "fwd":
        return y, S
    hL, dy = S, s["dy"][:, first:first + L].double()
    dS = dhL.double() if dhL is not None else torch.zeros_like(S)
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    g = dict(dx=new(Bt, L, h, P), ddt=new(Bt, L, h), dBm=new(Bt, L, groups, N), dCm=new(Bt, L, groups, N), dA=new(h),
             dDskip=new(h), ddt_bias=new(h))
    fold = lambda a: a.reshape(Bt, groups, rep, N).sum(2)  # noqa: E731
    for c in reversed(range(len(kept))):
        S, states = kept[c], []
        for i in range(c * CHUNK, min(L, (c + 1) * CHUNK)):
            before = S
            S, _ = _exact_step(S, x, (*lead, first + i))
            states.append((i, before, S))
        for i, before, S in reversed(states):
            at = (*lead, first + i)
            v, B, C = x["x"][at], *(x[n][at].repeat_interleave(rep, -2) for n in ("B", "C"))
            u = x["dt"][at] + x["bias"]
            step = torch.nn.functional.softplus(u, threshold=200)
            decay = torch.exp(step * x["A"])
            dyi = dy[:, i]
            dS = dS + C[..., :, None] * dyi[..., None, :]
            g["dCm"][:, i] = fold(torch.matmul(S, dyi[..., None])[..., 0])
            dSv, dSB = torch.matmul(dS, v[..., None])[..., 0], torch.matmul(B[..., None, :], dS)[..., 0, :]
            g["dBm"][:, i] = fold(step[..., None] * dSv)
            g["dx"][:, i] = step[..., None] * dSB + x["D"][:, None] * dyi
            da = decay * (dS * before).sum((-1, -2))
            ddt = ((B * dSv).sum(-1) + x["A"] * da) * torch.sigmoid(u)
            g["ddt"][:, i] = ddt
            g["dA"] += (step * da).sum(0)
            g["dDskip"] += (dyi * v).sum((0, 2))
            g["ddt_bias"] += ddt.sum(0)
            dS = decay[..., None, None] * dS
    return y, hL, dict(g, dh0=dS)


def _exact_norm(s):
    x = s["x"].double()
    h = x if s["residual"] is None else x + s["residual"].double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["w"].double()
    stream = None if s["residual"] is None else h
    if s["out"] != torch.float8_e4m3fn:
        return y, stream, None
    scales = torch.stack([b.abs().amax(-1) / 448 for b in y.split(BLOCK, -1)], -1).clamp(min=2.0 ** -126)
    return y / scales.repeat_interleave(BLOCK, -1)[:, :y.shape[1]], stream, scales


def _exact_norm_bwd(s):
    """The definition in 64 bits; its gradients through autograd."""
    h, w = s["h"].double().requires_grad_(), s["w"].double().requires_grad_()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * w
    dh, dw = torch.autograd.grad(y, (h, w), s["dy"].double())
    if s["dh"] is not None:
        dh = dh + s["dh"].double()
    return dict(dx=dh, dresidual=None if s["dh"] is None else dh, dweight=dw)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {F32: 4, BF16: 2, E4M3: 1, "": 0}
    e, op = size[case["dtype"]], case["op"]
    if op in ("norm", "norm_bwd"):
        rows, dim, stream = case["rows"], case["dim"], size[case["stream"]]
        n = rows * dim
        if op == "norm":
            scales = 4 * rows * -(-dim // BLOCK) if case["out"] == E4M3 else 0
            return {"bytes": n * (e + 2 * stream + size[case["out"]]) + scales + 4 * dim, "flops": n * 5}
        return {"bytes": n * ((stream or e) + 2 * e + 2 * stream) + 8 * dim, "flops": n * 11}
    groups, h, N, P = case["groups"], case["h"], case["N"], case["P"]
    if op == "update":
        b = case["batch"]
        return {"bytes": b * (8 * h * N * P + e * (2 * groups * N + 2 * h * P + h)), "flops": 5 * b * h * N * P}
    lens = _lens(case)
    tokens, state = sum(lens), 4 * len(lens) * h * N * P
    fwd = tokens * e * (2 * groups * N + 2 * h * P + h) + state * (2 if case["h0"] else 1)
    if op == "fwd":
        return {"bytes": fwd, "flops": 5 * tokens * h * N * P}
    # x, dy, B, C, dt in; dx, dB, dC, ddt out
    bwd = tokens * e * (4 * groups * N + 3 * h * P + 2 * h) + state * (3 if case["h0"] else 1)
    return {"bytes": fwd + bwd, "flops": 19 * tokens * h * N * P}
