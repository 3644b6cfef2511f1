"""The gated delta rule on the GPU (ssm_delta_fwd, ssm_delta_bwd,
ssm_delta_update) against the plain fp64 recurrence.

Error of a tensor: max |got - ref| / max(|ref|, rms(ref)).  Tolerances, from
the kernels' arithmetic:
  * fp32 inputs with K <= 128 keep 24 bits in every product (three bf16 terms)
    and sum in fp32: a value passes about 4 chained products of up to 256
    summands, 4 x sqrt(256) x 2^-24 = 4e-6 rms, 5 times that at the largest of
    ~1e5 elements: 2e-5.
  * two terms (bf16 inputs, or K > 128) leave at most 2^-17 of each operand,
    two operands in each of 4 chained products, 5 times their rms 2^-17/sqrt(3)
    x sqrt(8) at the largest element: 6e-5, doubled for the operands being
    larger than the result where terms cancel: 1.2e-4.
  * dg sums differences of such terms over the steps behind it: 4 times that.
  * a bf16 output adds half an ulp: half of torch.finfo(bfloat16).eps, 2^-8.
"""
import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from delta_reference import delta_batch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def tolerance(dtype, out, K, name=""):
    t = 2e-5 if dtype == F32 and K <= 128 else 1.2e-4
    t *= 4 if name == "dg" else 1
    return t + (torch.finfo(BF16).eps / 2 if out == BF16 else 0.0)


def error(got, ref):
    got, ref = got.double().cpu().numpy(), np.asarray(ref)
    assert got.shape == ref.shape and np.isfinite(got).all()
    if not ref.size:
        return 0.0
    rms = np.sqrt(np.mean(ref * ref))
    if rms == 0:
        return float(np.max(np.abs(got)))
    return float(np.max(np.abs(got - ref) / np.maximum(np.abs(ref), rms)))


def make(dtype, lens, packed, hk, h, K, V, seed=0, state=True, decay="mixed", keys="unit"):
    rng = np.random.default_rng(seed)
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    n = rng.standard_normal
    q, k, v = n((*lead, hk, K)), n((*lead, hk, K)), n((*lead, h, V))
    if keys == "unit":
        k /= np.linalg.norm(k, axis=-1, keepdims=True)
    elif keys == "same":  # one direction: M is full, the substitution's worst case that stays bounded
        k[:] = k[:, :1] / np.linalg.norm(k[:, :1], axis=-1, keepdims=True)
    beta = 1 / (1 + np.exp(-n((*lead, h))))
    g = {"mixed": -rng.exponential(0.3, (*lead, h)), "none": np.zeros((*lead, h)),
         "strong": -rng.uniform(0, 60, (*lead, h))}["mixed" if decay == "reset" else decay]
    if decay == "reset":
        g[rng.random(g.shape) < 0.1] = -np.inf
        beta[rng.random(g.shape) < 0.1] = 0.0
    t = {"q": torch.tensor(q).to(dtype), "k": torch.tensor(k).to(dtype), "v": torch.tensor(v).to(dtype),
         "g": torch.tensor(g, dtype=F32), "beta": torch.tensor(beta, dtype=F32),
         "dy": torch.tensor(n((*lead, h, V))).to(dtype),
         "h0": torch.tensor(n((len(lens), h, K, V)), dtype=F32) if state else None,
         "dhL": torch.tensor(n((len(lens), h, K, V)), dtype=F32) if state else None}
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32) if packed else None
    ref = {m: None if x is None else x.double().numpy() for m, x in t.items()}
    dev = {m: None if x is None else x.cuda() for m, x in t.items()}
    return dev, ref, None if cu is None else cu.cuda()


ARGS = ("q", "k", "v", "g", "beta")

#       dtype lens packed hk h K V options
CASES = [
    (F32, [1], False, 1, 1, 1, 1, {}),
    (F32, [1, 1, 1], False, 1, 2, 5, 3, {}),
    (BF16, [2, 2], False, 2, 2, 16, 17, dict(state=False)),
    (F32, [63], False, 2, 6, 64, 80, {}),
    (BF16, [64], False, 1, 3, 128, 128, {}),
    (F32, [65, 65], False, 3, 3, 33, 64, dict(decay="none")),
    (BF16, [130], False, 2, 4, 100, 40, dict(decay="reset")),
    (F32, [200], False, 1, 2, 128, 65, dict(decay="reset")),
    (F32, [129], False, 1, 2, 200, 24, {}),
    (BF16, [321], False, 2, 2, 256, 130, {}),
    (F32, [150], False, 1, 1, 256, 70, dict(state=False)),
    (BF16, [257], False, 4, 4, 72, 200, dict(decay="strong")),
    (F32, [257], False, 1, 2, 96, 33, dict(decay="strong")),
    (F32, [190], False, 1, 2, 64, 48, dict(keys="same", decay="none")),
    (BF16, [3, 0, 64, 1, 65, 0, 128, 10], True, 2, 4, 64, 72, {}),
    (F32, [100, 1, 37], True, 1, 2, 48, 16, {}),
    (F32, [0, 5, 0], True, 1, 1, 16, 8, {}),
    (BF16, [700, 324], True, 1, 2, 128, 64, dict(state=False)),
]


# sequences that the library cuts into segments (few heads, many chunks)
SPLIT = [
    (BF16, [2500], False, 1, 1, 128, 64, {}),
    (F32, [1100], False, 1, 2, 64, 40, dict(decay="none")),
    (F32, [1601], False, 1, 1, 100, 130, dict(decay="reset")),
    (BF16, [1500, 1500], False, 1, 2, 40, 200, dict(state=False)),
    (BF16, [1090], False, 1, 1, 256, 20, {}),
    (F32, [1153], False, 1, 1, 200, 10, {}),
    (BF16, [700, 0, 1, 1500, 64, 900], True, 1, 2, 64, 48, {}),
    (F32, [1024, 1025], True, 1, 1, 32, 16, dict(state=False, decay="strong")),
]


def name(c):
    return "%s-L%s%s-h%d.%d-K%d-V%d-%s" % (str(c[0])[6:], ".".join(map(str, c[1])), "p" if c[2] else "", c[3], c[4], c[5],
                                           c[6], "-".join(str(v) for v in c[7].values()))


@pytest.mark.parametrize("case", SPLIT, ids=name)
def test_split_sequences(case):
    dtype, lens, packed, hk, h, K, V, opt = case
    need = ssm.lib().ssm_delta_fwd_workspace_bytes
    size = (1 if packed else len(lens), sum(lens) if packed else lens[0], hk, h, K, V, len(lens) if packed else 0)
    # the split's planes are in the workspace: more than the chunks' share of a long batch's
    chunks = lambda b, L, n: (L + 63) // 64 + n if n else b * ((L + 63) // 64)  # noqa: E731
    wide = (512, 640, hk, h, K, V, 0)
    per = need(*wide) / chunks(512, 640, 0)
    assert need(*size) > 1.01 * per * chunks(size[0], size[1], size[6])
    test_forward_and_gradients(case)


# enough heads x sequences that eight waves share a workgroup
@pytest.mark.parametrize("case", [(BF16, [70] * 44, False, 1, 3, 128, 80, {}),
                                  (BF16, [65, 0, 130] * 12, True, 2, 4, 48, 72, dict(decay="reset"))],
                         ids=["44 x 3 heads", "packed 36 x 4 heads"])
def test_many_heads(case):
    test_forward_and_gradients(case)


@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward_and_gradients(case):
    dtype, lens, packed, hk, h, K, V, opt = case
    t, r, cu = make(dtype, lens, packed, hk, h, K, V, seed=len(name(case)), **opt)
    scale = K ** -0.5
    y0, h0, d0 = delta_batch(*(r[n] for n in ARGS), scale, lens if packed else None, r["h0"], r["dy"], r["dhL"])
    args = [t[n] for n in ARGS]
    kw = dict(h0=t["h0"], cu_seqlens=cu)
    y, hL = ssm.ssm_delta_fwd(*args, **kw)
    assert error(y, y0) <= tolerance(dtype, dtype, K)
    assert error(hL, h0) <= tolerance(dtype, F32, K)
    yf, _ = ssm.ssm_delta_fwd(*args, out_dtype=F32, return_final_state=False, **kw)
    assert error(yf, y0) <= tolerance(dtype, F32, K)
    # the same bits with checkpoints, and the same gradients from either start
    ws = ssm.ssm_delta_bwd_workspace(t["q"], t["v"], cu_seqlens=cu)
    yc, hc = ssm.ssm_delta_fwd(*args, checkpoints=ws, **kw)
    assert torch.equal(yc, y) and torch.equal(hc, hL)
    d = ssm.ssm_delta_bwd(*args, t["dy"], dhL=t["dhL"], workspace=ws, checkpoints_in_workspace=True, **kw)
    e = ssm.ssm_delta_bwd(*args, t["dy"], dhL=t["dhL"], **kw)
    for n in d0:
        assert torch.equal(d[n], e[n]), n
        out = dtype if n in ("dq", "dk", "dv") else F32
        assert error(d[n], d0[n]) <= tolerance(dtype, out, K, n), n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_mixed_types(dtype):
    """fp32 gradients of bf16 inputs and the other way round."""
    other = BF16 if dtype == F32 else F32
    t, r, _ = make(dtype, [150], False, 1, 2, 64, 72)
    t["dy"], r["dy"] = t["dy"].to(other), t["dy"].to(other).double().cpu().numpy()
    y0, h0, d0 = delta_batch(*(r[n] for n in ARGS), 64 ** -0.5, None, r["h0"], r["dy"], r["dhL"])
    args = [t[n] for n in ARGS]
    y, _ = ssm.ssm_delta_fwd(*args, h0=t["h0"], out_dtype=other)
    assert y.dtype == other and error(y, y0) <= tolerance(dtype, other, 64)
    d = ssm.ssm_delta_bwd(*args, t["dy"], h0=t["h0"], dhL=t["dhL"])
    for n in d0:
        assert error(d[n], d0[n]) <= tolerance(dtype, d[n].dtype, 64, n), n


@pytest.mark.parametrize("order", ["projection", "heads_first", "odd"])
def test_strides(order):
    """Slices of one projection, [batch, heads, L, .] tensors and rows that no
    16-byte access fits give the dense call's bits."""
    dtype, B, L, hk, h, K, V = BF16, 2, 150, 2, 4, 64, 72
    t, _, _ = make(dtype, [L] * B, False, hk, h, K, V, seed=5)
    dense = [t[n] for n in ARGS]
    y0, h0 = ssm.ssm_delta_fwd(*dense, h0=t["h0"])
    d0 = ssm.ssm_delta_bwd(*dense, t["dy"], h0=t["h0"], dhL=t["dhL"])
    kw = {}
    if order == "heads_first":
        move = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
        args = [move(x) for x in dense]
        dy = move(t["dy"])
        y = torch.empty(B, h, L, V, dtype=dtype, device="cuda").transpose(1, 2)
        kw = {n: torch.empty(B, heads, L, w, dtype=dtype, device="cuda").transpose(1, 2)
              for n, heads, w in (("dq", hk, K), ("dk", hk, K), ("dv", h, V))}
    else:
        pad = 3 if order == "odd" else 0
        sizes = [hk * K, hk * K, h * V]
        row = torch.full((B, L, sum(sizes) + pad), float("nan"), dtype=dtype, device="cuda")
        out = torch.full_like(row, float("nan"))
        parts, outs, at = [], [], pad
        for n, x in zip(sizes, dense):
            part = row[..., at:at + n].unflatten(-1, x.shape[2:])
            part.copy_(x)
            parts.append(part)
            outs.append(out[..., at:at + n].unflatten(-1, x.shape[2:]))
            at += n
        gates = torch.empty(B, L, 2 * h + 1, device="cuda")
        gates[..., :h], gates[..., h + 1:] = t["g"], t["beta"]
        args = [*parts, gates[..., :h], gates[..., h + 1:]]
        wide = torch.full((B, L, h, V + 1), float("nan"), dtype=dtype, device="cuda")
        dy = wide[..., :V] if order == "odd" else t["dy"]
        dy.copy_(t["dy"])
        y = torch.empty(B, L, h, V + 5, dtype=dtype, device="cuda")[..., 5:]
        kw = dict(zip(("dq", "dk", "dv"), outs))
    ws = ssm.ssm_delta_bwd_workspace(args[0], args[2])
    y1, h1 = ssm.ssm_delta_fwd(*args, h0=t["h0"], y=y, checkpoints=ws)
    assert torch.equal(y1, y0) and torch.equal(h1, h0)
    d1 = ssm.ssm_delta_bwd(*args, dy, h0=t["h0"], dhL=t["dhL"], workspace=ws, checkpoints_in_workspace=True, **kw)
    for n in d0:
        assert torch.equal(d1[n], d0[n]), n


@pytest.mark.parametrize("dtype,K,V", [(F32, 64, 40), (BF16, 128, 64)])
def test_resume_and_decode(dtype, K, V):
    """A sequence in pieces, its state handed on (in place), and its last steps one by one."""
    L, cuts = 200, [0, 1, 70, 190]
    t, r, _ = make(dtype, [L, L], False, 2, 4, K, V, seed=3)
    y0, h0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, r["h0"])
    state, ys = t["h0"].clone(), []
    for a, b in zip(cuts, cuts[1:]):
        y, hL = ssm.ssm_delta_fwd(*(t[n][:, a:b] for n in ARGS), h0=state, hL=state, out_dtype=F32)
        assert hL is state
        ys.append(y)
    for i in range(cuts[-1], L):
        ys.append(ssm.ssm_delta_update(state, *(t[n][:, i] for n in ARGS), out_dtype=F32)[:, None])
    assert error(torch.cat(ys, 1), y0) <= tolerance(dtype, F32, K)
    assert error(state, h0) <= tolerance(dtype, F32, K)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("batch,hk,h,K,V", [(1, 1, 1, 1, 1), (3, 2, 4, 20, 36), (2, 3, 3, 64, 65), (5, 1, 4, 128, 128),
                                            (70, 4, 16, 128, 64), (2, 1, 2, 256, 100)])
def test_update(dtype, batch, hk, h, K, V):
    t, r, _ = make(dtype, [1] * batch, False, hk, h, K, V, seed=batch)
    y0, h0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, r["h0"])
    state = t["h0"].clone()
    y = ssm.ssm_delta_update(state, *(t[n][:, 0] for n in ARGS))
    assert error(y, y0[:, 0]) <= tolerance(F32, dtype, 1) and error(state, h0) <= tolerance(F32, F32, 1)


def test_update_slots():
    """States in a pool; skipped rows leave every state alone and answer zero."""
    batch, hk, h, K, V = 6, 2, 4, 64, 48
    t, r, _ = make(BF16, [1] * batch, False, hk, h, K, V, seed=1)
    pool = torch.randn(9, h, K, V, device="cuda")
    at = [7, -1, 0, 9, 3, 1 << 30]
    before = pool.clone()
    y = ssm.ssm_delta_update(pool, *(t[n][:, 0] for n in ARGS),
                             slots=torch.tensor(at, dtype=torch.int32, device="cuda"), out_dtype=F32)
    live = [b for b, s in enumerate(at) if 0 <= s < 9]
    h0 = np.stack([before[at[b] if b in live else 0].double().cpu().numpy() for b in range(batch)])
    y0, h1 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, h0)
    for b in range(batch):
        if b in live:
            assert error(y[b], y0[b, 0]) <= 2e-5 and error(pool[at[b]], h1[b]) <= 2e-5
        else:
            assert not y[b].any()
    rest = [s for s in range(9) if s not in at]
    assert torch.equal(pool[rest], before[rest])


def test_update_far_slot():
    """A state behind 2^31 elements of the pool."""
    h, K, V = 16, 128, 128
    slots = (1 << 31) // (h * K * V) + 3
    pool = torch.empty(slots, h, K, V, device="cuda")
    t, r, _ = make(BF16, [1], False, h, h, K, V)
    pool[-1].copy_(t["h0"][0])
    y = ssm.ssm_delta_update(pool, *(t[n][:, 0] for n in ARGS),
                             slots=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"), out_dtype=F32)
    y0, h0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, r["h0"])
    assert error(y, y0[:, 0]) <= 2e-5 and error(pool[-1:], h0) <= 2e-5


def test_far_offsets():
    """Steps whose elements lie behind 2^31 of the tensors (a wide batch stride)."""
    L, h, K, V = 70, 2, 64, 64
    t, r, _ = make(BF16, [L, L], False, h, h, K, V, seed=8)
    far = (1 << 31) + 64
    kw, args = {}, []
    for n in ("q", "k", "v"):
        buf = torch.empty(far + L * h * 64, dtype=BF16, device="cuda")
        x = buf.as_strided((2, L, h, 64), (far, h * 64, 64, 1))
        x.copy_(t[n])
        args.append(x)
    out = torch.empty(far + L * h * V, dtype=BF16, device="cuda").as_strided((2, L, h, V), (far, h * V, V, 1))
    y, hL = ssm.ssm_delta_fwd(*args, t["g"], t["beta"], h0=t["h0"], y=out)
    y0, h0 = delta_batch(*(r[n] for n in ARGS), K ** -0.5, None, r["h0"])
    assert error(y, y0) <= tolerance(BF16, BF16, K) and error(hL, h0) <= tolerance(BF16, F32, K)


def test_clamped_bounds():
    """Bounds outside the tensors are clamped; covered steps are right, others are not written."""
    t, r, _ = make(F32, [100], False, 1, 2, 32, 16, seed=4)
    cu = torch.tensor([-7, 40, 90], dtype=torch.int32, device="cuda")
    y = torch.full((1, 100, 2, 16), 7.0, device="cuda")
    _, hL = ssm.ssm_delta_fwd(*(t[n] for n in ARGS), cu_seqlens=cu, y=y)
    y0, h0 = delta_batch(*(r[n][:, :90] for n in ARGS), 32 ** -0.5, [40, 50])
    assert error(y[:, :90], y0) <= 2e-5 and error(hL, h0) <= 2e-5
    assert (y[:, 90:] == 7.0).all()


def test_nonfinite_stays_in_its_sequence_and_head():
    lens = [70, 5, 100]
    t, _, cu = make(BF16, lens, True, 2, 4, 64, 64, seed=6)
    args = [t[n] for n in ARGS]
    y0, h0 = ssm.ssm_delta_fwd(*args, h0=t["h0"], cu_seqlens=cu)
    d0 = ssm.ssm_delta_bwd(*args, t["dy"], h0=t["h0"], dhL=t["dhL"], cu_seqlens=cu)
    t["v"][0, 71, 1] = float("nan")
    t["v"][0, 80, 3, 2] = float("inf")
    y1, h1 = ssm.ssm_delta_fwd(*args, h0=t["h0"], cu_seqlens=cu)
    d1 = ssm.ssm_delta_bwd(*args, t["dy"], h0=t["h0"], dhL=t["dhL"], cu_seqlens=cu)
    same = torch.ones(175, 4, dtype=torch.bool, device="cuda")
    same[70:75, 1] = False
    same[75:, 3] = False
    assert torch.equal(y1[0][same], y0[0][same])
    assert y1[0, 71, 1].isnan().all() and not y1[0, 80, 3, 2].isfinite()
    keep = torch.ones(3, 4, dtype=torch.bool)
    keep[1, 1] = keep[2, 3] = False
    assert torch.equal(h1[keep], h0[keep])
    for n in ("dv", "dg", "dbeta"):
        assert torch.equal(d1[n][0][same], d0[n][0][same]), n


def test_stream_and_graph():
    """On another stream than the inputs', and captured: every replay gives the eager bits."""
    lens = [130, 0, 65, 1]
    t, _, cu = make(BF16, lens, True, 2, 4, 64, 64, seed=9)
    args = [t[n] for n in ARGS]
    kw = dict(h0=t["h0"], cu_seqlens=cu)
    state = t["h0"].clone()
    one = [x[0, :4] for x in args]

    def step():
        ws = ssm.ssm_delta_bwd_workspace(t["q"], t["v"], cu_seqlens=cu)
        y, hL = ssm.ssm_delta_fwd(*args, checkpoints=ws, **kw)
        d = ssm.ssm_delta_bwd(*args, t["dy"], dhL=t["dhL"], workspace=ws, checkpoints_in_workspace=True, **kw)
        u = ssm.ssm_delta_update(state, *one)
        return [y, hL, u, *d.values()]

    ref = [x.clone() for x in step()]
    state.copy_(t["h0"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, hL = ssm.ssm_delta_fwd(*args, stream=side, **kw)
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
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, ref):
            assert torch.equal(got, want)
        torch.randn(64, 64, device="cuda").sum().item()


def test_layer_in_full():
    """The 5120-channel layer's shape against the recurrence, two of its 40 heads."""
    t, r, _ = make(BF16, [2048], False, 40, 40, 128, 128, seed=2, state=False)
    args = [t[n] for n in ARGS]
    y, hL = ssm.ssm_delta_fwd(*args, out_dtype=F32)
    d = ssm.ssm_delta_bwd(*args, t["dy"])
    for h in (0, 39):
        one = {n: x[:, :, h:h + 1] if x is not None else None for n, x in r.items()}
        y0, h0, d0 = delta_batch(*(one[n] for n in ARGS), 128 ** -0.5, None, None, one["dy"])
        assert error(y[:, :, h:h + 1], y0) <= tolerance(BF16, F32, 128)
        assert error(hL[:, h:h + 1], h0) <= tolerance(BF16, F32, 128)
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            out = BF16 if n in ("dq", "dk", "dv") else F32
            assert error(d[n][:, :, h:h + 1], d0[n]) <= tolerance(BF16, out, 128, n), n
