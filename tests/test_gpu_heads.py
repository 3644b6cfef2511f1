"""The selective scan with one decay a head on the GPU (ssm_head_scan_fwd,
ssm_head_scan_bwd, ssm_head_scan_update) against the plain fp64 recurrence.

Error of a tensor: max |got - ref| / max(|ref|, rms(ref)).  Tolerances, from
the kernels' arithmetic:
  * fp32 products and sums: a value passes about 4 chained products of up to
    256 summands, 4 x sqrt(256) x 2^-24 = 4e-6 rms, 5 times that at the largest
    of ~1e5 elements: 2e-5.  It covers the states of bf16 inputs too, whose
    operands keep 24 bits (three bf16 terms).
  * two terms (what forms y, dx, dB and dC of bf16 inputs) leave at most 2^-17
    of an operand, one in each of 2 chained products, 5 times their rms
    2^-17/sqrt(3) x sqrt(2) at the largest element: 3e-5, doubled for the
    operands being larger than the result where terms cancel: 6e-5.
  * ddt and the sums dA and ddt_bias are differences of such terms over the
    steps behind each step: 4 times that.
  * a bf16 output adds half an ulp: half of torch.finfo(bfloat16).eps, 2^-8.
"""
import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from heads_reference import head_scan_batch
from test_gpu_delta import error

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
ARGS = ("x", "dt", "A", "B", "C")


def tolerance(dtype, out, name="y"):
    t = 2e-5 if dtype == F32 or name in ("hL", "dh0", "dDskip") else 6e-5
    t *= 4 if name in ("ddt", "dA", "ddt_bias") else 1
    return t + (torch.finfo(BF16).eps / 2 if out == BF16 else 0.0)


def make(dtype, lens, packed, g, h, N, P, seed=0, state=True, steps="mixed", extras=True):
    rng = np.random.default_rng(seed)
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    n = rng.standard_normal
    bias = {"mixed": rng.uniform(-5, 0, h), "small": np.full(h, -9.0), "large": np.full(h, 4.0)}[steps]
    f32 = lambda a: torch.tensor(a, dtype=F32)  # noqa: E731
    t = {"x": torch.tensor(n((*lead, h, P))).to(dtype), "dt": torch.tensor(n((*lead, h))).to(dtype),
         "A": f32(-rng.uniform(0.5, 16, h)), "B": torch.tensor(n((*lead, g, N))).to(dtype),
         "C": torch.tensor(n((*lead, g, N))).to(dtype), "D": f32(n(h)) if extras else None,
         "bias": f32(bias) if extras else None, "dy": torch.tensor(n((*lead, h, P))).to(dtype),
         "h0": f32(n((len(lens), h, N, P))) if state else None,
         "dhL": f32(n((len(lens), h, N, P))) if state else None}
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32) if packed else None
    ref = {m: None if x is None else x.double().numpy() for m, x in t.items()}
    dev = {m: None if x is None else x.cuda() for m, x in t.items()}
    return dev, ref, None if cu is None else cu.cuda()


def reference(r, lens=None, grads=False):
    more = (r["dy"], r["dhL"]) if grads else ()
    return head_scan_batch(*(r[n] for n in ARGS), r["D"], r["bias"], lens, r["h0"], *more)


def call(t, cu=None, **kw):
    return ssm.ssm_head_scan_fwd(*(t[n] for n in ARGS), Dskip=t["D"], dt_bias=t["bias"], h0=t["h0"], cu_seqlens=cu, **kw)


def call_bwd(t, cu=None, **kw):
    return ssm.ssm_head_scan_bwd(*(t[n] for n in ARGS), t["dy"], Dskip=t["D"], dt_bias=t["bias"], h0=t["h0"],
                                 dhL=t["dhL"], cu_seqlens=cu, **kw)


#       dtype lens packed g h N P options
CASES = [
    (F32, [1], False, 1, 1, 1, 1, {}),
    (F32, [17, 17], False, 2, 4, 32, 40, {}),
    (BF16, [17, 17], False, 2, 4, 32, 40, {}),
    (F32, [64], False, 1, 2, 16, 64, dict(state=False)),
    (BF16, [65], False, 1, 3, 64, 16, dict(state=False, extras=False)),
    (F32, [200], False, 3, 6, 100, 36, {}),
    (BF16, [130, 130], False, 1, 5, 128, 64, {}),
    (BF16, [129], False, 2, 4, 128, 72, dict(steps="large")),
    (F32, [150], False, 1, 2, 128, 96, dict(steps="small")),
    (BF16, [70], False, 1, 2, 256, 64, {}),
    (F32, [70], False, 2, 2, 256, 33, {}),
    (F32, [70], False, 1, 2, 256, 64, {}),
    (BF16, [90], False, 1, 2, 217, 7, {}),
    (BF16, [1, 0, 63, 64, 65, 128, 7], True, 1, 4, 64, 64, {}),
    (F32, [0, 5, 200, 0, 1], True, 2, 4, 33, 20, {}),
    (BF16, [0, 0, 3], True, 1, 1, 128, 64, dict(state=False)),
    (BF16, [1500], False, 1, 2, 32, 16, {}),            # cut into segments
    (F32, [1100, 1100], False, 1, 2, 16, 24, {}),
    (BF16, [700, 40, 0, 900, 300], True, 1, 2, 64, 64, {}),
    (BF16, [900, 900], False, 1, 2, 128, 64, dict(state=False)),
    (BF16, [100], False, 1, 70, 16, 16, {}),            # many heads share B and C
    (BF16, [100], False, 1, 2, 64, 200, {}),            # several column tiles
]


def name(c):
    return "%s-%s%s-g%dh%d-N%dP%d%s" % (str(c[0])[6:], "p" if c[2] else "", "x".join(map(str, c[1])), *c[3:7],
                                        "".join("-%s" % k for k in c[7]))


@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward(case):
    dtype, lens, packed, g, h, N, P, opt = case
    t, r, cu = make(dtype, lens, packed, g, h, N, P, **opt)
    y0, h0 = reference(r, lens if packed else None)
    y, hL = call(t, cu)
    assert y.dtype == dtype
    assert error(y, y0) <= tolerance(dtype, dtype) and error(hL, h0) <= tolerance(dtype, F32, "hL")
    y, none = call(t, cu, out_dtype=F32, return_final_state=False)
    assert none is None and error(y, y0) <= tolerance(dtype, F32)


@pytest.mark.parametrize("case", CASES, ids=name)
def test_gradients(case):
    dtype, lens, packed, g, h, N, P, opt = case
    t, r, cu = make(dtype, lens, packed, g, h, N, P, **opt)
    y0, h0, d0 = reference(r, lens if packed else None, grads=True)
    ws = ssm.ssm_head_scan_bwd_workspace(t["x"], t["B"], cu_seqlens=cu)
    y, hL = call(t, cu)
    yc, hc = call(t, cu, checkpoints=ws)
    assert torch.equal(yc, y) and torch.equal(hc, hL)
    d = call_bwd(t, cu, workspace=ws, checkpoints_in_workspace=True)
    e = call_bwd(t, cu)
    for n in d0:
        if d[n] is None:
            assert not opt.get("extras", True) and n in ("dDskip", "ddt_bias")
            continue
        assert torch.equal(d[n], e[n]), n
        assert error(d[n], d0[n]) <= tolerance(dtype, d[n].dtype, n), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("batch,g,h,N,P", [(1, 1, 1, 1, 1), (3, 2, 4, 20, 36), (2, 3, 3, 64, 65), (5, 1, 4, 128, 64),
                                           (70, 4, 16, 128, 64), (2, 1, 2, 256, 100), (1, 1, 3, 217, 7)])
def test_update(dtype, batch, g, h, N, P):
    t, r, _ = make(dtype, [1] * batch, False, g, h, N, P, seed=batch)
    y0, h0 = reference(r)
    state = t["h0"].clone()
    y = ssm.ssm_head_scan_update(state, *(t[n] if n == "A" else t[n][:, 0] for n in ARGS), Dskip=t["D"],
                                 dt_bias=t["bias"])
    assert error(y, y0[:, 0]) <= tolerance(F32, dtype) and error(state, h0) <= tolerance(F32, F32)


@pytest.mark.parametrize("dtype,N,P", [(F32, 64, 40), (BF16, 128, 64)])
def test_resume_and_decode(dtype, N, P):
    """A sequence in pieces, its state handed on (in place), and its last steps one by one."""
    L, cuts = 200, [0, 1, 70, 190]
    t, r, _ = make(dtype, [L, L], False, 2, 4, N, P, seed=3)
    y0, h0 = reference(r)
    state, ys = t["h0"].clone(), []
    kw = dict(Dskip=t["D"], dt_bias=t["bias"], out_dtype=F32)
    for a, b in zip(cuts, cuts[1:]):
        y, hL = ssm.ssm_head_scan_fwd(*(t[n] if n == "A" else t[n][:, a:b] for n in ARGS), h0=state, hL=state, **kw)
        assert hL is state
        ys.append(y)
    for i in range(cuts[-1], L):
        ys.append(ssm.ssm_head_scan_update(state, *(t[n] if n == "A" else t[n][:, i] for n in ARGS), **kw)[:, None])
    assert error(torch.cat(ys, 1), y0) <= tolerance(dtype, F32)
    assert error(state, h0) <= tolerance(dtype, F32, "hL")
