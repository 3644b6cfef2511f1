"""Gradients of the head scan where a workgroup goes through many heads of a
chunk, all of them live: the heads' decays, sums and rows take turns in the same
places from head to head, and dB and dC add up over them; and what the records
that no sequence has leave alone.  Tolerances are those of test_gpu_heads (derived
there)."""
import numpy as np
import pytest
import torch

import selective_state_space_64_amd as ssm
from test_gpu_delta import error
from test_gpu_heads import BF16, F32, call, call_bwd, make, reference, tolerance

pytestmark = pytest.mark.gpu


def heads_a_part(lens, packed, g, h):
    """Heads that a workgroup of the gradients sums: a group's, in as many parts
    as 256 workgroups take (heads_parts)."""
    chunks = -(-sum(lens) // 64) + len(lens) if packed else len(lens) * -(-lens[0] // 64)
    rep, parts = h // g, -(-256 // (chunks * g))
    return -(-rep // min(parts, rep))


# many short sequences, so that whole groups stay together, beside some of several chunks
LONG = [65, 130, 64, 3]
ONE = dict(lens=[1] * 246 + LONG, packed=True, g=1, h=10)
TWO = dict(lens=[1, 2] * 60 + LONG, packed=True, g=2, h=18)
THREE = dict(lens=[1] * 90 + LONG, packed=True, g=1, h=9)  # three parts of three heads
ROWS = dict(lens=[67] * 64, packed=False, g=2, h=18)
#       inputs, gradients, N, P, sequences, heads a part
CASES = [
    (F32, F32, 256, 32, ONE, 10),    # one block of columns a head, two places for the decays
    (F32, F32, 256, 32, THREE, 3),
    (F32, F32, 200, 24, TWO, 9),
    (F32, F32, 217, 7, ONE, 10),
    (BF16, F32, 256, 32, ONE, 10),
    (F32, BF16, 256, 16, THREE, 3),
    (F32, F32, 256, 72, TWO, 9),
    (F32, F32, 128, 32, ONE, 10),
    (F32, F32, 100, 130, TWO, 9),
    (F32, F32, 64, 40, TWO, 9),
    (F32, F32, 16, 7, ROWS, 9),
    (BF16, BF16, 256, 32, ONE, 10),
    (BF16, BF16, 200, 72, TWO, 9),
    (BF16, BF16, 128, 64, TWO, 9),
    (BF16, BF16, 100, 130, THREE, 3),
    (BF16, BF16, 64, 7, ONE, 10),
    (BF16, BF16, 16, 32, ROWS, 9),
    (BF16, F32, 64, 40, TWO, 9),
]


@pytest.mark.parametrize("dtype,grad,N,P,seqs,each", CASES,
                         ids=["%s-%s-N%dP%d-%dseqs%dheads" % (str(c[0])[6:], str(c[1])[6:], c[2], c[3], len(c[4]["lens"]),
                                                              c[5]) for c in CASES])
def test_heads_of_a_part(dtype, grad, N, P, seqs, each):
    lens, packed, g, h = (seqs[n] for n in ("lens", "packed", "g", "h"))
    assert heads_a_part(lens, packed, g, h) == each
    t, r, cu = make(dtype, lens, packed, g, h, N, P, seed=N + P)
    t["dy"], r["dy"] = t["dy"].to(grad), t["dy"].to(grad).double().cpu().numpy()
    _, _, d0 = reference(r, lens if packed else None, grads=True)
    ws = ssm.ssm_head_scan_bwd_workspace(t["x"], t["B"], cu_seqlens=cu)
    call(t, cu, checkpoints=ws)
    d = call_bwd(t, cu, workspace=ws, checkpoints_in_workspace=True)
    e = call_bwd(t, cu)
    for n in d0:
        assert torch.equal(d[n], e[n]), n
        assert error(d[n], d0[n]) <= tolerance(dtype, d[n].dtype, n), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,cu,g", [(300, [130, 170, 240], 1), (300, [130, 170, 240], 2), (200, [64, 64, 199], 1),
                                    (1500, [700, 1450], 1), (1500, [250, 1400, 1400, 1499], 2)])
def test_steps_in_front_of_the_first_sequence(L, cu, g, dtype):
    """Bounds that begin behind the first chunk: the steps in front keep what the
    outputs held, and nothing of them is in the sums."""
    h, N, P = 2, 32, 16
    t, r, _ = make(dtype, [L], False, g, h, N, P, seed=L, state=False)
    bounds = torch.tensor(cu, dtype=torch.int32, device="cuda")
    held = lambda *shape: torch.full((1, L, *shape), 7.0, device="cuda", dtype=dtype)  # noqa: E731
    out = {"dx": held(h, P), "ddt": held(h), "dBm": held(g, N), "dCm": held(g, N)}
    y, hL = call(t, bounds, y=held(h, P))
    d = call_bwd(t, bounds, **out)
    inside = {n: v[:, cu[0]:cu[-1]] if n in ("x", "dt", "B", "C", "dy") else v for n, v in r.items()}
    inside["dhL"] = np.zeros((len(cu) - 1, h, N, P))
    y0, h0, d0 = reference(inside, list(np.diff(cu)), grads=True)
    assert error(hL, h0) <= tolerance(dtype, F32, "hL")
    for n, got, want in [("y", y, y0)] + [(n, d[n], d0[n]) for n in d0]:
        if n == "y" or n in out:
            assert (got[:, :cu[0]] == 7.0).all() and (got[:, cu[-1]:] == 7.0).all(), n
            got = got[:, cu[0]:cu[-1]]
        assert error(got, want) <= tolerance(dtype, got.dtype, n), n
