"""Sizes whose chunks no grid of the head scan's gradients can number (CPU: the
calls fail validation, device pointers are never followed)."""
import pytest

import selective_state_space_64_amd as ssm
from test_heads_rms_abi import P, SHAPE, scan

LONGEST = (1 << 28) - 4096
SMALL = dict(g=1, heads=1, N=1, P=1, wsb=1 << 62, h0=None, hL=None, cu=None)
MANY = [dict(batch=3, L=LONGEST), dict(batch=65535, L=64 * 129), dict(batch=1 << 14, L=64 * 512)]


@pytest.mark.parametrize("size", MANY, ids=str)
def test_more_chunks_than_a_grid_has(size):
    args = (size["batch"], size["L"], 1, 1, 1, 1, 0)
    assert ssm.lib().ssm_head_scan_bwd_workspace_bytes(*args) == 0
    assert scan("bwd", **SMALL, **size) == SHAPE and scan("bwd", flags=2, **SMALL, **size) == SHAPE
    assert scan("fwd", flags=2, **SMALL, **size) == SHAPE
    # the forward alone numbers sequences, not chunks: it goes on to the next check
    assert scan("fwd", **{**SMALL, **size, "y": P["x"]}) != SHAPE


def test_the_largest_sizes_have_a_workspace():
    f = ssm.lib().ssm_head_scan_bwd_workspace_bytes
    for batch, L in ((1, LONGEST), (65535, 64 * 127), ((1 << 14) - 1, 64 * 512)):
        assert f(batch, L, 1, 1, 1, 1, 0) >= 2 * 4096 * batch * (L // 64)
