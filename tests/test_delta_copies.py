"""The copies from memory to LDS in the code that the compiler emits (CPU: a
small kernel is compiled to assembly, nothing runs).  gfx950 wants one wait
state between a write of m0 and a copy that takes its LDS place from it, and
five between a vector instruction's write of an SGPR and a buffer access that
reads it; the copies are inline assembly, into which the compiler puts none."""
import os
import re
import subprocess

import pytest

from selective_state_space_64_amd._build import CSRC, HIPFLAGS, INCLUDE, hipcc

KERNEL = """
#include "delta_mfma.hpp"
using namespace ssm;
__global__ void k(const float *p, const int *rows, float *out)
{
    __shared__ __align__(16) float lds[1024];
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds_offset(lds));
    // a size that a vector instruction hands to the descriptor
    const sgpr4 buf = copy_buffer(p, __builtin_amdgcn_readfirstlane(rows[threadIdx.x]));
    copy_to_lds(buf, threadIdx.x * 16, to);
    copy_to_lds(buf, threadIdx.x * 16 + 1024, to + 1024);
    copy_linear<2048, 1>(p, to + 2048, 0);
    wait_loads<0>();
    __syncthreads();
    out[threadIdx.x] = lds[threadIdx.x * 16];
}
"""


def sgprs(operand):
    m = re.match(r"s\[(\d+):(\d+)\]|s(\d+)", operand.strip())
    if not m:
        return set()
    return {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def copies(text):
    """(wait states since m0 was written, since a vector instruction wrote the
    descriptor) of every copy, None where nothing of the kind stands before it."""
    code = [l.split(";")[0].strip() for l in text.splitlines() if l.startswith("\t") and not l.startswith("\t.")]
    code = [l for l in code if l]
    found = []
    for i, line in enumerate(code):
        if not (line.startswith("buffer_load") and re.search(r"\blds\b", line)):
            continue
        descriptor = sgprs(line.split(",")[1])
        assert len(descriptor) == 4, line
        waits, m0, vector = 0, None, None
        for before in reversed(code[:i]):
            op, _, args = before.partition(" ")
            target = args.split(",")[0].strip()
            if m0 is None and target == "m0":
                m0 = waits
            if vector is None and op.startswith("v_") and sgprs(target) & descriptor:
                vector = waits
            waits += int(args, 0) + 1 if op == "s_nop" else 1
        found.append((m0, vector))
    return found


@pytest.mark.skipif(not os.path.exists(hipcc()), reason="hipcc not found")
def test_wait_states_before_copies(tmp_path):
    src, asm = tmp_path / "copies.hip", tmp_path / "copies.s"
    src.write_text(KERNEL)
    flags = [f for f in HIPFLAGS if f != "-fPIC"]
    r = subprocess.run([hipcc(), *flags, "-I", INCLUDE, "-I", CSRC, "--cuda-device-only", "-S", str(src), "-o", str(asm)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "inline-asm" not in r.stderr, r.stderr  # warnings of the asm block
    found = copies(asm.read_text())
    assert len(found) == 4
    assert all(m0 is not None and m0 >= 1 for m0, _ in found), found
    assert any(vector is not None for _, vector in found), "the descriptor comes from a vector instruction"
    assert all(vector is None or vector >= 5 for _, vector in found), found
