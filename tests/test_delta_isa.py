"""The waits in the built library's code (CPU: it is disassembled, nothing runs).
The hardware does not wait for a matrix instruction's result by itself, nor a
copy to LDS for m0: the states stand in the code, put there by the compiler or
by hand, and this looks at every kernel for those that it needs."""
import os

import pytest

import isa
from selective_state_space_64_amd._build import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(isa.OBJDUMP), reason="llvm-objdump not found")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    return isa.kernels(LIB, str(tmp_path_factory.mktemp("isa")))


def test_matrix_results_are_waited_for(kernels):
    early = {name: isa.early_uses(code) for name, code in kernels.items()}
    assert sum(any(op in isa.MATRIX_WAITS for _, op, _ in code) for code in kernels.values()) > 100
    assert not {name: found for name, found in early.items() if found}


def test_copies_to_lds_wait(kernels):
    found = {name: isa.copy_waits(code) for name, code in kernels.items()}
    assert sum(map(len, found.values())) > 1000
    late = {name: [c for c in copies if c[0] is None or c[0] < 1 or (c[1] is not None and c[1] < 5)]
            for name, copies in found.items()}
    assert not {name: bad for name, bad in late.items() if bad}


L = "L1"


@pytest.mark.parametrize("code,early", [
    # read behind eight wait states, behind seven; the sum taken on at once, in other registers
    ([(None, "s_nop", ["7"]), (None, "v_add_f32_e32", ["v9", "v8", "v3"])], 0),
    ([(None, "s_nop", ["6"]), (None, "v_add_f32_e32", ["v9", "v8", "v3"])], 1),
    ([(None, "v_mfma_f32_16x16x32_bf16", ["v[0:3]", "v[4:7]", "v[8:11]", "v[0:3]"]), (None, "s_endpgm", [""])], 0),
    ([(None, "v_mfma_f32_16x16x32_bf16", ["v[20:23]", "v[4:7]", "v[8:11]", "v[2:5]"]), (None, "s_endpgm", [""])], 1),
    ([(None, "v_mfma_f32_16x16x32_bf16", ["v[20:23]", "v[0:3]", "v[8:11]", "v[20:23]"]), (None, "s_endpgm", [""])], 1),
    # late on the way through, early behind the branch
    ([(None, "s_cbranch_scc1", [L]), (None, "s_nop", ["7"]), (L, "ds_write_b32", ["v9", "v0"])], 1),
    # overwritten
    ([(None, "s_nop", ["5"]), (None, "v_mov_b32_e32", ["v1", "0"])], 1),
    ([(None, "s_nop", ["6"]), (None, "v_mov_b32_e32", ["v1", "0"])], 0),
], ids=str)
def test_the_look_itself(code, early):
    first = (None, "v_mfma_f32_16x16x32_bf16", ["v[0:3]", "v[4:7]", "v[8:11]", "0"])
    assert len(isa.early_uses([first, *code])) == early
