"""The machine code of the built library, as far as its matrix instructions and
its copies to LDS are concerned: the waits that gfx950 does not make by itself
and that have to stand in the code."""
import os
import re
import shutil
import subprocess

ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
OBJDUMP = os.path.join(ROCM, "llvm", "bin", "llvm-objdump")


def kernels(library, workdir):
    """{kernel: [(label or None, instruction, operands)]} of a library built here."""
    local = os.path.join(workdir, "library.so")
    shutil.copyfile(library, local)
    subprocess.run([OBJDUMP, "--offloading", local], cwd=workdir, check=True, capture_output=True)
    found = {}
    for name in sorted(os.listdir(workdir)):
        if name.startswith("library.so.") and name.endswith("gfx950"):
            text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", "--symbolize-operands", name],
                                  cwd=workdir, check=True, capture_output=True, text=True).stdout
            code, label = None, None
            for line in text.splitlines():
                m = re.match(r"^<(\w+)>:", line)
                if m and re.fullmatch(r"L\d+", m[1]):
                    label = m[1]
                elif m:
                    code, label = found.setdefault(m[1], []), None
                elif line.startswith("\t") and code is not None:
                    op, _, args = line.split("//")[0].strip().partition(" ")
                    code.append((label, op, [a.strip() for a in args.split(",")]))
                    label = None
    return found


def registers(operand):
    """The registers that an operand names: {"v3", "v4"}."""
    m = re.match(r"-?\|?([vas])(?:\[(\d+):(\d+)\]|(\d+)\b)", operand)
    if not m:
        return set()
    return {m[1] + str(i) for i in (range(int(m[2]), int(m[3]) + 1) if m[2] else [int(m[4])])}


def waits(op, args):
    return int(args[0], 0) + 1 if op == "s_nop" else 1


def copy_waits(code):
    """Of every copy from memory to LDS: (wait states since m0 was written, since a
    vector instruction wrote an SGPR of its descriptor; None: not in the last 64)."""
    out = []
    for i, (_, op, args) in enumerate(code):
        if op.startswith("buffer_load") and args[-1].endswith(" lds"):
            descriptor, n, m0, vector = registers(args[1]), 0, None, None
            assert len(descriptor) == 4, args
            for _, before, b in reversed(code[max(0, i - 64):i]):
                if m0 is None and b[0] == "m0":
                    m0 = n
                if vector is None and before.startswith("v_") and registers(b[0]) & descriptor:
                    vector = n
                n += waits(before, b)
            out.append((m0, vector))
    return out


# wait states until a result may be read, or taken as the left or right operand of
# another matrix instruction, and until its registers may be written by another
# instruction: passes + 4 and + 3 for bf16 (4 passes), passes + 2 for fp32 (8)
MATRIX_WAITS = {"v_mfma_f32_16x16x32_bf16": (8, 7), "v_mfma_f32_16x16x4_f32": (10, 10)}


def early_uses(code):
    """(instruction, index, wait states, what uses it) of every matrix result that is read
    or overwritten too early on some path through the code."""
    at = {label: i for i, (label, _, _) in enumerate(code) if label}
    uses = []  # (read early, taken as the sum to go on with, written)
    for _, op, args in code:
        if op.startswith("s_"):
            uses.append((set(), set(), set()))
            continue
        stores = op.startswith(("ds_write", "scratch_store", "global_store", "buffer_store")) or args[-1].endswith(" lds")
        own = set() if stores or op.startswith("v_cmp") else registers(args[0])
        matrix = op.startswith("v_mfma")
        read = set().union(*[registers(a) for a in (args[1:3] if matrix else args if stores else args[1:])], set())
        if op.startswith(("v_fmac", "v_dot2c")):
            read |= own
        uses.append((read, registers(args[3]) if matrix else set(), own))
    found = []
    for i, (_, op, args) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        (need, free), result, seen, paths = MATRIX_WAITS[op], registers(args[0]), {}, [(i + 1, 0)]
        while paths:
            j, n = paths.pop()
            while n < need and j < len(code) and seen.get(j, need) > n:
                seen[j] = n
                _, use, b = code[j]
                read, going_on, own = uses[j]
                if read & result or (going_on & result and going_on != result):
                    found.append((op, i, n, use))
                    break
                if own & result and not use.startswith("v_mfma") and n < free:
                    found.append((op, i, n, use))
                if use == "s_endpgm" or own & result:
                    break
                n += waits(use, b)
                if use == "s_branch":
                    j = at[b[0]]
                    continue
                if use.startswith("s_cbranch"):
                    paths.append((at[b[0]], n))
                j += 1
    return found
