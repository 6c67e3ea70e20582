"""The built code of the wide block-scaled kernels: their instruction streams are laid out by hand, with vector
instructions in inline assembly, for which the compiler inserts no waits.  So that no build (another compiler, an edit
nearby) reads a matrix instruction's result too early, every path through the code is followed here: a 16 x 16 x 128
MFMA of e4m3 leaves the unit eight passes after it was issued, and eleven wait states have to lie between it and
a vector, LDS or memory instruction that reads or overwrites its result.  Each instruction is a state at least, s_nop n is n + 1,
and a second MFMA eight, since it is issued when the first has passed."""
import os
import re
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dense_gemm_design_amd", "libdgemm.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
STATES, PASSES = 11, 8
KERNEL = re.compile(r"^[0-9a-f]+ <(_ZN2dg\S*wide_block_kernel\S*)>:", re.M)


def code_objects():
    """The gfx950 code objects in the library that hold the kernels."""
    data, at, magic = open(LIB, "rb").read(), 0, b"__CLANG_OFFLOAD_BUNDLE__"
    while (at := data.find(magic, at)) >= 0:
        (count,) = struct.unpack_from("<Q", data, at + 24)
        entry = at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            image = data[at + offset:at + offset + size]
            if target.endswith(b"gfx950") and b"wide_block_kernel" in image:
                yield image
        at += len(magic)


def registers(text):
    """v and a registers that an operand list names; an a register is numbered from 1000."""
    found = set()
    for kind, one, low, high in re.findall(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])", text):
        base = 1000 if kind == "a" else 0
        found |= {base + int(one)} if one else set(range(base + int(low), base + int(high) + 1))
    return found


class Instruction:
    def __init__(self, address, op, operands):
        self.address, self.op = address, op
        self.mfma = op.startswith("v_mfma")
        parts = operands.split(", ", 1)
        first, rest = registers(parts[0]), registers(parts[1] if len(parts) > 1 else "")
        vector = op.startswith("v_")
        loads = op.startswith(("ds_read", "buffer_load", "global_load")) and not operands.endswith(" lds")
        self.writes = first if vector or loads else set()
        self.touches = set() if self.mfma else first | rest
        self.states = int(operands) + 1 if op == "s_nop" else PASSES if self.mfma else 1
        self.target = None


def kernels(tmp_path):
    for k, image in enumerate(code_objects()):
        path = tmp_path / f"{k}.co"
        path.write_bytes(image)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True,
                              text=True, check=True).stdout
        for m in KERNEL.finditer(text):
            start = int(m[0].split()[0], 16)
            body = text[m.end():]
            body = body[:body.find("\n\n")] if "\n\n" in body else body
            code = []
            for line in body.splitlines():
                hit = re.match(r"\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):", line)
                if not hit:
                    continue
                code.append(Instruction(int(hit[3], 16), hit[1], hit[2]))
                to = re.search(r"<\S+?\+0x([0-9a-f]+)>", line)
                if hit[1].startswith(("s_branch", "s_cbranch")):
                    code[-1].target = start + int(to[1], 16) if to else start
            yield m[1], code


def early_touches(code):
    """Instructions that touch an MFMA's result too early on some path, as (address, operation)."""
    index = {i.address: n for n, i in enumerate(code)}
    pending = [None] * len(code)     # at entry: register -> the fewest states since its MFMA
    bad, work = set(), [(0, {})]
    while work:
        n, state = work.pop()
        while n < len(code):
            known = pending[n]
            if known is not None:
                if all(r in known and known[r] <= s for r, s in state.items()):
                    break
                state = {r: min(state.get(r, STATES), known.get(r, STATES)) for r in {*state, *known}}
            pending[n] = dict(state)
            i = code[n]
            if state and i.touches & state.keys():
                bad.add((i.address, i.op))
            state = {r: s + i.states for r, s in state.items()
                     if s + i.states < STATES and r not in i.writes}
            if i.mfma:
                state.update((r, 0) for r in i.writes)
            if i.op.startswith("s_endpgm"):
                break
            if i.target is not None:
                if i.op.startswith("s_branch"):
                    n = index[i.target]
                    continue
                work.append((index[i.target], dict(state)))
            n += 1
    return sorted(bad)


@pytest.mark.skipif(not os.path.exists(LIB) or not shutil.which(OBJDUMP), reason="no built library or no objdump")
def test_no_result_is_touched_before_it_has_left_the_matrix_unit(tmp_path):
    seen = 0
    for name, code in kernels(tmp_path):
        mfmas = sum(i.mfma for i in code)
        assert mfmas >= 96, (name, mfmas)
        assert early_touches(code) == [], name
        seen += 1
    assert seen == 3


def instructions(text):
    return [Instruction(4 * n, *(line.split(" ", 1) if " " in line else (line, "")))
            for n, line in enumerate(text)]


def test_the_check_sees_early_touches():
    """On streams written here: age by MFMAs, by waits, along a branch, and what is no result."""
    mfma = "v_mfma_scale_f32_16x16x128_f8f6f4 v[{}:{}], a[0:7], a[8:15], 0, v90, v90"
    a, b, c = (mfma.format(k, k + 3) for k in (0, 4, 8))
    add = "v_fmac_f32 v50, v1, v60"
    for text, early in (([a, b, c, add], 0), ([a, b, add], 1), ([a, add], 1),
                        ([a, "s_nop 7", "s_nop 7", add], 0), ([a, "s_nop 9", add], 1),
                        ([a, "s_nop 10", add], 0), ([a, b, "s_nop 2", add], 0), ([a, b, "s_nop 1", add], 1),
                        ([a, "v_mov_b32_e32 v50, v4"], 0), ([a, "v_mov_b32_e32 v1, v50"], 1),
                        ([a, "buffer_store_dwordx4 v[0:3], v70, s[4:7], 0 offen"], 1),
                        ([a, "ds_read_b128 v[2:5], v70"], 1)):
        assert len(early_touches(instructions(text))) == early, text
    # a loop whose end leaves results to its beginning
    loop = instructions([add, b, c, a, "s_cbranch_scc1 65535", "s_endpgm "])
    loop[4].target = 0
    assert len(early_touches(loop)) == 1
    loop = instructions(["v_mov_b32_e32 v70, v71", b, c, a, b, c, "s_cbranch_scc1 65535", add, "s_endpgm "])
    loop[6].target = 0
    assert early_touches(loop) == []
