"""The built code of the int8 product's kernels whose instruction streams are laid out by hand: their matrix
instructions are inline assembly, for which the compiler inserts no waits.  Every path is followed, as for the
block-scaled kernels; a 16 x 16 x 64 MFMA of int8 passes in four states, and eight have to lie between it and what
reads or overwrites its result, for which the check's eleven stand.  What a vector instruction wrote is two states
old before an MFMA reads it."""
import os
import re
import shutil
import struct
import subprocess

import pytest

import test_wide_kernel_code as W

KERNEL = re.compile(r"^[0-9a-f]+ <(_ZN2dg\S*(?:wide_int8_kernel|pipe_kernel)\S*)>:", re.M)
PASSES = 4


def code_objects():
    data, at, magic = open(W.LIB, "rb").read(), 0, b"__CLANG_OFFLOAD_BUNDLE__"
    while (at := data.find(magic, at)) >= 0:
        (count,) = struct.unpack_from("<Q", data, at + 24)
        entry = at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            image = data[at + offset:at + offset + size]
            if target.endswith(b"gfx950") and (b"wide_int8_kernel" in image or b"pipe_kernel" in image):
                yield image
        at += len(magic)


def kernels(tmp_path):
    for k, image in enumerate(code_objects()):
        path = tmp_path / f"{k}.co"
        path.write_bytes(image)
        text = subprocess.run([W.OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True,
                              text=True, check=True).stdout
        for m in KERNEL.finditer(text):
            start, body, code = int(m[0].split()[0], 16), text[m.end():], []
            for line in body.split("\n\n")[0].splitlines():
                hit = re.match(r"\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):", line)
                if not hit:
                    continue
                i = W.Instruction(int(hit[3], 16), hit[1], hit[2])
                i.states = PASSES if i.mfma else i.states
                i.reads = W.registers(hit[2].split(", ", 1)[1]) if i.mfma else set()
                to = re.search(r"<\S+?\+0x([0-9a-f]+)>", line)
                if i.op.startswith(("s_branch", "s_cbranch")):
                    i.target = start + int(to[1], 16) if to else start
                code.append(i)
            yield m[1], code


def early_operands(code):
    """MFMAs that read what a vector instruction wrote less than two states ago."""
    bad = []
    for n, i in enumerate(code):
        states, k = 0, n - 1
        while i.mfma and states < 2 and k >= 0:
            if code[k].op.startswith("v_") and not code[k].mfma and code[k].writes & i.reads:
                bad.append((i.address, code[k].op))
            states, k = states + code[k].states, k - 1
    return bad


@pytest.mark.skipif(not os.path.exists(W.LIB) or not shutil.which(W.OBJDUMP),
                    reason="no built library or no objdump")
def test_no_result_is_touched_before_it_has_left_the_matrix_unit(tmp_path):
    seen = 0
    for name, code in kernels(tmp_path):
        mfmas = [i for i in code if i.mfma]
        assert len(mfmas) >= 32, (name, len(mfmas))
        # the sums stay where they are: none but an MFMA's own is written by one
        assert all(i.op == "v_mfma_i32_16x16x64_i8" and min(i.writes) >= 1000 for i in mfmas), name
        assert W.early_touches(code) == [], name
        assert early_operands(code) == [], name
        seen += 1
    assert seen == 16   # seven tiles, rows on lines of memory and not, and 256 x 256 to two types
