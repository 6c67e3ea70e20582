"""The built code of the int8 product's kernels whose instruction streams are laid out by hand: what a vector
instruction wrote is two wait states old before an MFMA, which is inline assembly there, reads it.  Paths are followed
from instruction to instruction, through branches and round loops; streams written here show what the check sees."""
import os
import shutil

import pytest

import test_int8_kernel_code as K
import test_wide_kernel_code as W

STATES = 2
BOTH = ("v_swap_", "v_permlane16_swap", "v_permlane32_swap")   # these write their second operand too


def written(i):
    """The registers that a vector instruction other than an MFMA writes."""
    if not i.op.startswith("v_") or i.mfma:
        return set()
    return i.writes | (i.touches if i.op.startswith(BOTH) else set())


def early_operands(code):
    """MFMAs that read what a vector instruction wrote too few states ago on some path, as (address, operation)."""
    index = {i.address: n for n, i in enumerate(code)}
    seen = [None] * len(code)        # at entry: register -> the fewest states since it was written
    bad, work = set(), [(0, {})]
    while work:
        n, state = work.pop()
        while n < len(code):
            known = seen[n]
            if known is not None:
                if all(r in known and known[r] <= s for r, s in state.items()):
                    break
                state = {r: min(state.get(r, STATES), known.get(r, STATES)) for r in {*state, *known}}
            seen[n] = dict(state)
            i = code[n]
            if i.mfma and state.keys() & i.reads:
                bad.add((i.address, i.op))
            state = {r: s + i.states for r, s in state.items() if s + i.states < STATES}
            state.update((r, 0) for r in written(i))
            if i.op.startswith("s_endpgm"):
                break
            if i.target is not None:
                if i.op.startswith("s_branch"):
                    n = index[i.target]
                    continue
                work.append((index[i.target], dict(state)))
            n += 1
    return sorted(bad)


@pytest.mark.skipif(not os.path.exists(W.LIB) or not shutil.which(W.OBJDUMP),
                    reason="no built library or no objdump")
def test_no_operand_is_read_too_early(tmp_path):
    seen = 0
    for name, code in K.kernels(tmp_path):
        mfmas = [i for i in code if i.mfma]
        assert len(mfmas) >= 32 and all(i.reads for i in mfmas), name
        assert sum(bool(written(i)) for i in code) > len(mfmas), name
        assert early_operands(code) == [], name
        seen += 1
    assert seen == 16


def stream(*lines, target=None):
    """Instructions of four bytes each; target: {index of a branch: index it goes to}."""
    code = W.instructions(list(lines))
    for i in code:
        i.states = K.PASSES if i.mfma else i.states
        i.reads = set()
    for n, line in enumerate(lines):
        if code[n].mfma:
            code[n].reads = W.registers(line.split(" ", 1)[1].split(", ", 1)[1])
    for n, to in (target or {}).items():
        code[n].target = 4 * to
    return code


MFMA = "v_mfma_i32_16x16x64_i8 a[0:3], v[4:7], v[8:11], a[0:3]"
OTHER = "v_mfma_i32_16x16x64_i8 a[4:7], v[20:23], v[24:27], a[4:7]"
MOVE = "v_mov_b32_e32 v5, v60"
AWAY = "v_mov_b32_e32 v50, v60"
END = "s_endpgm "


def test_the_check_sees_early_operands():
    for lines, early in (((MOVE, MFMA), 1), ((MOVE, AWAY, MFMA), 1), ((MOVE, AWAY, AWAY, MFMA), 0),
                         ((MOVE, "s_nop 0", MFMA), 1), ((MOVE, "s_nop 1", MFMA), 0), ((MOVE, OTHER, MFMA), 0),
                         ((AWAY, MFMA), 0), (("v_mov_b32_e32 v12, v5", MFMA), 0),
                         (("v_accvgpr_write_b32 a2, v60", MFMA), 1),
                         (("v_permlane32_swap_b32_e32 v60, v9", MFMA), 1), ((MFMA, MOVE), 0),
                         (("ds_read_b128 v[4:7], v70", MFMA), 0)):   # (loads have waits of their own)
        assert len(early_operands(stream(*lines, END))) == early, lines


def test_the_check_follows_branches():
    # from a loop's end to the MFMA at its beginning
    assert early_operands(stream(MFMA, AWAY, MOVE, "s_cbranch_scc1 0", END, target={3: 0}))
    assert not early_operands(stream(MFMA, MOVE, AWAY, "s_cbranch_scc1 0", END, target={3: 0}))
    # over a jump, and not over code that is jumped past
    assert early_operands(stream(MOVE, "s_branch 3", AWAY, AWAY, MFMA, END, target={1: 4}))
    assert not early_operands(stream("s_branch 2", MOVE, MFMA, END, target={0: 2}))
    # from one of two ways to the same place
    assert early_operands(stream("s_cbranch_scc1 3", AWAY, "s_branch 4", MOVE, MFMA, END, target={0: 3, 2: 4}))
