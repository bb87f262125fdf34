"""The vocabulary head's kernels in assembly (CPU only: compiled and read, never
run): the matrix instructions written as inline assembly keep their distance
from vector instructions that the compiler places around them without knowing of
them, and the debug build checks the indexes that come from data."""
import os
import re

import pytest

from mixture_experts_layer_permute_amd import build

from test_debug_build import device_asm, traps_in

SRC = "head.hip"
# A vector instruction reads or overwrites a result of v_mfma_f32_16x16x32_bf16
# (8 passes of 4 cycles) at the earliest 11 wait states behind it; a matrix
# instruction reads what a vector instruction wrote 2 behind that one.
AFTER, BEFORE = 11, 2


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not os.path.exists(build.hipcc()):
        pytest.skip("no hipcc")
    d = str(tmp_path_factory.mktemp("head"))
    return {debug: device_asm(SRC, debug, d) for debug in (False, True)}


def regs(tok):
    m = re.match(r"([av])\[(\d+):(\d+)\]$", tok)
    if m:
        return [(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)]
    m = re.match(r"([av])(\d+)$", tok)
    return [(m.group(1), int(m.group(2)))] if m else []


def distances(body):
    """(inline matrix instructions, fewest wait states from a vector write to one
    that reads it, fewest from one to a vector instruction on its result), in the
    order of the text; an instruction counts one, s_nop n counts n + 1."""
    inline, now, result, written = False, 0, {}, {}
    count, before, after = 0, 10 ** 9, 10 ** 9
    for line in body.split("\n"):
        if ";;#ASMSTART" in line or ";;#ASMEND" in line:
            inline = "START" in line
            continue
        if not line.startswith("\t") or line.strip().startswith((".", ";")):
            continue
        p = line.split(";")[0].replace(",", " ").split()
        op, toks = p[0], p[1:]
        if op.startswith("v_mfma"):
            if inline:
                count += 1
                for r in (r for t in toks[1:] for r in regs(t)):
                    before = min(before, now - written[r]) if r in written else before
            now += 1
            for r in regs(toks[0]):
                result[r] = (now, inline)
                written.pop(r, None)
            continue
        now += int(toks[0]) + 1 if op == "s_nop" else 1
        if not op.startswith(("v_", "global_store", "buffer_store", "scratch_store", "ds_write")):
            continue
        for r in (r for t in toks for r in regs(t)):
            if r in result and result[r][1]:
                after = min(after, now - 1 - result[r][0])
        if op.startswith("v_"):
            for r in regs(toks[0]):
                result.pop(r, None)
                written[r] = now
    return count, before, after


def test_inline_matrix_instructions_keep_their_distance(asm):
    seen = 0
    for m in re.finditer(r"^(_ZN3moe\w*head_\w+):", asm[False], re.M):
        body = asm[False][m.end():asm[False].find(".Lfunc_end", m.end())]
        n, before, after = distances(body)
        seen += n
        assert before >= BEFORE and after >= AFTER, (m.group(1), n, before, after)
    assert seen >= 256                      # the products of the bf16 kernels


def test_the_reader_sees_a_short_distance():
    near = "\t;;#ASMSTART\n\tv_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n\t;;#ASMEND\n"
    assert distances(near + "\ts_nop 3\n\tv_accvgpr_read_b32 v9, a2\n")[2] == 4
    assert distances(near + "\ts_nop 15\n\tv_accvgpr_mov_b32 a3, a8\n")[2] == 16
    assert distances("\tv_mov_b32_e32 v5, 0\n" + near)[1] == 0
    assert distances("\tv_mov_b32_e32 v5, 0\n\ts_nop 1\n" + near)[1] == 2


def test_no_spills_in_the_loops_of_products(asm):
    for m in re.finditer(r"^(_ZN3moe\w*head_\w+):", asm[False], re.M):
        body = asm[False][m.end():asm[False].find(".Lfunc_end", m.end())]
        for block in re.split(r"^\.LBB\w+:", body, flags=re.M):
            if block.count("v_mfma") >= 64:
                assert "scratch_" not in block, m.group(1)


def test_debug_build_checks_the_row_lists(asm):
    for k in ("head_compact_kernel", "head_start_kernel", "head_gather_kernel"):
        assert traps_in(asm[True], k) > 0, k
        assert traps_in(asm[False], k) == 0, k
