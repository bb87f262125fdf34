"""Inline assembly in the built kernels keeps the wait states that the hardware
does not keep by itself, on every way through the control flow (CPU only: the
kernels are compiled to assembly and read, never run)."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from mixture_experts_layer_permute_amd import build

from _waits import blocks, functions, scan
from test_debug_build import device_asm

# the sources with loads or matrix instructions in inline assembly
SOURCES = ("head.hip", "ggemm.hip")


@pytest.fixture(scope="module")
def found(tmp_path_factory):
    if not os.path.exists(build.hipcc()):
        pytest.skip("no hipcc")
    d = str(tmp_path_factory.mktemp("waits"))
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        asm = dict(zip(SOURCES, ex.map(lambda s: device_asm(s, False, d), SOURCES)))
    return {s: {n: (b, scan(b)) for n, b in functions(a, r"_ZN3moe\w+")} for s, a in asm.items()}


@pytest.fixture(scope="module")
def found_debug(tmp_path_factory):
    if not os.path.exists(build.hipcc()):
        pytest.skip("no hipcc")
    d = str(tmp_path_factory.mktemp("waits_debug"))
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        asm = dict(zip(SOURCES, ex.map(lambda s: device_asm(s, True, d), SOURCES)))
    return {s: {n: (b, scan(b)) for n, b in functions(a, r"_ZN3moe\w+")} for s, a in asm.items()}


def short(found, src, rules):
    return [(n, x) for n, (_, f) in found[src].items() for x in f if x[0] in rules]


@pytest.mark.parametrize("src", SOURCES)
def test_a_descriptor_is_there_when_a_load_reads_it(found, src):
    loads = sum(i.inline and i.lds_load for b, _ in found[src].values() for ins, _ in b for i in ins)
    assert loads >= 32                       # (the reader sees the loads)
    assert short(found, src, ("sgpr",)) == []


@pytest.mark.parametrize("src", SOURCES)
def test_m0_is_there_when_a_load_into_lds_reads_it(found, src):
    assert short(found, src, ("m0",)) == []


@pytest.mark.parametrize("src", SOURCES)
def test_the_debug_build_waits_too(found_debug, src):
    """Its checks move the registers around."""
    assert short(found_debug, src, ("sgpr", "m0", "mfma in", "mfma out")) == []


def test_matrix_instructions_keep_their_distance_over_a_loops_end_too(found):
    inline = sum(i.inline and i.mfma for b, _ in found["head.hip"].values()
                 for ins, _ in b for i in ins)
    assert inline >= 256
    assert short(found, "head.hip", ("mfma in", "mfma out")) == []


LOAD = "\t;;#ASMSTART\n\ts_add_u32 m0, s9, 0\n\ts_nop %d\n\tbuffer_load_dwordx4 v1, s[4:7], 0 " \
       "offen lds\n\t;;#ASMEND\n"
MFMA = "\t;;#ASMSTART\n\tv_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n\t;;#ASMEND\n"


def rules(text):
    return [(x[0], x[1]) for x in scan(blocks(text))]


def test_the_reader_sees_short_distances():
    write = "\tv_readfirstlane_b32 s5, v2\n"
    assert rules(write + LOAD % 0) == [("sgpr", 2)]
    assert rules(write + LOAD % 2) == [("sgpr", 4)]
    assert rules(write + LOAD % 3) == []
    assert rules(write + "\ts_mov_b32 s5, s3\n" + LOAD % 0) == []       # a scalar one instead
    near = "\t;;#ASMSTART\n\ts_mov_b32 m0, s9\n\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds\n" \
           "\t;;#ASMEND\n"
    assert rules(near) == [("m0", 0)]
    assert rules("\tv_mov_b32_e32 v5, 0\n" + MFMA) == [("mfma in", 0)]
    assert rules("\tv_mov_b32_e32 v5, 0\n\ts_nop 1\n" + MFMA) == []
    assert rules(MFMA + "\ts_nop 3\n\tv_accvgpr_read_b32 v9, a2\n") == [("mfma out", 4)]
    assert rules(MFMA + "\ts_nop 7\n\tv_accvgpr_read_b32 v9, a2\n") == []


def test_the_reader_follows_branches():
    # a vector write at a loop's end before the load or the product at its head
    loop = ".LBB0_1:\n%s\ts_nop 9\n\ts_nop 9\n%s\ts_cbranch_scc1 .LBB0_1\n\ts_endpgm\n"
    assert rules(loop % (LOAD % 0, "\tv_readlane_b32 s4, v3, 2\n")) == [("sgpr", 3)]
    assert rules(loop % (MFMA, "\tv_add_u32_e32 v6, 1, v6\n")) == [("mfma in", 1)]
    assert rules(loop % (LOAD % 0, "")) == rules(loop % (MFMA, "")) == []
    # the product at the end, its result read at the head
    assert rules(loop % ("\tv_accvgpr_read_b32 v9, a2\n", MFMA)) == [("mfma out", 1)]
    # the shorter of two ways counts
    two = "\tv_readfirstlane_b32 s5, v2\n\ts_cbranch_scc1 .LBB0_2\n\ts_nop 9\n.LBB0_2:\n" + LOAD % 0
    assert rules(two) == [("sgpr", 3)]
