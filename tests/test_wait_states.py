"""What the loads to LDS that the experts' products issue from inline assembly
owe the compiler: it inserts the wait states that the hardware needs between its
own instructions, not before one inside an asm block, and takes M0 for unchanged
unless the block says otherwise.  Sources are compiled to assembly and read;
nothing runs on a GPU."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from combine_ep_dispatch_amd import build

SOURCES = ("expert_gemm", "expert_nvfp4")
VALU_SGPR_TO_VMEM = 5  # wait states between a vector instruction's write of an SGPR and a memory instruction that reads it
M0_TO_LDS_LOAD = 1     # and between a write of M0 and a load to LDS
TWO_RESULTS = ("v_add_co", "v_addc_co", "v_sub_co", "v_subb_co", "v_subrev_co", "v_subbrev_co", "v_div_scale", "v_mad_u64",
               "v_mad_i64")


def sgprs(operand):
    """Numbers of the SGPRs that an operand names."""
    out = set()
    for word in operand.split():
        if m := re.fullmatch(r"s\[(\d+):(\d+)\]", word):
            out |= set(range(int(m[1]), int(m[2]) + 1))
        elif m := re.fullmatch(r"s(\d+)", word):
            out.add(int(m[1]))
    return out


def short_waits(assembly):
    """(line number, line, wait states) of the memory instructions that come too
    soon behind a vector instruction's write of one of their SGPRs, or of M0, and
    how many loads to LDS there are."""
    bad, before, loads = [], [], 0  # before: (SGPRs written by a vector instruction, M0 written, wait states of the instruction)
    for number, line in enumerate(assembly.splitlines(), 1):
        code = line.split(";")[0].strip()
        if not code or code.startswith(".") or code.endswith(":"):
            continue
        op, _, rest = code.partition(" ")
        operands = [o.strip() for o in re.split(r",(?![^\[]*\])", rest)]
        if op.startswith(("buffer_", "global_", "flat_", "scratch_")):
            used = set().union(*map(sgprs, operands))
            to_lds = operands[-1].split()[-1] == "lds"
            loads += to_lds
            waits = 0
            for written, m0, states in reversed(before):
                if waits >= VALU_SGPR_TO_VMEM:
                    break
                if written & used or (to_lds and m0 and waits < M0_TO_LDS_LOAD):
                    bad.append((number, code, waits))
                    break
                waits += states
        written = set()
        if op.startswith("v_"):
            written = sgprs(operands[0]) | (sgprs(operands[1]) if op.startswith(TWO_RESULTS) else set())
        before.append((written, operands[0] == "m0", int(operands[0]) + 1 if op == "s_nop" else 1))
        del before[:-8]
    return bad, loads


def test_the_reader_sees_short_waits():
    read = "\tv_readfirstlane_b32 s6, v1\n\ts_mov_b32 m0, s0\n\ts_nop %d\n\tbuffer_load_dwordx4 v0, s[4:7], 0 offen lds\n"
    assert short_waits(read % 0)[0] == [(4, "buffer_load_dwordx4 v0, s[4:7], 0 offen lds", 2)]
    assert short_waits(read % 3) == ([], 1)
    assert short_waits("\ts_mov_b32 m0, s0\n\tbuffer_load_dword v0, s[4:7], s9 offen lds\n")[0][0][2] == 0
    assert short_waits("\tv_cmp_gt_i32_e64 s[8:9], v0, v1\n\tbuffer_load_dword v0, s[4:7], s9 offen lds\n")[0][0][2] == 0
    assert short_waits("\tv_cmp_gt_i32_e64 s[8:9], v0, v1\n\tbuffer_load_dword v0, s[4:7], s10 offen lds\n") == ([], 1)


def compiled(source, out):
    """The device assembly of a source, as the library's build compiles it."""
    subprocess.run([build.hipcc(), *build.compile_flags(), "-S", "--cuda-device-only", "-o", out, source], check=True,
                   capture_output=True)
    with open(out) as f:
        return f.read()


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    at = tmp_path_factory.mktemp("assembly")

    def one(name):
        return compiled(os.path.join(build.CSRC, f"{name}.hip"), str(at / f"{name}.s"))

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        return dict(zip(SOURCES, pool.map(one, SOURCES)))


@pytest.mark.parametrize("name", SOURCES)
def test_loads_to_lds_wait_for_their_descriptors(assembly, name):
    bad, loads = short_waits(assembly[name])
    assert loads > 50
    assert not bad


@pytest.mark.parametrize("name", SOURCES)
def test_loads_to_lds_keep_their_offset_in_the_range_check(assembly, name):
    """The check of an address against the buffer's size leaves the scalar offset
    out: with one, a load past the buffer's last bytes is not caught."""
    loads = re.findall(r"buffer_load_\w+ (v\d+), (\S)\S+ (\S+) offen lds", assembly[name])
    assert len(loads) > 50 and {v[1:] for v in loads} == {("s", "0")}


def test_a_value_in_m0_is_written_again_behind_a_load(tmp_path):
    """Two messages whose operand is m0, a load between them: m0 has to be set for
    the second one too."""
    source = tmp_path / "m0.hip"
    source.write_text("""
        #include "expert_device.h"
        __global__ void k(const int* p, int n, int m) {
            __shared__ int lds[64];
            __builtin_amdgcn_s_sendmsg(1, m);
            epx::load_to_lds<4>(p, n, lds, threadIdx.x * 4);
            __builtin_amdgcn_s_sendmsg(1, m);
        }
    """)
    lines = compiled(str(source), str(tmp_path / "m0.s")).splitlines()
    on = [line.split()[0] for line in lines if re.search(r"\bs_sendmsg\b|\bm0,|offen lds", line)]
    assert on == ["s_mov_b32", "s_sendmsg", "s_mov_b32", "buffer_load_dword", "s_mov_b32", "s_sendmsg"]
