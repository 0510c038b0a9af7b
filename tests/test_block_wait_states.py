"""What the loads to LDS owe the compiler (see test_wait_states.py), in the kernels
of the gated block and of the products with adapters, along every way that the
branches leave open.  Nothing runs on a GPU."""

import os
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from combine_ep_dispatch_amd import build
from test_wait_states import M0_TO_LDS_LOAD, TWO_RESULTS, VALU_SGPR_TO_VMEM, compiled, sgprs

SOURCES = ("expert_gated", "expert_lora", "expert_nvfp4_block")


class Line:
    """An instruction: what it writes and how many wait states it is."""

    def __init__(self, number, code):
        self.number, self.code = number, code
        self.op, _, rest = code.partition(" ")
        self.operands = [o.strip() for o in re.split(r",(?![^\[]*\])", rest)]
        self.written = set()  # SGPRs, by a vector instruction
        if self.op.startswith("v_"):
            self.written = sgprs(self.operands[0]) | (sgprs(self.operands[1]) if self.op.startswith(TWO_RESULTS) else set())
        self.m0 = self.operands[0] == "m0"
        self.states = int(self.operands[0]) + 1 if self.op == "s_nop" else 1
        self.to_lds = self.op.startswith("buffer_") and self.operands[-1].split()[-1] == "lds"
        self.before = []


def functions(assembly):
    """The instructions of every function, each with those that may run right before it."""
    out = []
    for body in re.findall(r"^\S+:[^\n]*@\S+\n(.*?)^\.Lfunc_end", assembly, re.S | re.M):
        lines, labels, waiting, last = [], {}, [], None
        for number, text in enumerate(body.splitlines(), 1):
            code = text.split(";")[0].strip()
            if not code or (code.startswith(".") and not code.endswith(":")):
                continue
            if code.endswith(":"):
                waiting.append(code[:-1])
                continue
            line = Line(number, code)
            for name in waiting:
                labels[name] = line
            waiting = []
            if last is not None and last.op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                line.before.append(last)
            lines.append(line)
            last = line
        for line in lines:
            if line.op.startswith(("s_branch", "s_cbranch")) and line.operands[0] in labels:
                labels[line.operands[0]].before.append(line)
        out.append(lines)
    return out


def short_waits(lines):
    """Memory instructions that may come too soon behind a vector instruction's write
    of one of their SGPRs, or, to LDS, behind a write of M0."""
    bad = []
    for line in lines:
        if not line.op.startswith(("buffer_", "global_", "flat_", "scratch_")):
            continue
        used = set().union(*map(sgprs, line.operands))
        todo, seen = [(b, 0) for b in line.before], {}
        while todo:
            b, waits = todo.pop()
            if waits >= VALU_SGPR_TO_VMEM or seen.get(b, VALU_SGPR_TO_VMEM) <= waits:
                continue
            seen[b] = waits
            if b.written & used or (line.to_lds and b.m0 and waits < M0_TO_LDS_LOAD):
                bad.append((line.number, line.code, b.code, waits))
                break
            todo += [(p, waits + b.states) for p in b.before]
    return bad


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    at = tmp_path_factory.mktemp("assembly")

    def one(name):
        return compiled(os.path.join(build.CSRC, f"{name}.hip"), str(at / f"{name}.s"))

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        return dict(zip(SOURCES, pool.map(one, SOURCES)))


def test_the_reader_follows_branches():
    text = ("k:  ; @k\n\tv_readlane_b32 s6, v1, 0\n\ts_cbranch_scc1 .LBB0_2\n\ts_nop 4\n.LBB0_2:\n"
            "\ts_mov_b32 m0, s0\n\ts_nop 0\n\tbuffer_load_dwordx4 v0, s[4:7], 0 offen lds\n\ts_endpgm\n.Lfunc_end0:\n")
    assert [b[2:] for b in short_waits(functions(text)[0])] == [("v_readlane_b32 s6, v1, 0", 3)]
    assert short_waits(functions(text.replace("s_nop 0", "s_nop 2"))[0]) == []
    assert short_waits(functions(text.replace("\ts_nop 0\n", "").replace("v_readlane_b32 s6", "v_readlane_b32 s9"))[0])


@pytest.mark.parametrize("name", SOURCES)
def test_loads_to_lds_wait_for_their_descriptors_and_m0(assembly, name):
    loads = 0
    for lines in functions(assembly[name]):
        loads += sum(line.to_lds for line in lines)
        assert not short_waits(lines)
    assert loads > 50


@pytest.mark.parametrize("name", SOURCES)
def test_loads_to_lds_keep_their_offset_in_the_range_check(assembly, name):
    loads = re.findall(r"buffer_load_\w+ (v\d+), (\S)\S+ (\S+) offen lds", assembly[name])
    assert len(loads) > 50 and {v[1:] for v in loads} == {("s", "0")}


@pytest.mark.parametrize("name", SOURCES)
def test_branches_reach(assembly, name):
    """Kernels stay small enough for their branches: past that the compiler goes by
    computed addresses, which the reader above does not follow."""
    assert "s_setpc" not in assembly[name]


@pytest.mark.parametrize("name", SOURCES)
def test_m0_is_written_for_every_load_and_for_nothing_else(assembly, name):
    """A load's LDS address is set some instructions ahead of it: nothing else may
    write M0 in between, or at all."""
    for lines in functions(assembly[name]):
        writes = [line for line in lines if any(re.search(r"\bm0\b", o) for o in line.operands)]
        assert all(line.m0 and line.op in ("s_mov_b32", "s_add_u32") for line in writes)
        kinds = [line.to_lds for line in lines if line.m0 or line.to_lds]
        assert kinds == [False, True] * (len(kinds) // 2)
