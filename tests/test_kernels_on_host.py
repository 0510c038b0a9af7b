"""Kernels run on the host, lane by lane (host/kernels.h): no load reads past its
operand, the last expert's last rows included, and no result depends on when loads to
LDS land or on which wave of a workgroup runs ahead.  Nothing runs on a GPU."""

import os
import re
import subprocess

import pytest

from combine_ep_dispatch_amd import build

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "host")
SOURCES = {"expert_gated": 0, "expert_lora": 1, "expert_nvfp4_block": 2, "expert_gemm": 3, "expert_nvfp4": 4}  # name, number in expert_block.cpp
HEADERS = ("epx_device", "expert_device", "expert_tile", "expert_loop", "lora_device", "gated_device", "nvfp4_tile")

# What the inline assembly does, in the host's words.
ASSEMBLY = [
    (r'"s_mov_b32 m0, %0\\n\\ts_nop 3\\n\\tbuffer_load_dwordx4 %1, %2, 0 offen lds".*?', "host::aim(to); host::load(16, rs, voff);"),
    (r'"s_mov_b32 m0, %0\\n\\ts_nop 3\\n\\tbuffer_load_dword %1, %2, 0 offen lds".*?', "host::aim(to); host::load(4, rs, voff);"),
    (r'"s_mov_b32 m0, %0\\n\\ts_nop 3\\n\\tbuffer_load_ubyte %1, %2, 0 offen lds".*?', "host::aim(to); host::load(1, rs, voff);"),
    (r'"s_add_u32 m0, %0, %1\\n\\ts_nop 0\\n\\tbuffer_load_dwordx4 %2, %3, 0 offen lds".*?',
     "host::aim(to + OFF); host::load(16, rs, voff);"),
    (r'"s_add_u32 m0, %0, %1" .*?', "host::aim(to + OFF);"),
    (r'"buffer_load_dwordx4 %0, %1, 0 offen lds".*?', "host::load(16, rs, voff);"),
    (r'"s_waitcnt vmcnt\(%0\)" ::"n"\((.*?)\) : "memory"', r"host::vmcnt(\1);"),
    (r'"s_waitcnt vmcnt\(0\)" ::: "memory"', "host::vmcnt(0);"),
    (r'"s_waitcnt lgkmcnt\(0\)" ::: "memory"', "host::exchange(host::kWave, 0);"),
    (r'"s_nop 4" : "\+s"\(rs\)', ""),
    (r'"" : "\+a"\(v\)', ""),
]


def on_the_host(text):
    for pattern, words in ASSEMBLY:
        text = re.sub(r"asm volatile\(" + pattern + r"\);", "{ " + words + " }", text, flags=re.S)
    text = text.replace("__attribute__((address_space(3)))", "")
    text = text.replace("constexpr int kCus = 256;", "constexpr int kCus = 8;")  # few, so that workgroups take many tiles
    assert "asm" not in re.sub(r"//.*", "", text).replace("Winline-asm", "")
    return text


@pytest.fixture(scope="module")
def programs(tmp_path_factory):
    """A host program of each source."""
    at = tmp_path_factory.mktemp("host")
    (at / "hip").mkdir()
    with open(os.path.join(HERE, "kernels.h")) as f:
        (at / "hip" / "hip_runtime.h").write_text(f.read())
    for name in [h + ".h" for h in HEADERS] + [s + ".hip" for s in SOURCES]:
        with open(os.path.join(build.CSRC, name)) as f:
            (at / name).write_text(on_the_host(f.read()))
    clang = os.path.join(os.path.dirname(os.path.realpath(build.hipcc())), "..", "lib", "llvm", "bin", "clang++")
    if not os.path.exists(clang):
        clang = "/opt/rocm/llvm/bin/clang++"
    runs = [subprocess.Popen([clang, "-x", "c++", "-std=c++17", "-O2", "-w", "-ffp-contract=off", "-no-pie", f"-DSOURCE={n}",
                              "-I", str(at), "-I", build.INCLUDE, os.path.join(HERE, "expert_block.cpp"), "-o", str(at / name)],
                             stderr=subprocess.PIPE, text=True) for name, n in SOURCES.items()]
    for run in runs:
        _, errors = run.communicate()
        assert run.returncode == 0, errors
    return {name: str(at / name) for name in SOURCES}


def run(program, ins, outs):
    """One process for each of ins."""
    runs = [subprocess.Popen([program, str(n), "x", *map(str, outs)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            for n in ins]
    said = [r.communicate()[0] for r in runs]
    for r, text in zip(runs, said):
        assert r.returncode == 0 and re.fullmatch(r"\d+ cases\n", text), text


@pytest.mark.parametrize("name", ["expert_gated", "expert_lora"])
def test_products(programs, name):
    """Workgroups that go from tile to tile and from one kind of tiles to the next."""
    run(programs[name], (8, 136, 264), (8, 136))


def test_four_bit_products(programs):
    """Widths of which a tile's last waves have nothing, and those that fill one."""
    run(programs["expert_nvfp4_block"], (16, 64, 272), (8, 40, 136))
    run(programs["expert_nvfp4"], (16, 64, 272, 320), (8, 40, 136, 264))


def test_products_without_an_end_of_their_own(programs):
    """The products and both gradients, in small and in wide tiles."""
    run(programs["expert_gemm"], (8, 136, 264), (136,))
