"""What the loads to LDS owe the compiler (see test_wait_states.py), in the kernels
of the gated block and of the products with adapters.  Nothing runs on a GPU."""

import os
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from combine_ep_dispatch_amd import build
from test_wait_states import compiled, short_waits

SOURCES = ("expert_gated", "expert_lora", "expert_nvfp4_block")


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
    loads = re.findall(r"buffer_load_\w+ (v\d+), (\S)\S+ (\S+) offen lds", assembly[name])
    assert len(loads) > 50 and {v[1:] for v in loads} == {("s", "0")}
