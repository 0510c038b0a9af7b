"""Argument checks of the expert layer's calls (ep_route, ep_swiglu,
ep_expert_gemm and their backward calls): every invalid argument is refused
on the host before anything is enqueued.  No call here reaches a launch."""

import ctypes
import os

import pytest
import torch

import combine_ep_dispatch_amd as epx
from combine_ep_dispatch_amd import _lib
from combine_ep_dispatch_amd._lib import EpLayout, EpRoute

FAKE = 0x10000  # an aligned address that is never dereferenced
INVALID = -1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from combine_ep_dispatch_amd import build

        build.build()
    return _lib.lib()


def cfg(**kw):
    base = dict(num_tokens=16, hidden=64, num_experts=8, num_segments=2, top_k=2, align=4, recv_rows=4096)
    return epx.EpConfig(**{**base, **kw})


def lay(**kw):
    layout = EpLayout(*([FAKE] * 8))
    for k, v in kw.items():
        setattr(layout, k, v)
    return layout


def route(**kw):
    base = dict(score=0, normalize=1, num_groups=1, top_groups=1, scale=1.0, logits_type=0, reserved0=0, reserved1=0)
    base.update(kw)
    return EpRoute(*[base[n] for n, _ in EpRoute._fields_])


def test_route_struct_is_the_headers():
    assert ctypes.sizeof(EpRoute) == 32
    assert EpRoute.scale.offset == 16


BAD_ROUTES = [dict(score=2), dict(score=-1), dict(normalize=2), dict(num_groups=0), dict(num_groups=3),
              dict(num_groups=-1), dict(top_groups=0), dict(top_groups=2), dict(num_groups=4, top_groups=5),
              dict(scale=float("inf")), dict(scale=float("nan")), dict(logits_type=2), dict(reserved0=1),
              dict(reserved1=1)]


@pytest.mark.parametrize("bad", BAD_ROUTES, ids=str)
def test_route_refuses_a_bad_description(L, bad):
    c, r = cfg().to_c(), route(**bad)
    assert L.ep_route(ctypes.byref(c), ctypes.byref(r), FAKE, None, None, FAKE, FAKE, None) == INVALID
    assert L.ep_route_bwd(ctypes.byref(c), ctypes.byref(r), FAKE, FAKE, FAKE, FAKE, None) == INVALID


def test_route_refuses_bad_pointers_and_sizes(L):
    c, r = cfg().to_c(), route()
    fwd = [FAKE, None, None, FAKE, FAKE]
    for i, v in ((0, None), (0, FAKE + 8), (1, FAKE + 2), (3, None), (3, FAKE + 1), (4, None), (4, FAKE + 2)):
        a = list(fwd)
        a[i] = v
        assert L.ep_route(ctypes.byref(c), ctypes.byref(r), *a, None) == INVALID, (i, v)
    for i in range(4):
        for v in (None, FAKE + 2):
            a = [FAKE] * 4
            a[i] = v
            assert L.ep_route_bwd(ctypes.byref(c), ctypes.byref(r), *a, None) == INVALID, (i, v)
    assert L.ep_route(None, ctypes.byref(r), *fwd, None) == INVALID
    assert L.ep_route(ctypes.byref(c), None, *fwd, None) == INVALID
    many = cfg(num_experts=128, num_segments=1).to_c()
    r65 = route(num_groups=128)
    assert L.ep_route(ctypes.byref(many), ctypes.byref(r65), *fwd, None) == INVALID
    huge = cfg(num_tokens=1 << 26).to_c()
    assert L.ep_route(ctypes.byref(huge), ctypes.byref(r), *fwd, None) == INVALID


@pytest.mark.parametrize("inter", [0, -8, 4, 12, (1 << 20) + 8])
def test_swiglu_refuses_bad_widths(L, inter):
    c, y = cfg().to_c(), lay()
    assert L.ep_swiglu(ctypes.byref(c), ctypes.byref(y), inter, FAKE, None, FAKE, None) == INVALID
    assert L.ep_swiglu_bwd(ctypes.byref(c), ctypes.byref(y), inter, FAKE, None, FAKE, FAKE, None, None) == INVALID


def test_swiglu_refuses_bad_pointers(L):
    c, y = cfg().to_c(), lay()
    for a in ((None, None, FAKE), (FAKE + 8, None, FAKE), (FAKE, FAKE + 2, FAKE), (FAKE, None, None), (FAKE, None, FAKE + 4)):
        assert L.ep_swiglu(ctypes.byref(c), ctypes.byref(y), 64, *a, None) == INVALID, a
    good = [FAKE, None, FAKE, FAKE, None]
    for i, v in ((0, None), (0, FAKE + 8), (1, FAKE + 2), (2, None), (2, FAKE + 8), (3, None), (3, FAKE + 8), (4, FAKE + 1)):
        a = list(good)
        a[i] = v
        assert L.ep_swiglu_bwd(ctypes.byref(c), ctypes.byref(y), 64, *a, None) == INVALID, (i, v)
    assert L.ep_swiglu(ctypes.byref(c), None, 64, FAKE, None, FAKE, None) == INVALID
    none = lay(token_row=None)
    assert L.ep_swiglu(ctypes.byref(c), ctypes.byref(none), 64, FAKE, None, FAKE, None) == INVALID
    short = cfg(recv_rows=1).to_c()
    assert L.ep_swiglu(ctypes.byref(short), ctypes.byref(y), 64, FAKE, None, FAKE, None) == INVALID


def products(L):
    """Each product call as (name, function of (cfg, layout, in, out, pointers), pointers)."""
    return [
        ("gemm", L.ep_expert_gemm, 3, ()),
        ("bwd_x", L.ep_expert_gemm_bwd_x, 3, ()),
        ("bwd_w", L.ep_expert_gemm_bwd_w, 3, (0,)),
        ("nvfp4", L.ep_expert_gemm_nvfp4, 5, ()),
    ]


@pytest.mark.parametrize("which", range(4), ids=["gemm", "bwd_x", "bwd_w", "nvfp4"])
def test_products_refuse_bad_arguments(L, which):
    name, call, n, extra = products(L)[which]
    c, y = cfg().to_c(), lay()

    def go(c=c, y=y, i=64, o=64, ptrs=None, extra=extra):
        return call(None if c is None else ctypes.byref(c), None if y is None else ctypes.byref(y), i, o,
                    *(ptrs or [FAKE] * n), *extra, None)

    bad_in = [0, -16, 4, 12, (1 << 20) + 16] + ([8, 24] if name == "nvfp4" else [])
    for i in bad_in:
        assert go(i=i) == INVALID, i
    for o in (0, -8, 4, 12, (1 << 20) + 8):
        assert go(o=o) == INVALID, o
    for k in range(n):
        for v in (None, FAKE + 1):
            ptrs = [FAKE] * n
            ptrs[k] = v
            assert go(ptrs=ptrs) == INVALID, (k, v)
    assert go(c=None) == INVALID
    assert go(y=None) == INVALID
    for field in ("counts", "row_offsets", "seg_base"):
        assert go(y=lay(**{field: None})) == INVALID, field
    assert go(c=cfg(recv_rows=1).to_c()) == INVALID
    if name == "bwd_w":
        for kind in (-1, 3):
            assert go(extra=(kind,)) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    c = cfg()
    ids, p = torch.zeros(16, 2, dtype=torch.int32), torch.zeros(16, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        epx.ep_route(c, epx.RouteConfig(), torch.zeros(16, 8), ids, p)
    with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
        epx.ep_route(c, epx.RouteConfig(), torch.zeros(16, 8, dtype=torch.float16), ids, p)
    with pytest.raises(ValueError, match="score"):
        epx.ep_route(c, epx.RouteConfig(score="relu"), torch.zeros(16, 8), ids, p)
    rows = torch.zeros(c.recv_rows, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="columns"):
        epx.ep_expert_gemm(c, None, rows.view(-1), rows, rows)
    with pytest.raises(ValueError, match="GPU tensor"):
        epx.ep_expert_gemm(c, None, rows, rows, rows)
    with pytest.raises(ValueError, match="GPU tensor"):
        epx.ep_swiglu(c, None, rows, None, rows)
    with pytest.raises(ValueError, match="grad_w"):
        epx.ep_expert_gemm_bwd_w(c, None, rows, rows, torch.zeros(8, 64, 64, dtype=torch.float16))
