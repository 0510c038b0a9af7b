"""Argument checks of the gated block's calls and of those with adapters: every
invalid argument is refused on the host before anything is enqueued.  No call here
reaches a launch."""

import ctypes

import pytest
import torch

import combine_ep_dispatch_amd as epx
from combine_ep_dispatch_amd._lib import EpLora
from test_expert_layer_args import FAKE, INVALID, L, cfg, lay  # noqa: F401

GOOD = dict(token_adapter=FAKE, a=FAKE, b=FAKE, scale=None, num_adapters=4, rank=16, reserved0=0, reserved1=0)


def lora(**kw):
    return EpLora(*[{**GOOD, **kw}[n] for n, _ in EpLora._fields_])


# name: (multiple of in_dim, dimensions, pointers behind them (? may be NULL), what follows, reads a, reads b)
CALLS = {
    "ep_lora_down": (8, "i", "**", (), True, False),
    "ep_lora_bwd_u": (8, "o", "**", (), False, True),
    "ep_lora_bwd_w": (8, "io", "******", (1,), False, False),
    "ep_expert_gemm_lora": (8, "io", "****", (), False, True),
    "ep_expert_gemm_nvfp4_lora": (16, "io", "******", (), False, True),
    "ep_expert_gemm_bwd_x_lora": (8, "io", "****", (), True, False),
    "ep_expert_gated": (8, "io", "**?**", (), False, True),
    "ep_expert_gated_nvfp4": (16, "io", "****?**", (), False, True),
    "ep_expert_gated_bwd": (8, "io", "**?***??", (FAKE, 1 << 20), False, True),
}


def call(L, name, c=None, y=None, lo=None, i=64, o=64, ptrs=None, extra=None):  # noqa: F811
    _, dims, pointers, more, _, _ = CALLS[name]
    c, y, lo = c or cfg().to_c(), y or lay(), lora() if lo is None else lo
    sizes = [{"i": i, "o": o}[k] for k in dims]
    ref = lambda v: None if v == "null" else ctypes.byref(v)  # noqa: E731
    return getattr(L, name)(ref(c), ref(y), ref(lo), *sizes, *(ptrs or [FAKE] * len(pointers)),
                            *(more if extra is None else extra), None)


def test_lora_struct_is_the_headers():
    assert ctypes.sizeof(EpLora) == 48
    assert EpLora.num_adapters.offset == 32


@pytest.mark.parametrize("name", CALLS)
def test_bad_sizes_pointers_and_layouts(L, name):  # noqa: F811
    multiple, dims, pointers, _, _, _ = CALLS[name]
    for i in [0, -16, 4, 12, (1 << 20) + 16] + ([8, 24] if multiple == 16 else []):
        if "i" in dims:
            assert call(L, name, i=i) == INVALID, i
    for o in (0, -8, 4, 12, (1 << 20) + 8):
        if "o" in dims:
            assert call(L, name, o=o) == INVALID, o
    for k, kind in enumerate(pointers):
        for v in ([FAKE + 1] if kind == "?" else [None, FAKE + 1]):
            ptrs = [FAKE] * len(pointers)
            ptrs[k] = v
            assert call(L, name, ptrs=ptrs) == INVALID, (k, v)
    assert call(L, name, c="null") == INVALID
    assert call(L, name, y="null") == INVALID
    for field in ("counts", "row_offsets", "seg_base", "src_info"):
        assert call(L, name, y=lay(**{field: None})) == INVALID, field
    assert call(L, name, y=lay(src_info=FAKE + 4)) == INVALID
    assert call(L, name, c=cfg(recv_rows=1).to_c()) == INVALID


@pytest.mark.parametrize("name", CALLS)
def test_bad_adapters(L, name):  # noqa: F811
    _, _, _, _, reads_a, reads_b = CALLS[name]
    bad = [dict(num_adapters=0), dict(num_adapters=-1), dict(num_adapters=65537), dict(rank=0), dict(rank=4),
           dict(rank=12), dict(rank=136), dict(rank=-8), dict(reserved0=1), dict(reserved1=1), dict(token_adapter=None),
           dict(token_adapter=FAKE + 2), dict(scale=FAKE + 2)]
    bad += [dict(a=v) for v in (None, FAKE + 8) if reads_a] + [dict(b=v) for v in (None, FAKE + 8) if reads_b]
    for kw in bad:
        assert call(L, name, lo=lora(**kw)) == INVALID, kw
    if not name.startswith("ep_expert_gated"):
        assert call(L, name, lo="null") == INVALID


def test_u_without_adapters_is_refused(L):  # noqa: F811
    for name in ("ep_expert_gated", "ep_expert_gated_nvfp4", "ep_expert_gated_bwd"):
        assert call(L, name, lo="null") == INVALID, name


def test_gated_bwd_refuses_a_small_or_missing_workspace(L):  # noqa: F811
    need = 16 * 2 * 2 * 4  # T * K * ceil(64 / 32) floats
    for extra in ((None, 1 << 20), (FAKE + 8, 1 << 20), (FAKE, need - 1), (FAKE, 0), (FAKE, -1)):
        assert call(L, "ep_expert_gated_bwd", extra=extra) == INVALID, extra
    assert call(L, "ep_expert_gated_bwd", y=lay(token_row=None)) == INVALID


def test_lora_bwd_w_refuses_unknown_types(L):  # noqa: F811
    for kind in (-1, 3):
        assert call(L, "ep_lora_bwd_w", extra=(kind,)) == INVALID


@pytest.mark.parametrize("dims", [(8, 8192), (8192, 8)], ids=str)
def test_lora_bwd_w_refuses_both_gradients_where_one_passes_a_grid(L, dims):  # noqa: F811
    """65536 adapters of 8 experts: 2^19 tiles of one gradient, 2^24 of the other.  The call
    launches twice and answers before the first launch (and before it asks for a device)."""
    big = lora(num_adapters=65536, rank=8)
    assert cfg().num_experts == 8
    assert call(L, "ep_lora_bwd_w", lo=big, i=dims[0], o=dims[1]) == INVALID


def test_gated_nvfp4_refuses_weights_past_32_bit_offsets(L):  # noqa: F811
    assert call(L, "ep_expert_gated_nvfp4", i=1 << 20, o=1 << 14) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    c = cfg()
    rows = torch.zeros(c.recv_rows, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(4, 8, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 8, 64, 16, dtype=torch.bfloat16)
    ids, u = torch.zeros(16, dtype=torch.int32), torch.zeros(c.recv_rows, 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        epx.ep_lora_down(c, None, rows, epx.Adapters(ids, a, b), u)
    with pytest.raises(ValueError, match="GPU tensor"):
        epx.ep_expert_gated(c, None, rows, rows, None, rows)
    with pytest.raises(ValueError, match="columns"):
        epx.ep_expert_gated(c, None, rows.view(-1), rows, None, rows)
    for bad in (epx.Adapters(ids, a[0], b), epx.Adapters(ids, a, b[:3]), epx.Adapters(ids, a[..., :32], b),
                epx.Adapters(ids, a[:, :7], b), epx.Adapters(ids, a, b[..., :8])):
        with pytest.raises(ValueError, match="adapters|columns|GPU"):
            bad.to_c(c, 64, 64, torch.device("cpu"))
    with pytest.raises(ValueError, match="without adapters"):
        epx._lora(c, None, u, 64, 64, None)
    with pytest.raises(ValueError, match="grad_a"):
        epx.ep_lora_bwd_w(c, None, rows, rows, epx.Adapters(ids, a, b), u, u, a.half(), b.half())


def test_dispatcher_refuses_a_scale_that_asks_for_a_gradient():
    from combine_ep_dispatch_amd.autograd import _parts

    a, b = torch.zeros(4, 8, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 8, 64, 16, dtype=torch.bfloat16)
    adapters = epx.Adapters(torch.zeros(16, dtype=torch.int32), a, b, torch.ones(4, requires_grad=True))
    with pytest.raises(ValueError, match="scale gets no gradient"):
        _parts(adapters)
    with torch.no_grad():
        assert not _parts(adapters)[3].requires_grad
