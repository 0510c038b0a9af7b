"""The expert layer's operators on the GPU where memory ends, where keys and
groups are too close to tell in 32 bits, where logits are not finite, and on
several streams at once."""

import numpy as np
import pytest
import torch

from test_gpu_expert_layer import G, Rows, filled, normal, nvfp4_weights  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Memory
# ---------------------------------------------------------------------------
def at_the_end(t):
    """t's values in the last bytes of an allocation of their own."""
    size = t.numel() * t.element_size()
    whole = torch.empty(-(-max(size, 32 << 20) // (2 << 20)) * (2 << 20), dtype=torch.uint8, device=t.device)
    out = whole[whole.numel() - size:].view(t.dtype).view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("n_in", [16, 48, 272, 320, 528, 1040])
@pytest.mark.parametrize("name", ["one", "odd", "aligned", "twenty", "tall"])
def test_operands_that_end_with_their_memory(G, name, n_in):  # noqa: F811
    """Every operand of the products in the last bytes of its allocation (codes of
    widths off 32 end in the middle of a load's 16 bytes): the bits of the same call
    on operands with memory behind them."""
    G.say(f"[gpu] ends of memory {name} in={n_in}")
    d, n_out = Rows(G, name), 80
    x, w = normal(1, d.R, n_in), normal(3, d.experts, n_out, n_in)
    gy = normal(2, d.R, n_out)
    q, _, _ = nvfp4_weights(5, d.experts, n_out, n_in)

    def run(x, gy, w, codes, scales, rowscale):
        y, yq, gx = filled(d.R, n_out), filled(d.R, n_out), filled(d.R, n_in)
        gw = filled(d.experts, n_out, n_in)
        G.epx.ep_expert_gemm_nvfp4(d.cfg, d.lay, x, codes, scales, rowscale, yq)
        G.epx.ep_expert_gemm(d.cfg, d.lay, x, w, y)
        G.epx.ep_expert_gemm_bwd_x(d.cfg, d.lay, gy, w, gx)
        G.epx.ep_expert_gemm_bwd_w(d.cfg, d.lay, gy, x, gw)
        return [v.view(torch.int16).cpu() for v in (y, yq, gx, gw)]

    for got, want in zip(run(*map(at_the_end, (x, gy, w, *q))), run(x, gy, w, *q)):
        assert torch.equal(got, want)
