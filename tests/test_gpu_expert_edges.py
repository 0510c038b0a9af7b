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


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("E,groups,top", [(64, 1, 1), (64, 8, 3), (96, 4, 2), (256, 8, 4)])
def test_softmax_over_a_nan_or_infinity_shows_in_the_weights(G, E, groups, top):  # noqa: F811
    """A token with a NaN or +infinity among its logits gets K experts, chosen by the
    logits with a bias too, and NaN for their weights: it is not left out."""
    T, K = 33, 6
    rng = np.random.default_rng(E)
    z = rng.standard_normal((T, E)).astype(np.float32)
    z[::3, 5] = np.nan
    z[1::3, 7] = np.inf
    cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K)
    logits, bias = torch.from_numpy(z).to("cuda:0"), normal(1, E, dtype=torch.float32)
    r = G.epx.RouteConfig(num_groups=groups, top_groups=top)
    seen = []
    for b in (bias, None):
        ids, p = torch.full((T, K), -7, dtype=torch.int32, device="cuda:0"), torch.zeros(T, K, device="cuda:0")
        G.epx.ep_route(cfg, r, logits, ids, p, bias=b)
        seen.append((ids.cpu().numpy(), p.cpu().numpy()))
    off = np.arange(T) % 3 < 2
    for ids, p in seen:
        assert ((ids >= 0) & (ids < E)).all()
        assert np.isnan(p[off]).all() and np.isfinite(p[~off]).all()
        assert (ids[1::3, 0] == 7).all() and not (ids[::3] == 5).any()
    np.testing.assert_array_equal(seen[0][0][off], seen[1][0][off])
    assert (seen[0][0][~off] != seen[1][0][~off]).any()


def test_gate_of_a_slice_that_begins_off_16_bytes(G):  # noqa: F811
    """A batch's logits from its second token on, 37 experts wide: the results and
    gradients of an aligned copy."""
    from combine_ep_dispatch_amd.autograd import EpDispatcher

    T, E, K = 9, 37, 3
    d = EpDispatcher(G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K), "cuda:0")
    for dtype in (torch.float32, torch.bfloat16):
        batch, g = normal(1, T + 1, E, dtype=dtype), normal(2, T, K, dtype=torch.float32)
        slices = [batch.clone().requires_grad_(), batch[1:].clone().requires_grad_()]
        assert slices[0][1:].data_ptr() % 16 != 0
        out = []
        for z, leaf in ((slices[0][1:], slices[0]), (slices[1], slices[1])):
            ids, p = d.gate(z, G.epx.RouteConfig())
            p.backward(g)
            out.append((ids, p.detach(), leaf.grad[-T:]))
        for a, b in zip(*out):
            assert torch.equal(a, b)
