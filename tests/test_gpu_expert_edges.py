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


RANKED = [(64, 8, 3), (64, 64, 9), (128, 16, 4), (256, 8, 4), (256, 64, 20), (512, 8, 2), (2048, 64, 7)]


def close_groups(E, groups, top, T, size, rng):
    """Logits and bias of T tokens whose groups number top and top + 1 (and here and
    there the one after) have keys that tie, or differ by one ulp of one logit.
    Experts of a group lie far apart; size: of the scores, which the bias stays below."""
    per = E // groups
    lo = 0.0 if per == 1 else -1.5
    base = np.linspace(lo, 1.5, per, dtype=np.float32) if per > 1 else np.zeros(1, np.float32)
    bias = np.tile((rng.standard_normal(per) * 0.02 * size).astype(np.float32), groups)
    z = np.empty((T, groups, per), np.float32)
    for t in range(T):
        order = rng.permutation(groups)
        level = np.linspace(1.0, -1.0, groups, dtype=np.float32)  # of the groups, best first
        same = rng.integers(2, 4)
        for rank, g in enumerate(order):
            z[t, g] = base + (level[top - 1] if top - 1 <= rank < top - 1 + same else level[rank])
        kind = t % 4
        if kind:  # 0: a tie.  Otherwise one expert of one of the groups: the best, the second, or one that does not count
            g = order[top - 1 + rng.integers(0, same)] if top - 1 + same <= groups else order[top - 1]
            e = np.argsort(-z[t, g])[min(kind - 1, per - 1)]
            z[t, g, e] = np.nextafter(z[t, g, e], np.float32(np.inf if rng.random() < 0.5 else -np.inf))
    return z.reshape(T, E), bias


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,top", RANKED)
def test_groups_too_close_to_tell_in_32_bits(G, E, groups, top, score):  # noqa: F811
    """Which groups stay, and with them the ids, as 64-bit scores say: ties to the
    lower index, differences of one ulp of one logit.  The groups' keys are closer
    than fp32 can tell (a rounding of a key of about 1 is 2^-24), the experts' are not."""
    from test_gpu_expert_layer import plain_route

    T, K = 200, min(8, top * (E // groups))
    G.say(f"[gpu] close groups E={E} groups={groups} top={top} {score}")
    z, bias = close_groups(E, groups, top, T, 1.0 if score == "sigmoid" else 1.0 / E,
                           np.random.default_rng(E + groups))
    logits, b = torch.from_numpy(z).to("cuda:0"), torch.from_numpy(bias).to("cuda:0")
    s = 1 / (1 + np.exp(-z.astype(np.float64))) if score == "sigmoid" else np.exp(z.astype(np.float64))
    if score == "softmax":
        s = s / s.sum(1, keepdims=True)
    keys = np.sort((s + bias.astype(np.float64)).reshape(T, groups, -1), axis=2)
    of_group = np.sort(keys[..., -2:].sum(2), axis=1)[:, ::-1]
    gap = of_group[:, top - 1] - of_group[:, top]
    assert (gap < 2.0 ** -20).all() and (gap[::4] == 0).all() and (gap > 0).sum() > T // 8
    cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K)
    r = G.epx.RouteConfig(score=score, num_groups=groups, top_groups=top)
    ids, p = torch.empty(T, K, dtype=torch.int32, device="cuda:0"), torch.empty(T, K, device="cuda:0")
    G.epx.ep_route(cfg, r, logits, ids, p, bias=b)
    np.testing.assert_array_equal(ids.cpu().numpy(), plain_route(logits, b, None, K, r)[0])


# ---------------------------------------------------------------------------
# Streams
# ---------------------------------------------------------------------------
def test_different_calls_on_two_streams(G):  # noqa: F811
    """Every operator on two streams at once, each with its own layout, inputs and
    sizes (and so other tiles): each gives the bits that it gives alone."""
    def work(seed, name, n_in, n_out, T, E):
        d = Rows(G, name)
        x, gy, w = normal(seed, d.R, n_in), normal(seed + 1, d.R, n_out), normal(seed + 2, d.experts, n_out, n_in)
        q, _, _ = nvfp4_weights(seed, d.experts, n_out, n_in)
        h, ga = normal(seed + 3, d.R, 2 * n_out), normal(seed + 4, d.R, n_out)
        cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=4)
        r = G.epx.RouteConfig(score="sigmoid", num_groups=4, top_groups=2)
        z, bias, gp = (normal(seed + 5 + i, *s, dtype=torch.float32) for i, s in enumerate(((T, E), (E,), (T, 4))))
        e = G.epx

        def buffers():
            f32 = dict(dtype=torch.float32, device="cuda:0")
            return dict(y=filled(d.R, n_out), yq=filled(d.R, n_out), gx=filled(d.R, n_in), gw=filled(d.experts, n_out, n_in),
                        act=filled(d.R, n_out), gh=filled(d.R, 2 * n_out), gprobs=torch.zeros(d.T, d.K, **f32),
                        ids=torch.zeros(T, 4, dtype=torch.int32, device="cuda:0"), p=torch.zeros(T, 4, **f32),
                        gz=torch.zeros(T, E, **f32))

        def calls(b, st):
            return [
                lambda: e.ep_expert_gemm(d.cfg, d.lay, x, w, b["y"], stream=st),
                lambda: e.ep_route(cfg, r, z, b["ids"], b["p"], bias=bias, stream=st),
                lambda: e.ep_expert_gemm_nvfp4(d.cfg, d.lay, x, *q, b["yq"], stream=st),
                lambda: e.ep_swiglu(d.cfg, d.lay, h, d.probs, b["act"], stream=st),
                lambda: e.ep_expert_gemm_bwd_w(d.cfg, d.lay, gy, x, b["gw"], stream=st),
                lambda: e.ep_swiglu_bwd(d.cfg, d.lay, h, d.probs, ga, b["gh"], b["gprobs"], stream=st),
                lambda: e.ep_expert_gemm_bwd_x(d.cfg, d.lay, gy, w, b["gx"], stream=st),
                lambda: e.ep_route_bwd(cfg, r, z, b["ids"], gp, b["gz"], stream=st),
            ]

        return buffers, calls

    jobs = [work(1, "tall", 528, 1040, 700, 256), work(50, "odd", 272, 72, 129, 64)]
    want = []
    for buffers, calls in jobs:
        b = buffers()
        for call in calls(b, None):
            call()
        torch.cuda.synchronize()
        want.append(b)
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        got = [buffers() for buffers, _ in jobs]
        torch.cuda.synchronize()
        both = [calls(b, st) for (_, calls), b, st in zip(jobs, got, streams)]
        for pair in zip(both[0], both[1]):
            for call in pair:
                call()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for n in w:
                assert torch.equal(g[n].view(torch.uint8), w[n].view(torch.uint8)), n


def test_captured_training_step_replays_like_the_eager_one(G):  # noqa: F811
    """The layer through EpDispatcher, forward and gradients, captured into one
    graph: every replay gives the eager step's bits, with new inputs in between."""
    from combine_ep_dispatch_amd.autograd import EpDispatcher

    T, H, E, K, inter = 40, 64, 8, 2, 32
    shapes = dict(x=(T, H), logits=(T, E), w1=(E, 2 * inter, H), w2=(E, H, inter))
    gy = normal(9, T, H)

    def inputs(seed):
        return {n: normal(seed + i, *s, dtype=torch.float32 if n == "logits" else torch.bfloat16)
                for i, (n, s) in enumerate(shapes.items())}

    def step(d, t):
        ids, p = d.gate(t["logits"], G.epx.RouteConfig(score="sigmoid", num_groups=4, top_groups=2))
        y = d.combine(d.linear(d.swiglu(d.linear(d.dispatch(t["x"], ids), t["w1"]), p), t["w2"]), None)
        return [ids, y.detach(), *torch.autograd.grad(y, [t[n] for n in shapes], gy)]

    def dispatcher():
        return EpDispatcher(G.epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=2, top_k=K, align=8), "cuda:0")

    eager, d = dispatcher(), dispatcher()
    leaves = {n: v.requires_grad_() for n, v in inputs(1).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step(d, leaves)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d, leaves)
    for i in range(4):
        new = inputs(100 * i)
        with torch.no_grad():
            for n, v in new.items():
                leaves[n].copy_(v)
        want = step(eager, {n: v.requires_grad_() for n, v in new.items()})
        torch.cuda.synchronize()
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (i, k)
