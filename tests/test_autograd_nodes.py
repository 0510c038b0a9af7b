"""The autograd nodes of EpDispatcher without a GPU: their library calls are
replaced by plain CPU forms, so that what is tested is the marshalling."""

import pytest
import torch

import combine_ep_dispatch_amd as epx
from combine_ep_dispatch_amd import autograd as ag

T, H, E, K, INTER = 3, 8, 2, 1, 8


@pytest.fixture
def plain(monkeypatch):
    """CPU forms of the calls for one expert a token, token t in row t, expert 0."""
    calls = {}

    def put(name, f):
        monkeypatch.setattr(ag, name, lambda *a, **kw: calls.setdefault(name, []).append((a, kw)) or f(*a, **kw))

    def route(cfg, r, logits, ids, probs, bias=None, token_mask=None):
        ids.zero_()
        probs.copy_(torch.sigmoid(logits[:, :1]))

    def route_bwd(cfg, r, logits, ids, g, out):
        s = torch.sigmoid(logits[:, :1])
        out.zero_()[:, :1] = g * s * (1 - s)

    def swiglu(cfg, lay, h, p, act):
        a, b = h.float().chunk(2, 1)
        act.copy_(p * a * torch.sigmoid(a) * b)

    def swiglu_bwd(cfg, lay, h, p, ga, gh, gp):
        a, b = h.float().chunk(2, 1)
        s = torch.sigmoid(a)
        gh.copy_(torch.cat([p * ga * b * s * (1 + a * (1 - s)), p * ga * a * s], 1))
        if gp is not None:
            gp.copy_((ga * a * s * b).sum(1, keepdim=True))

    put("ep_route", route)
    put("ep_route_bwd", route_bwd)
    put("ep_swiglu", swiglu)
    put("ep_swiglu_bwd", swiglu_bwd)
    put("ep_expert_gemm", lambda cfg, lay, x, w, y: y.copy_(x @ w[0].t()))
    put("ep_expert_gemm_bwd_x", lambda cfg, lay, gy, w, gx: gx.copy_(gy @ w[0]))
    put("ep_expert_gemm_bwd_w", lambda cfg, lay, gy, x, gw: gw.zero_()[0].copy_(gy.t() @ x))
    put("ep_dispatch", lambda cfg, lay, x, recv: recv.copy_(x))
    put("ep_dispatch_bwd", lambda cfg, lay, g, gx: gx.copy_(g))
    put("ep_combine", lambda cfg, lay, eo, p, y: y.copy_((eo.view(T, H) * p.view(T, 1)).view(-1)))
    put("ep_combine_bwd", lambda cfg, lay, gy, p, g: g.copy_((gy.view(T, H) * p.view(T, 1)).view(-1)))
    put("ep_combine_bwd_probs", lambda cfg, lay, gy, eo, gp: gp.copy_((gy * eo).view(T, H).sum(1)))
    return calls


def nodes():
    """name: (leaf, result of the leaf) of each autograd node."""
    gen = torch.Generator().manual_seed(1)
    cfg = epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=1, top_k=K, recv_rows=T)

    def leaf(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen).to(dtype).requires_grad_()

    logits, h, x, w = leaf(T, E, dtype=torch.float32), leaf(T, 2 * INTER), leaf(T, H), leaf(E, INTER, H)
    p = leaf(T, K, dtype=torch.float32)
    return {
        "gate": (logits, lambda: ag._Gate.apply(logits, None, None, cfg, epx.RouteConfig())[1]),
        "linear": (x, lambda: ag._Linear.apply(x, w, cfg, None)),
        "linear, weights": (w, lambda: ag._Linear.apply(x, w, cfg, None)),
        "swiglu": (h, lambda: ag._Swiglu.apply(h, p, cfg, None)),
        "swiglu, weights": (p, lambda: ag._Swiglu.apply(h, p, cfg, None)),
        "dispatch": (x, lambda: ag._Dispatch.apply(x, cfg, None)),
        "combine": (x, lambda: ag._Combine.apply(x, p, cfg, None)),
        "combine, weights": (p, lambda: ag._Combine.apply(x, p, cfg, None)),
    }


@pytest.mark.parametrize("name", list(nodes()))
def test_second_derivatives_are_refused(plain, name):
    """The backward calls have no gradients of their own: a gradient of a gradient
    is an error, not the derivative of the other terms alone."""
    leaf, result = nodes()[name]
    first, = torch.autograd.grad(result().float().square().sum() + leaf.float().square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated twice"):
        torch.autograd.grad(first.float().sum(), leaf)


@pytest.mark.parametrize("name", list(nodes()))
def test_first_derivatives_run_with_a_graph(plain, name):
    leaf, result = nodes()[name]
    once, = torch.autograd.grad(result().float().sum(), leaf)
    graph, = torch.autograd.grad(result().float().sum(), leaf, create_graph=True)
    assert torch.isfinite(once).all() and once.abs().max() > 0 and torch.equal(once, graph)


def dispatcher():
    d = object.__new__(ag.EpDispatcher)
    d.cfg = epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=1, top_k=K, recv_rows=T)
    d.layout, d.workspace, d.device = None, None, torch.device("cpu")
    return d


def test_strided_inputs(plain):
    """Inputs in another order than the calls take: the same results and first
    derivatives, and the second ones refused."""
    gen = torch.Generator().manual_seed(2)
    d = dispatcher()
    leaves = [torch.randn(*s, generator=gen).requires_grad_() for s in ((E, T), (2 * INTER, T), (H, T), (H, INTER, E), (K, T))]
    z, h, x, w, p = leaves
    turned = [z.t(), h.t().bfloat16(), x.t().bfloat16(), w.permute(2, 1, 0).bfloat16(), p.t().double()]
    outs = []
    for z, h, x, w, p in (turned, [v.contiguous() for v in turned]):
        out = [d.gate(z, epx.RouteConfig())[1], d.linear(x, w), d.swiglu(h, p), d.combine(x, p)]
        total = sum(v.float().square().sum() for v in out) + sum(v.square().sum() for v in leaves)
        first = torch.autograd.grad(total, leaves, create_graph=True)
        outs.append(out + list(first))
        for g, leaf in zip(first, leaves):
            with pytest.raises(RuntimeError, match="differentiated twice"):
                torch.autograd.grad(g.sum(), leaf, retain_graph=True)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_inputs_and_gradients_off_16_bytes(plain):
    """Contiguous slices that begin off 16 bytes, and gradients that arrive as such,
    reach the calls as aligned copies."""
    gen = torch.Generator().manual_seed(3)
    d = dispatcher()

    def flat(*shape, dtype=torch.bfloat16):  # the last values of a buffer one value longer
        t = torch.randn(torch.Size(shape).numel() + 1, generator=gen).to(dtype).requires_grad_()
        out = t[1:].view(*shape)
        assert out.is_contiguous() and out.data_ptr() % 16 != 0
        return out

    z, h, x, w = flat(T, E, dtype=torch.float32), flat(T, 2 * INTER), flat(T, H), flat(E, INTER, H)
    p = flat(T, K, dtype=torch.float32)
    outs = [d.gate(z, epx.RouteConfig())[1], d.linear(x, w), d.swiglu(h, p), d.combine(x, p), d.dispatch(x)]
    for out in outs:
        gy = torch.randn(out.numel() + 1, generator=gen).to(out.dtype)[1:].view(out.shape)
        assert gy.data_ptr() % 16 != 0
        out.backward(gy)
    needs = {"ep_route": (2,), "ep_route_bwd": (2, 5), "ep_swiglu": (2, 4), "ep_swiglu_bwd": (2, 4, 5), "ep_expert_gemm": (2, 3, 4),
             "ep_expert_gemm_bwd_x": (2, 3, 4), "ep_expert_gemm_bwd_w": (2, 3, 4), "ep_dispatch": (2, 3),
             "ep_dispatch_bwd": (2, 3), "ep_combine": (2, 4), "ep_combine_bwd": (2, 4), "ep_combine_bwd_probs": (2, 3)}
    assert set(plain) == set(needs)
    for name, at in needs.items():
        for args, _ in plain[name]:
            for i in at:
                assert args[i].is_contiguous() and args[i].data_ptr() % 16 == 0, (name, i)
