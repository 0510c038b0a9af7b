"""The gated block (both projections, the activation and the routing weight in one
kernel, bf16 and 4-bit weights, with its backward pass) and the low-rank adapters
beside the experts' products, on the GPU against plain forms in 64 bits.

Tolerances: an output in bf16 is off by at most half a step, 2^-8 of its value, on
top of the fp32 error before it.  A sum of n products in fp32 is off by at most n +
1 roundings (2^-24) of the sum of the terms' magnitudes.  The products take u as two
bf16, the second of what the first left: off by at most 2^-8 of 2^-8, 2^-16 of its
value; the adapters' gradients as three, off by 2^-24.
Rows that no slot owns have to stay as they were.
"""

import pytest
import torch

from test_gpu_expert_edges import at_the_end
from test_gpu_expert_layer import (FILL, HALF_BF16, LAYOUTS, MANY, U32, G, Rows, check, expert_sums,  # noqa: F401
                                   filled, normal, nvfp4_weights, rounded)

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -127  # where exp(-g) passes the largest float (g < -88.7) s is 0 instead of less than 2^-127


def spoiled(d, t):
    """t with NaN in the rows that no slot owns: they are never read."""
    nan = torch.zeros(d.R, 1, dtype=torch.bfloat16)
    nan[~d.kept] = float("nan")
    return t + nan.to(t)


def words(rows, rank):
    """A buffer for u or grad_u that marks untouched rows."""
    return torch.full((rows, 2 * rank), FILL, dtype=torch.int16, device="cuda:0").view(torch.float32)


class Lora:
    """Adapters of a layout's tokens and what the plain form needs of them."""

    def __init__(self, G, d, rank, n_in, n_out, n=3, scaled=True, seed=40):
        gen = torch.Generator().manual_seed(seed)
        ids = torch.randint(-1, n, (d.T,), generator=gen, dtype=torch.int32)
        ids[3::11] = n + 5  # outside: none, as -1
        ids[4::13] = -7
        self.n, self.rank = n, rank
        self.a, self.b = normal(seed, n, d.experts, rank, n_in, std=n_in ** -0.5), normal(seed + 1, n, d.experts, n_out, rank)
        self.scale = (0.5 + torch.rand(n, generator=gen)).cuda() if scaled else None
        self.c = G.epx.Adapters(ids.cuda(), self.a, self.b, self.scale)
        self.s = (self.scale if scaled else torch.ones(n)).double().cpu()
        token = d.slots // d.cfg.kp
        of = ids.long()[token]
        self.of = torch.where((of >= 0) & (of < n), of, -1)  # of d.rows

    def each(self, on):
        """(adapter, positions in on) of the rows `on` of one expert."""
        for k in range(self.n):
            some = (self.of[on] == k).nonzero().view(-1)
            if len(some):
                yield k, some


def u_of(x, a, s, taken=2.0 ** -24):
    """u of rows x and its error, as taken: in 32 bits, or as two bf16 (2^-16)."""
    u = s * (x @ a.T)
    return u, s * (x.abs() @ a.abs().T) * (x.shape[1] + 4) * U32 + u.abs() * taken + 2.0 ** -130


def add_lora(lora, e, on, x, want, err):
    """want += B u over the rows of expert e, err along."""
    for k, some in lora.each(on):
        a, b = lora.a[k, e].double().cpu(), lora.b[k, e].double().cpu()
        u, eu = u_of(x[some], a, lora.s[k], 2.0 ** -16)
        want[some] += u @ b.T
        err[some] += eu @ b.abs().T + (u.abs() + eu) @ b.abs().T * (2 * lora.rank + 2) * U32


def check_u(lora, d, x, weights, got, what):
    g = got.double().cpu()
    for e in range(d.experts):
        on = (d.expert == e).nonzero().view(-1)
        want, err = torch.zeros(len(on), lora.rank, dtype=torch.float64), torch.zeros(len(on), lora.rank, dtype=torch.float64)
        for k, some in lora.each(on):
            want[some], err[some] = u_of(x[d.rows[on][some]], weights(k, e), lora.s[k])
        check(g[d.rows[on]], want, err, f"{what}, expert {e}")
    d.untouched(got.view(torch.bfloat16))


def silu_parts(g):
    s = torch.sigmoid(g)
    return s, g * s


def check_gated(d, n_in, inter, weights, x, probs, act, lora=None, grads=None, scale=None):
    """act (and the backward pass's results, in grads) against the definition."""
    w = (d.w if probs is not None else torch.ones_like(d.w))[:, None]
    xc, actc = x.double().cpu(), act.cpu()
    if grads is not None:
        gac, ghc = grads["grad_act"].double().cpu(), grads["grad_h"].cpu()
        gp, gpe = torch.zeros(d.T * d.cfg.kp, dtype=torch.float64), torch.zeros(d.T * d.cfg.kp, dtype=torch.float64)

    def one(e, on, rows):
        m = weights(e)
        h, err = xc[rows] @ m.T, xc[rows].abs() @ m.abs().T * (n_in + 2) * U32
        if scale is not None:
            h, err = h * scale[e], err * scale[e]
        if lora is not None:
            add_lora(lora, e, on, xc[rows], h, err)
            err += h.abs() * 2 * U32
        (g, u), (eg, eu) = h.split(inter, 1), err.split(inter, 1)
        s, silu = silu_parts(g)
        p = w[on]
        # |silu'| <= 1.1 and |silu''| <= 0.5; the sigmoid's own error counts |g| and a
        # few roundings, the products a few more
        own = (24 + g.abs()) * U32
        want = p * silu * u
        e_act = p * (1.1 * eg * (u.abs() + eu) + silu.abs() * eu) + want.abs() * own + (p * g * u).abs() * TINY + TINY
        check(actc[rows], want, rounded(want, e_act), f"act, expert {e}")
        if grads is None:
            return
        ga = gac[rows]
        slope = s * (1 + g * torch.sigmoid(-g))
        want = torch.cat([p * ga * u * slope, p * ga * silu], 1)
        gabs = (p * ga).abs()
        size = torch.cat([gabs * u.abs() * (1 + g.abs()), gabs * g.abs()], 1)
        ss = torch.cat([s, s], 1)
        e_h = torch.cat([gabs * (1.1 * eu + (u.abs() + eu) * 0.5 * eg), gabs * 1.1 * eg], 1)
        e_h = e_h + size * (ss * (32 + torch.cat([g, g], 1).abs()) * U32 + TINY) + TINY
        check(ghc[rows], want, rounded(want, e_h), f"grad_h, expert {e}")
        gp[d.slots[on]] = (ga * silu * u).sum(1)
        terms = ga.abs() * (1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (silu * u).abs() * (own + inter * U32) +
                            (g * u).abs() * TINY)
        gpe[d.slots[on]] = terms.sum(1) + TINY

    expert_sums(d, one)
    d.untouched(act)
    if grads is not None:
        d.untouched(grads["grad_h"])
        want, err = (v.view(d.T, d.cfg.kp)[:, : d.K] for v in (gp, gpe))
        check(grads["grad_probs"], want, err, "grad_probs")


# ---------------------------------------------------------------------------
# The gated block
# ---------------------------------------------------------------------------
# (in, inter): the smallest, odd, past one tile each way, wide and flat
DIMS = [(8, 8), (40, 136), (136, 72), (264, 264), (1416, 24)]


def few(name, n_in, n_out, step=8):
    """Smaller widths where 2000 experts' weights would be large."""
    if name == "many-groups" and n_in * n_out > 10000:
        return n_in // 16 // step * step + step, n_out // 16 // 8 * 8 + 8
    return n_in, n_out


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("rank", [0, 8, 24])
def test_gated_forward_and_backward(G, name, dims, rank):  # noqa: F811
    n_in, inter = few(name, *dims)
    G.say(f"[gpu] gated {name} in={n_in} inter={inter} rank={rank}")
    d = Rows(G, name)
    x, ga = spoiled(d, normal(1, d.R, n_in)), spoiled(d, normal(2, d.R, inter))
    w = normal(3, d.experts, 2 * inter, n_in, std=2.0 * n_in ** -0.5)
    probs = None if rank == 8 else d.probs
    lora, kw = None, {}
    if rank:
        lora = Lora(G, d, rank, n_in, 2 * inter, scaled=rank != 8)
        kw = dict(adapters=lora.c, u=words(d.R, rank))
        G.epx.ep_lora_down(d.cfg, d.lay, x, lora.c, kw["u"])
        check_u(lora, d, x.double().cpu(), lambda k, e: lora.a[k, e].double().cpu(), kw["u"], "u")
    act, act2 = filled(d.R, inter), filled(d.R, inter)
    grads = dict(grad_act=ga, grad_h=filled(d.R, 2 * inter),
                 grad_probs=torch.full((d.T, d.K), float("nan"), device="cuda:0"))
    ws = G.epx.gated_workspace_for(d.cfg, inter, "cuda:0").fill_(0xFF)
    G.epx.ep_expert_gated(d.cfg, d.lay, x, w, probs, act, **kw)
    G.epx.ep_expert_gated_bwd(d.cfg, d.lay, x, w, probs, ga, grads["grad_h"], act=act2, grad_probs=grads["grad_probs"],
                              workspace=ws, **kw)
    check_gated(d, n_in, inter, lambda e: w[e].double().cpu(), x, probs, act, lora, grads)
    assert torch.equal(act2.view(torch.int16), act.view(torch.int16))
    # without act and the weights' gradient: the same grad_h
    gh = filled(d.R, 2 * inter)
    G.epx.ep_expert_gated_bwd(d.cfg, d.lay, x, w, probs, ga, gh, **kw)
    assert torch.equal(gh.view(torch.int16), grads["grad_h"].view(torch.int16))


@pytest.mark.parametrize("name", MANY)
@pytest.mark.parametrize("rank", [0, 128])
def test_gated_of_many_rows(G, name, rank):  # noqa: F811
    test_gated_forward_and_backward(G, name, (328, 312), rank)


def test_gated_of_large_values(G):  # noqa: F811
    """Gates where exp(-g) underflows and overflows, of either sign."""
    d = Rows(G, "odd")
    x, ga = normal(1, d.R, 64), normal(2, d.R, 40)
    w = normal(3, d.experts, 80, 64, std=8.0)  # |g| up to 250
    act, gh, gp = filled(d.R, 40), filled(d.R, 80), torch.empty(d.T, d.K, device="cuda:0")
    G.epx.ep_expert_gated(d.cfg, d.lay, x, w, d.probs, act)
    G.epx.ep_expert_gated_bwd(d.cfg, d.lay, x, w, d.probs, ga, gh, grad_probs=gp,
                              workspace=G.epx.gated_workspace_for(d.cfg, 40, "cuda:0"))
    check_gated(d, 64, 40, lambda e: w[e].double().cpu(), x, d.probs, act, None,
                dict(grad_act=ga, grad_h=gh, grad_probs=gp))


def test_gated_gradient_against_differences(G):  # noqa: F811
    """grad_h taken through the weights, and grad_probs, against central differences
    of the definition in 64 bits (step 1e-4: 1e-8 of truncation; grad_h is off by
    2^-8 of its value, and the sums over it by that of their terms' magnitudes)."""
    d = Rows(G, "odd")
    n_in, inter = 16, 8
    x, ga, w = normal(1, d.R, n_in), normal(2, d.R, inter), normal(3, d.experts, 2 * inter, n_in, std=0.3)
    gh, gp, gx = filled(d.R, 2 * inter), torch.empty(d.T, d.K, device="cuda:0"), filled(d.R, n_in)
    G.epx.ep_expert_gated_bwd(d.cfg, d.lay, x, w, d.probs, ga, gh, grad_probs=gp,
                              workspace=G.epx.gated_workspace_for(d.cfg, inter, "cuda:0"))
    G.epx.ep_expert_gemm_bwd_x(d.cfg, d.lay, gh, w, gx)
    m = w.double().cpu()[d.expert]
    xr, g, p = x.cpu()[d.rows].double(), ga.cpu()[d.rows].double(), d.w[:, None]

    def loss(x, p):
        a, b = torch.einsum("rh,rnh->rn", x, m).split(inter, 1)
        return (p * a * torch.sigmoid(a) * b * g).sum(1)

    got, size = gx.cpu()[d.rows].double(), (gh.cpu()[d.rows].double().abs()[:, :, None] * m.abs()).sum(1)
    for j in range(n_in):
        e = torch.zeros_like(xr)
        e[:, j] = 1e-4
        slope = (loss(xr + e, p) - loss(xr - e, p)) / 2e-4
        assert ((got[:, j] - slope).abs() <= (slope.abs() + size[:, j]) * HALF_BF16 * 1.01 + 1e-5).all()
    slope = (loss(xr, p + 1e-4) - loss(xr, p - 1e-4)) / 2e-4
    full = torch.zeros(d.T * d.cfg.kp, dtype=torch.float64)
    full[d.slots] = slope
    assert ((gp.cpu().double() - full.view(d.T, -1)[:, : d.K]).abs() <= 1e-5).all()


NV_DIMS = [(16, 8), (48, 136), (64, 72), (272, 40), (320, 136), (1040, 72), (1152, 264)]


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("dims", NV_DIMS, ids=str)
@pytest.mark.parametrize("rank", [0, 16, 40])
def test_gated_nvfp4(G, name, dims, rank):  # noqa: F811
    n_in, inter = few(name, *dims, step=16)
    G.say(f"[gpu] gated_nvfp4 {name} in={n_in} inter={inter} rank={rank}")
    d = Rows(G, name)
    x = spoiled(d, normal(1, d.R, n_in))
    q, w, rs = nvfp4_weights(5, d.experts, 2 * inter, n_in)
    q[2] = (q[2].float() * 2.0 ** -4).to(torch.bfloat16)  # gates of a few units
    rs = q[2].double().cpu()
    lora, kw = None, {}
    if rank:
        lora = Lora(G, d, rank, n_in, 2 * inter, n=20)
        kw = dict(adapters=lora.c, u=words(d.R, rank))
        G.epx.ep_lora_down(d.cfg, d.lay, x, lora.c, kw["u"])
    act = filled(d.R, inter)
    probs = d.probs if rank != 16 else None
    G.epx.ep_expert_gated_nvfp4(d.cfg, d.lay, x, *q, probs, act, **kw)
    check_gated(d, n_in, inter, lambda e: w[e], x, probs, act, lora, scale=rs)


# ---------------------------------------------------------------------------
# Adapters beside the products
# ---------------------------------------------------------------------------
LORA_DIMS = [(8, 8, 8), (136, 72, 16), (40, 264, 24), (264, 520, 64), (1416, 88, 128)]


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("dims", LORA_DIMS, ids=str)
def test_adapters_and_gradients(G, name, dims):  # noqa: F811
    n_in, n_out, rank = dims
    if name == "many-groups":
        (n_in, n_out), rank = few(name, n_in, n_out), min(rank, 16)
    G.say(f"[gpu] adapters {name} in={n_in} out={n_out} rank={rank}")
    d = Rows(G, name)
    x, gy = spoiled(d, normal(1, d.R, n_in)), spoiled(d, normal(2, d.R, n_out))
    w = normal(3, d.experts, n_out, n_in)
    lora = Lora(G, d, rank, n_in, n_out, n=2 if name == "many-groups" else 5)
    u, gu = words(d.R, rank), words(d.R, rank)
    y, gx = filled(d.R, n_out), filled(d.R, n_in)
    G.epx.ep_lora_down(d.cfg, d.lay, x, lora.c, u)
    G.epx.ep_expert_gemm_lora(d.cfg, d.lay, x, w, y, lora.c, u)
    G.epx.ep_lora_bwd_u(d.cfg, d.lay, gy, lora.c, gu)
    G.epx.ep_expert_gemm_bwd_x_lora(d.cfg, d.lay, gy, w, gx, lora.c, gu)
    ga, gb = torch.full_like(lora.a, float("nan")), torch.full_like(lora.b, float("nan"))
    G.epx.ep_lora_bwd_w(d.cfg, d.lay, x, gy, lora.c, u, gu, ga, gb)
    ga32, gb32 = (torch.full(t.shape, float("nan"), device="cuda:0") for t in (lora.a, lora.b))
    G.epx.ep_lora_bwd_w(d.cfg, d.lay, x, gy, lora.c, u, gu, ga32, gb32)
    acc = [torch.full_like(t, 0.5) for t in (ga32, gb32)]
    G.epx.ep_lora_bwd_w(d.cfg, d.lay, x, gy, lora.c, u, gu, *acc, accumulate=True)
    for t, of in zip(acc, (ga32, gb32)):
        assert torch.equal(t, of + 0.5)
    for t, of in zip((ga, gb), (ga32, gb32)):
        assert torch.equal(t, of.to(torch.bfloat16))
    xc, gc, ga32, gb32 = x.double().cpu(), gy.double().cpu(), ga32.cpu(), gb32.cpu()
    check_u(lora, d, xc, lambda k, e: lora.a[k, e].double().cpu(), u, "u")
    check_u(lora, d, gc, lambda k, e: lora.b[k, e].double().cpu().T, gu, "grad_u")
    yc, gxc = y.cpu(), gx.cpu()
    seen = torch.zeros(lora.n, d.experts, dtype=torch.bool)

    def one(e, on, rows):
        m = w[e].double().cpu()
        want, err = xc[rows] @ m.T, xc[rows].abs() @ m.abs().T * (n_in + 1) * U32
        add_lora(lora, e, on, xc[rows], want, err)
        check(yc[rows], want, rounded(want, err + want.abs() * U32), f"y, expert {e}")
        want, err = gc[rows] @ m, gc[rows].abs() @ m.abs() * (n_out + 1) * U32
        for k, some in lora.each(on):
            seen[k, e] = True
            a, b = lora.a[k, e].double().cpu(), lora.b[k, e].double().cpu()
            xs, gs = xc[rows[some]], gc[rows[some]]
            (us, eu), (vs, ev) = u_of(xs, a, lora.s[k]), u_of(gs, b.T, lora.s[k])
            want[some] += vs @ a
            e2 = ev + vs.abs() * 2.0 ** -16
            err[some] += e2 @ a.abs() + (vs.abs() + e2) @ a.abs() * (2 * rank + 2) * U32
            n = 3 * len(some) + 2
            check(ga32[k, e], vs.T @ xs, (ev.T + (vs.abs() + ev).T * n * U32) @ xs.abs(), f"grad_a {k}, expert {e}")
            check(gb32[k, e], gs.T @ us, gs.abs().T @ (eu + (us.abs() + eu) * n * U32), f"grad_b {k}, expert {e}")
        check(gxc[rows], want, rounded(want, err + want.abs() * U32), f"grad_x, expert {e}")

    expert_sums(d, one)
    assert (ga32[~seen] == 0).all() and (gb32[~seen] == 0).all()
    d.untouched(y)
    d.untouched(gx)


@pytest.mark.parametrize("name", MANY)
def test_adapters_and_gradients_of_many_rows(G, name):  # noqa: F811
    test_adapters_and_gradients(G, name, (520, 328, 32))


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("dims", [(16, 8, 8), (48, 264, 16), (320, 136, 40), (1040, 72, 128)], ids=str)
def test_adapters_nvfp4(G, name, dims):  # noqa: F811
    n_in, n_out, rank = dims
    n_in, n_out = few(name, n_in, n_out, step=16)
    G.say(f"[gpu] adapters_nvfp4 {name} in={n_in} out={n_out} rank={rank}")
    d = Rows(G, name)
    x = spoiled(d, normal(1, d.R, n_in))
    q, w, rs = nvfp4_weights(5, d.experts, n_out, n_in)
    lora, u, y = Lora(G, d, rank, n_in, n_out, n=3), words(d.R, rank), filled(d.R, n_out)
    G.epx.ep_lora_down(d.cfg, d.lay, x, lora.c, u)
    G.epx.ep_expert_gemm_nvfp4_lora(d.cfg, d.lay, x, *q, y, lora.c, u)
    xc, yc = x.double().cpu(), y.cpu()

    def one(e, on, rows):
        want, err = xc[rows] @ w[e].T * rs[e], xc[rows].abs() @ w[e].abs().T * rs[e] * (n_in + 3) * U32
        add_lora(lora, e, on, xc[rows], want, err)
        check(yc[rows], want, rounded(want, err + want.abs() * U32), f"expert {e}")

    expert_sums(d, one)
    d.untouched(y)


def test_no_adapters_is_the_product_itself(G):  # noqa: F811
    """Tokens without adapters: the plain product's bits, u zero."""
    d = Rows(G, "tall")
    x, w = normal(1, d.R, 264), normal(3, d.experts, 136, 264)
    lora, u = Lora(G, d, 16, 264, 136), words(d.R, 16)
    lora.c.token_adapter.fill_(-1)
    G.epx.ep_lora_down(d.cfg, d.lay, x, lora.c, u)
    want, y = filled(d.R, 136), filled(d.R, 136)
    G.epx.ep_expert_gemm(d.cfg, d.lay, x, w, want)
    G.epx.ep_expert_gemm_lora(d.cfg, d.lay, x, w, y, lora.c, u)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    assert (u.cpu()[d.rows] == 0).all()


# ---------------------------------------------------------------------------
# Rows apart from each other
# ---------------------------------------------------------------------------
def block_calls(G, d, x, ga, w, q, lora, rank, inter):  # noqa: F811
    """Every row output of the block's calls, by name."""
    e, out = G.epx, {}
    u = words(d.R, rank)
    n_in, n_out = x.shape[1], 2 * inter
    e.ep_lora_down(d.cfg, d.lay, x, lora.c, u)
    for k, n in (("act", inter), ("actq", inter), ("actl", inter), ("actql", inter), ("gh", n_out), ("ghl", n_out),
                 ("y", n_out), ("yq", n_out), ("gx", n_in)):
        out[k] = filled(d.R, n)
    e.ep_expert_gated(d.cfg, d.lay, x, w, d.probs, out["act"])
    e.ep_expert_gated_nvfp4(d.cfg, d.lay, x, *q, d.probs, out["actq"])
    e.ep_expert_gated(d.cfg, d.lay, x, w, d.probs, out["actl"], lora.c, u)
    e.ep_expert_gated_nvfp4(d.cfg, d.lay, x, *q, d.probs, out["actql"], lora.c, u)
    e.ep_expert_gated_bwd(d.cfg, d.lay, x, w, d.probs, ga, out["gh"])
    e.ep_expert_gated_bwd(d.cfg, d.lay, x, w, d.probs, ga, out["ghl"], adapters=lora.c, u=u)
    e.ep_expert_gemm_lora(d.cfg, d.lay, x, w, out["y"], lora.c, u)
    e.ep_expert_gemm_nvfp4_lora(d.cfg, d.lay, x, *q, out["yq"], lora.c, u)
    gu = words(d.R, rank)
    gh = out["ghl"].clone()
    gh.view(torch.int16)[~d.kept.to(gh.device)] = 0
    e.ep_lora_bwd_u(d.cfg, d.lay, gh, lora.c, gu)
    e.ep_expert_gemm_bwd_x_lora(d.cfg, d.lay, gh, w, out["gx"], lora.c, gu)
    out["u"], out["gu"] = u.view(torch.bfloat16), gu.view(torch.bfloat16)
    return {k: v.view(torch.int16).cpu() for k, v in out.items()}


def block_inputs(G, d, n_in, inter, rank, n=3):  # noqa: F811
    q, _, _ = nvfp4_weights(5, d.experts, 2 * inter, n_in)
    return [normal(1, d.R, n_in), normal(2, d.R, inter), normal(3, d.experts, 2 * inter, n_in, std=n_in ** -0.5), q,
            Lora(G, d, rank, n_in, 2 * inter, n=n), rank, inter]


@pytest.mark.parametrize("name", ["aligned", "tall"])
@pytest.mark.parametrize("rank", [8, 32])
def test_infinities_and_nan_stay_where_they_are(G, name, rank):  # noqa: F811
    """Rows with an infinity or NaN, and an adapter full of them, spoil the rows
    that hold or use them and no other."""
    d = Rows(G, name)
    t = block_inputs(G, d, 64, 72, rank)
    clean = block_calls(G, d, *t)
    lora, bad = t[4], d.rows[::7]
    t[0][bad.cuda()[::2], 3] = float("inf")
    t[0][bad.cuda()[1::2], 60] = float("nan")
    of = lora.of == 1
    lora.a[1, :, 5] = float("nan")
    lora.b[1, ::2] = float("nan")
    lora.b[1, 1::2] = float("inf")
    got = block_calls(G, d, *t)
    keep = torch.ones(d.R, dtype=torch.bool)
    keep[bad] = False
    uses = keep.clone()
    uses[d.rows[of]] = False
    assert uses[d.rows].any() and not uses[d.rows].all()
    for k, v in got.items():
        rows = keep if k in ("act", "actq", "gh") else uses
        assert torch.equal(v[rows], clean[k][rows]), k
    spoiled_rows = torch.cat([bad, d.rows[of]])
    assert not torch.isfinite(got["y"].view(torch.bfloat16)[spoiled_rows].float()).all(1).any()


@pytest.mark.parametrize("rank", [16, 72])
def test_a_rows_results_do_not_depend_on_the_batch(G, rank):  # noqa: F811
    """The same row alone, among few and among many rows of its expert (other tile
    sizes), of the same and of other adapters: the same bits."""
    n_in, inter, n = 448, 136, 4
    x1, w = normal(1, 1, n_in), normal(3, 1, 2 * inter, n_in, std=n_in ** -0.5)
    q, _, _ = nvfp4_weights(5, 1, 2 * inter, n_in)
    a, b = normal(6, n, 1, rank, n_in, std=n_in ** -0.5), normal(7, n, 1, 2 * inter, rank)
    ga1 = normal(8, 1, inter)
    seen = []
    for E, T in ((1, 1), (1, 20), (1, 40), (1, 100), (1, 200), (1, 700), (1, 9000), (160, 1600)):
        cfg = G.epx.EpConfig(num_tokens=T, hidden=16, num_experts=E, num_segments=1, top_k=1)
        cfg.recv_rows = G.epx.ep_query(cfg).min_recv_rows
        lay = G.epx.Layout.empty(cfg, "cuda:0")
        ids = torch.arange(T, dtype=torch.int32, device="cuda:0") % E
        G.epx.ep_dispatch_layout(cfg, ids, G.epx.workspace_for(cfg, "cuda:0"), lay)
        at = lay.token_row.view(-1)[T // 2].item()
        of = torch.randint(-1, n, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
        of[T // 2] = 2
        probs = torch.rand(T, 1, generator=torch.Generator().manual_seed(T)).cuda()
        probs[T // 2] = 0.375
        many = lambda t, dim: t.repeat(*[E if k == dim else 1 for k in range(t.dim())]).contiguous()  # noqa: E731

        class d:  # what block_calls reads of a layout
            R, kept = T, torch.ones(T, dtype=torch.bool)

        class lora:
            c = G.epx.Adapters(of.cuda(), many(a, 1), many(b, 1))

        d.cfg, d.lay, d.probs = cfg, lay, probs
        x, ga = normal(T, T, n_in), normal(T + 1, T, inter)
        x[at], ga[at] = x1[0], ga1[0]
        out = block_calls(G, d, x, ga, many(w, 0), [many(v, 0) for v in q], lora, rank, inter)
        seen.append({k: v[at] for k, v in out.items()})
    for other in seen[1:]:
        for k, v in other.items():
            assert torch.equal(seen[0][k], v), k


def test_pad_rows_are_zeroed_on_request(G):  # noqa: F811
    d = Rows(G, "aligned", flags=G.epx.EP_ZERO_PAD_ROWS)
    pad = d.pad_rows()
    assert pad.any()
    for k, v in block_calls(G, d, *block_inputs(G, d, 64, 40, 8)).items():
        if k != "gx":  # its input's pad rows were cleared by hand
            d.untouched(v.view(torch.bfloat16), zeroed=pad)


@pytest.mark.parametrize("n_in", [16, 48, 272, 320, 528, 1040])
@pytest.mark.parametrize("name", ["one", "odd", "aligned", "twenty", "tall"])
def test_operands_that_end_with_their_memory(G, name, n_in):  # noqa: F811
    """Every operand in the last bytes of its allocation: the bits of the same call on
    operands with memory behind them."""
    G.say(f"[gpu] ends of memory {name} in={n_in}")
    d = Rows(G, name)
    x, ga, w, q, lora, rank, inter = block_inputs(G, d, n_in, 40, 24)
    want = block_calls(G, d, x, ga, w, q, lora, rank, inter)
    lora.c = G.epx.Adapters(*map(at_the_end, (lora.c.token_adapter, lora.a, lora.b, lora.scale)))
    got = block_calls(G, d, *map(at_the_end, (x, ga, w)), list(map(at_the_end, q)), lora, rank, inter)
    for k, v in got.items():
        assert torch.equal(v, want[k]), k


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def lora_leaves(n, experts, rank, n_in, n_out, T, seed):
    gen = torch.Generator().manual_seed(seed)
    of = torch.randint(-1, n, (T,), generator=gen, dtype=torch.int32).cuda()
    return dict(a=normal(seed, n, experts, rank, n_in, std=n_in ** -0.5).requires_grad_(),
                b=normal(seed + 1, n, experts, n_out, rank, std=0.5 * rank ** -0.5).requires_grad_(), of=of,
                scale=(0.5 + torch.rand(n, generator=gen)).cuda())


def dense_lora(x, w, l, refs, e):
    """x @ (w[e] + scale b a)^T of every token's adapter, in 64 bits."""
    out = x @ w[e].T
    for k in range(refs["a"].shape[0]):
        on = (l["of"].cpu() == k).double()[:, None]
        out = out + on * l["scale"][k].double().cpu() * ((x @ refs["a"][k, e].T) @ refs["b"][k, e].T)
    return out


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("rank", [0, 8])
def test_layer_forward_and_backward(G, shared, rank):  # noqa: F811
    """The layer with the gated block (and adapters beside both products) through
    EpDispatcher against a dense form in 64 bits.  Forward the layer rounds to bf16
    after three row operations, each at most 2^-8 of the value: results differ by at
    most 3 * 2^-8 = 0.012 of their norm; gradients, up to six such roundings on the
    way, by 6 * 2^-8 = 0.024."""
    from combine_ep_dispatch_amd.autograd import EpDispatcher

    T, H, E, K, inter = 65, 72, 8, 3, 40
    x, logits, gy = normal(1, T, H).requires_grad_(), normal(2, T, E, dtype=torch.float32).requires_grad_(), normal(5, T, H)
    w1 = normal(3, E + shared, 2 * inter, H, std=H ** -0.5).requires_grad_()
    w2 = normal(4, E + shared, H, inter, std=inter ** -0.5).requires_grad_()
    cfg = G.epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=2, top_k=K, align=16,
                         shared_expert=shared, src_segment=1 if shared else 0)
    leaves, l1, l2, ad1, ad2 = dict(x=x, logits=logits, w1=w1, w2=w2), None, None, None, None
    if rank:
        l1, l2 = (lora_leaves(3, E + shared, rank, *dims, T, seed) for dims, seed in (((H, 2 * inter), 60), ((inter, H), 70)))
        l2["of"] = l1["of"]
        ad1, ad2 = (G.epx.Adapters(l["of"], l["a"], l["b"], l["scale"]) for l in (l1, l2))
        leaves |= dict(a1=l1["a"], b1=l1["b"], a2=l2["a"], b2=l2["b"])
    d = EpDispatcher(cfg, "cuda:0")
    ids, probs = d.gate(logits, G.epx.RouteConfig(score="sigmoid", scale=1.5))
    act = d.gated(d.dispatch(x, ids), w1, probs, ad1)
    y = d.combine(d.linear(act, w2, ad2), None)
    y.backward(gy)

    ref = {n: v.detach().double().cpu().requires_grad_() for n, v in leaves.items()}
    s = torch.sigmoid(ref["logits"]).gather(1, ids.long().cpu())
    p = torch.zeros(T, E + shared, dtype=torch.float64).scatter(1, ids.long().cpu(), 1.5 * s / s.sum(1, keepdim=True))
    if shared:
        p[:, E] = 1.0
    want = 0
    for e in range(E + shared):
        if rank:
            h = dense_lora(ref["x"], ref["w1"], l1, dict(a=ref["a1"], b=ref["b1"]), e)
        else:
            h = ref["x"] @ ref["w1"][e].T
        g, u = h.split(inter, 1)
        z = torch.nn.functional.silu(g) * u
        o = dense_lora(z, ref["w2"], l2, dict(a=ref["a2"], b=ref["b2"]), e) if rank else z @ ref["w2"][e].T
        want = want + p[:, e:e + 1] * o
    want.backward(gy.double().cpu())
    off = lambda g, v: ((g.double().cpu() - v).norm() / v.norm()).item()  # noqa: E731
    assert off(y.detach(), want.detach()) < 0.012
    for name, v in leaves.items():
        assert off(v.grad, ref[name].grad) < 0.024, name


def test_only_the_gradients_that_are_needed(G):  # noqa: F811
    """Frozen weights get no gradient, and the adapters' are the same bits as beside
    weights that do; a second derivative is refused."""
    from combine_ep_dispatch_amd.autograd import EpDispatcher

    T, H, E, inter = 33, 64, 4, 24
    cfg = G.epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=1, top_k=2, align=8)
    d = EpDispatcher(cfg, "cuda:0")
    ids = torch.argsort(normal(9, T, E, dtype=torch.float32), dim=1)[:, :2].int().contiguous()
    got = []
    for frozen in (True, False):
        l = lora_leaves(2, E, 8, H, 2 * inter, T, 30)
        w = normal(3, E, 2 * inter, H, std=H ** -0.5).requires_grad_(not frozen)
        act = d.gated(d.dispatch(normal(1, T, H), ids), w, None, G.epx.Adapters(l["of"], l["a"], l["b"], l["scale"]))
        act.backward(normal(2, *act.shape))
        assert (w.grad is None) == frozen
        got.append((act.detach(), l["a"].grad, l["b"].grad))
    for one, other in zip(*got):
        assert torch.equal(one, other)
    x = normal(1, T, H).requires_grad_()
    l = lora_leaves(2, E, 8, H, 2 * inter, T, 30)
    act = d.gated(d.dispatch(x, ids), normal(3, E, 2 * inter, H), None, G.epx.Adapters(l["of"], l["a"], l["b"]))
    (gx,) = torch.autograd.grad(act.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated twice"):
        gx.float().sum().backward()


@pytest.mark.parametrize("which", ["of", "scale"])
@pytest.mark.parametrize("gated", [False, True])
def test_adapters_changed_before_the_backward_pass_are_refused(G, gated, which):  # noqa: F811
    """The tokens' adapters or their scales written over between the passes: the gradients would not be the results'."""
    from combine_ep_dispatch_amd.autograd import EpDispatcher

    T, H, E, inter = 17, 64, 4, 16
    cfg = G.epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=1, top_k=2, align=8)
    d = EpDispatcher(cfg, "cuda:0")
    ids = torch.argsort(normal(9, T, E, dtype=torch.float32), dim=1)[:, :2].int().contiguous()
    l = lora_leaves(2, E, 8, H, 2 * inter, T, 30)
    rows, w = d.dispatch(normal(1, T, H), ids), normal(3, E, 2 * inter, H, std=H ** -0.5)
    adapters = G.epx.Adapters(l["of"], l["a"], l["b"], l["scale"])
    y = d.gated(rows, w, None, adapters) if gated else d.linear(rows, w, adapters)
    l[which].zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()


def step_of(G, cfg, t, b):  # noqa: F811
    """A training step of the layer by the calls themselves, into the buffers b."""
    e, lay = G.epx, t["lay"]
    e.ep_dispatch_with_layout(cfg, t["ids"].view(-1), t["ws"], lay, t["x"].view(-1), b["recv"].view(-1))
    e.ep_lora_down(cfg, lay, b["recv"], t["lora"], b["u"])
    e.ep_expert_gated(cfg, lay, b["recv"], t["w1"], t["probs"], b["act"], t["lora"], b["u"])
    e.ep_expert_gated_nvfp4(cfg, lay, b["recv"], *t["q"], t["probs"], b["actq"], t["lora"], b["u"])
    e.ep_expert_gemm(cfg, lay, b["act"], t["w2"], b["out"])
    e.ep_combine(cfg, lay, b["out"].view(-1), None, b["y"].view(-1))
    e.ep_expert_gemm_bwd_x(cfg, lay, b["out"], t["w2"], b["gact"])
    e.ep_expert_gated_bwd(cfg, lay, b["recv"], t["w1"], t["probs"], b["gact"], b["gh"], grad_probs=b["gp"],
                          workspace=b["parts"], adapters=t["lora"], u=b["u"])
    e.ep_lora_bwd_u(cfg, lay, b["gh"], t["lora"], b["gu"])
    e.ep_expert_gemm_bwd_x_lora(cfg, lay, b["gh"], t["w1"], b["gx"], t["lora"], b["gu"])
    e.ep_lora_bwd_w(cfg, lay, b["recv"], b["gh"], t["lora"], b["u"], b["gu"], b["ga"], b["gb"])
    e.ep_expert_gemm_bwd_w(cfg, lay, b["gh"], b["recv"], b["gw"])
    e.ep_expert_gemm_nvfp4_lora(cfg, lay, b["recv"], *t["q"], b["yq"], t["lora"], b["u"])


def step_inputs(G, T, H, E, inter, rank, seed):  # noqa: F811
    K, n = 2, 3
    cfg = G.epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=1, top_k=K, align=8)
    R = cfg.recv_rows = G.epx.ep_query(cfg).min_recv_rows
    q, _, _ = nvfp4_weights(seed, E, 2 * inter, H)
    l = lora_leaves(n, E, rank, H, 2 * inter, T, seed)
    t = dict(x=normal(seed, T, H), ids=torch.argsort(normal(seed + 1, T, E, dtype=torch.float32), dim=1)[:, :K].int().contiguous(),
             w1=normal(seed + 2, E, 2 * inter, H, std=H ** -0.5), w2=normal(seed + 3, E, H, inter, std=inter ** -0.5), q=q,
             probs=torch.rand(T, K, generator=torch.Generator().manual_seed(seed)).cuda(),
             lora=G.epx.Adapters(l["of"], l["a"].detach(), l["b"].detach(), l["scale"]),
             ws=G.epx.workspace_for(cfg, "cuda:0"), lay=G.epx.Layout.empty(cfg, "cuda:0"))
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    f = torch.float32
    b = dict(recv=z(R, H), u=z(R, rank, dtype=f), act=z(R, inter), actq=z(R, inter), out=z(R, H), y=z(T, H),
             gact=z(R, inter), gh=z(R, 2 * inter), gp=z(T, K, dtype=f), gu=z(R, rank, dtype=f), gx=z(R, H),
             ga=z(n, E, rank, H), gb=z(n, E, 2 * inter, rank), gw=z(E, 2 * inter, H), yq=z(R, 2 * inter),
             parts=G.epx.gated_workspace_for(cfg, inter, "cuda:0").zero_())
    return cfg, t, b


def test_captured_step_replays_like_the_eager_one(G):  # noqa: F811
    """A step captured into a graph: every replay gives the eager call's bits, with
    new inputs and other work in between."""
    cfg, t, b = step_inputs(G, 20, 64, 8, 32, 16, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step_of(G, cfg, t, b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_of(G, cfg, t, b)
    for i in range(4):
        t["x"].copy_(normal(40 + i, *t["x"].shape))
        t["ids"].copy_(torch.argsort(normal(50 + i, 20, 8, dtype=torch.float32), dim=1)[:, :2].int())
        t["lora"].token_adapter.copy_(torch.randint(-1, 3, (20,), generator=torch.Generator().manual_seed(i)).int())
        for v in b.values():
            v.zero_()
        step_of(G, cfg, t, b)
        torch.cuda.synchronize()
        want = {n: v.clone() for n, v in b.items()}
        for v in b.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in b.items():
            assert torch.equal(v.view(torch.uint8), want[n].view(torch.uint8)), (i, n)


def test_steps_on_two_streams(G):  # noqa: F811
    """Two different steps at once, each with buffers of its own on a stream of its own."""
    steps = [step_inputs(G, 300, 144, 4, 72, 24, 5), step_inputs(G, 33, 64, 8, 40, 8, 9)]
    want = []
    for cfg, t, b in steps:
        step_of(G, cfg, t, b)
        torch.cuda.synchronize()
        want.append({n: v.clone() for n, v in b.items()})
        for v in b.values():
            v.zero_()
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(3):
        for (cfg, t, b), stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                step_of(G, cfg, t, b)
    torch.cuda.synchronize()
    for (_, _, b), w in zip(steps, want):
        for n, v in b.items():
            assert torch.equal(v.view(torch.uint8), w[n].view(torch.uint8)), n


def test_offsets_past_32_bits(G):  # noqa: F811
    """Receive rows, weights and adapters of more than 2^32 bytes: the last ones are right."""
    dev = "cuda:0"

    def one_row(cfg, lay, e, x, w, gate, up, lo, u):
        row = int(lay.token_row.view(-1)[cfg.num_tokens - 1])
        act = torch.zeros(cfg.recv_rows, gate.shape[0], dtype=torch.bfloat16, device=dev)
        G.epx.ep_lora_down(cfg, lay, x, lo, u)
        G.epx.ep_expert_gated(cfg, lay, x, w, None, act, lo, u)
        y = torch.zeros(cfg.recv_rows, 2 * gate.shape[0], dtype=torch.bfloat16, device=dev)
        G.epx.ep_expert_gemm_lora(cfg, lay, x, w, y, lo, u)
        k = int(lo.token_adapter[-1])
        v = x[row].double().cpu()
        m, a, b = torch.cat([gate, up]).double().cpu(), lo.a[k, e].double().cpu(), lo.b[k, e].double().cpu()
        uu, eu = u_of(v[None], a, 1.0, 2.0 ** -16)
        want = m @ v + (uu @ b.T)[0]
        err = (m.abs() @ v.abs() * (len(v) + 2) + (uu.abs() @ b.abs().T)[0] * (2 * a.shape[0] + 4)) * U32 + (eu @ b.abs().T)[0]
        check(y[row], want, rounded(want, err), "y")
        (g, uv), (eg, ev) = want.split(len(want) // 2), err.split(len(want) // 2)
        s, silu = silu_parts(g)
        e_act = 1.1 * eg * (uv.abs() + ev) + silu.abs() * ev + (silu * uv).abs() * (24 + g.abs()) * U32 + TINY
        check(act[row], silu * uv, rounded(silu * uv, e_act), "act")

    # 330 000 rows of 7168 values (4.7 GB)
    T, H, inter, rank = 330_000, 7168, 8, 8
    cfg = G.epx.EpConfig(num_tokens=T, hidden=16, num_experts=2, num_segments=1, top_k=1)
    cfg.recv_rows = T
    lay = G.epx.Layout.empty(cfg, dev)
    ids = torch.ones(T, dtype=torch.int32, device=dev)
    G.epx.ep_dispatch_layout(cfg, ids, G.epx.workspace_for(cfg, dev), lay)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=dev).normal_()
    w = normal(3, 2, 2 * inter, H, std=H ** -0.5)
    of = torch.full((T,), -1, dtype=torch.int32, device=dev)
    of[-1] = 1
    lo = G.epx.Adapters(of, normal(4, 2, 2, rank, H, std=H ** -0.5), normal(5, 2, 2, 2 * inter, rank))
    G.say("[gpu] far rows")
    one_row(cfg, lay, 1, x, w, w[1, :inter], w[1, inter:], lo, torch.empty(T, rank, device=dev))
    del x, w
    # 160 experts of 4096 x 4096 (5.4 GB), 5 adapters of rank 128 beside them (1.7 GB)
    E, H, inter, rank, n = 160, 4096, 2048, 128, 5
    cfg = G.epx.EpConfig(num_tokens=3, hidden=16, num_experts=E, num_segments=1, top_k=1)
    cfg.recv_rows = 3
    lay = G.epx.Layout.empty(cfg, dev)
    G.epx.ep_dispatch_layout(cfg, torch.tensor([0, 3, E - 1], dtype=torch.int32, device=dev), G.epx.workspace_for(cfg, dev), lay)
    w = torch.empty(E, 2 * inter, H, dtype=torch.bfloat16, device=dev).normal_(0, H ** -0.5)
    a = torch.empty(n, E, rank, H, dtype=torch.bfloat16, device=dev).normal_(0, H ** -0.5)
    b = torch.empty(n, E, 2 * inter, rank, dtype=torch.bfloat16, device=dev).normal_(0, rank ** -0.5)
    lo = G.epx.Adapters(torch.tensor([-1, 0, n - 1], dtype=torch.int32, device=dev), a, b)
    G.say("[gpu] far weights and adapters")
    one_row(cfg, lay, E - 1, normal(8, 3, H), w, w[E - 1, :inter], w[E - 1, inter:], lo, torch.empty(3, rank, device=dev))
