"""The gated block and the products with adapters on the GPU where they are least
ordinary: infinite adapters and rows, beside the calls that it replaces, workgroups that go through many tiles of every
height, batches of many slots."""

import pytest
import torch

import test_gpu_expert_block as block
from test_gpu_expert_block import TINY, Lora, silu_parts, words
from test_gpu_expert_layer import HALF_BF16, U32, G, Rows, check, filled, normal, nvfp4_weights  # noqa: F401

pytestmark = pytest.mark.gpu

INF = float("inf")


def half_rounded(seed, *shape):
    """fp32 values of which every other one is a bf16 too: nothing is left of it by the rounding."""
    t = normal(seed, *shape, dtype=torch.float32)
    t.view(-1)[::2] = t.view(-1)[::2].to(torch.bfloat16).float()
    assert (t != 0).all()
    return t


def same_kinds(got, want, what):
    """The same infinities, signs included, and NaN in the same places."""
    got, want = got.double().cpu(), want.cpu()
    assert torch.isinf(want).any() and torch.isfinite(want).any()
    for v in (INF, -INF):
        assert torch.equal(got == v, want == v), what
    assert torch.equal(got.isnan(), want.isnan()), what


def with_adapters(d, lora, base, u, weights):
    """base + the adapters' part of the kept rows, term by term (infinities as they are)."""
    out = base.clone()
    for e in range(d.experts):
        on = (d.expert == e).nonzero().view(-1)
        for k, some in lora.each(on):
            rows = d.rows[on][some]
            out[rows] += (weights(k, e)[None] * u[rows][:, None]).sum(2)
    return out


@pytest.mark.parametrize("name", ["odd", "tall"])
@pytest.mark.parametrize("rank", [8, 40])
def test_infinite_adapters_make_infinite_results(G, name, rank):  # noqa: F811
    """An infinity in an adapter times u is an infinity of that sign, whatever the
    rounding of u leaves of it, and two that cancel are NaN."""
    d = Rows(G, name)
    n_in, inter = 64, 72
    x, gy = normal(1, d.R, n_in), normal(2, d.R, 2 * inter)
    w = normal(3, d.experts, 2 * inter, n_in, std=n_in ** -0.5)
    q, wq, rs = nvfp4_weights(5, d.experts, 2 * inter, n_in)
    lora, u = Lora(G, d, rank, n_in, 2 * inter), half_rounded(9, d.R, rank)
    lora.b[1, :, inter::3, 5] = INF  # of the up projection
    lora.b[1, :, inter + 1::3, 2] = -INF
    lora.b[0, :, inter + 2::9, 1:3] = INF
    lora.a[1, :, 4, ::3] = -INF
    lora.a[2, :, :2, 1::5] = INF
    y, yq, gx, act, actq = (filled(d.R, n) for n in (2 * inter, 2 * inter, n_in, inter, inter))
    G.epx.ep_expert_gemm_lora(d.cfg, d.lay, x, w, y, lora.c, u)
    G.epx.ep_expert_gemm_nvfp4_lora(d.cfg, d.lay, x, *q, yq, lora.c, u)
    G.epx.ep_expert_gemm_bwd_x_lora(d.cfg, d.lay, gy, w, gx, lora.c, u)
    G.epx.ep_expert_gated(d.cfg, d.lay, x, w, None, act, lora.c, u)
    G.epx.ep_expert_gated_nvfp4(d.cfg, d.lay, x, *q, None, actq, lora.c, u)
    r, uc, xc, gc, wc = d.rows, u.double().cpu(), x.double().cpu(), gy.double().cpu(), w.double().cpu()

    def product(t, m):
        out = torch.zeros(d.R, m.shape[1], dtype=torch.float64)
        for e in range(d.experts):
            rows = r[d.expert == e]
            out[rows] = t[rows] @ m[e].T
        return out

    b, a = (lambda k, e: lora.b[k, e].double().cpu()), (lambda k, e: lora.a[k, e].double().cpu().T)
    h = with_adapters(d, lora, product(xc, wc), uc, b)
    hq = with_adapters(d, lora, product(xc, wq * rs[:, :, None]), uc, b)
    same_kinds(y.cpu()[r], h[r], "y")
    same_kinds(yq.cpu()[r], hq[r], "y, 4-bit")
    same_kinds(gx.cpu()[r], with_adapters(d, lora, product(gc, wc.transpose(1, 2)), uc, a)[r], "grad_x")
    for got, v, what in ((act, h, "act"), (actq, hq, "act, 4-bit")):
        # below g = -86 the sigmoid nears 2^-126 (exp(86) = 2^124.1; g itself is off by less than 1),
        # where 32 bits have 0, and 0 times an infinity is NaN: those are not looked at
        g, up = v[r].split(inter, 1)
        seen = g >= -86
        same_kinds(got.cpu()[r][seen], (torch.nn.functional.silu(g) * up)[seen], what)


@pytest.mark.parametrize("name", ["odd", "tall"])
@pytest.mark.parametrize("rank", [8, 24, 128])
def test_infinite_rows_make_infinite_gradients(G, name, rank):  # noqa: F811
    """The adapters' gradients over rows with infinities: those, of the sign of what
    they are multiplied with, and NaN where both signs meet."""
    d = Rows(G, name)
    n_in, n_out = 264, 72
    x, gy = normal(1, d.R, n_in), normal(2, d.R, n_out)
    lora, u, gu = Lora(G, d, rank, n_in, n_out), half_rounded(8, d.R, rank), half_rounded(9, d.R, rank)
    first = torch.cat([d.rows[on[some]][:1] for e in range(d.experts) for on in [(d.expert == e).nonzero().view(-1)]
                       for _, some in lora.each(on)]).cuda()
    x[first, 3], x[first, 260], gy[first, 7] = INF, -INF, -INF
    x[d.rows.cuda()[::5], 100] = INF  # some of both signs meet
    grads = []
    for dtype in (torch.bfloat16, torch.float32):
        ga, gb = (torch.full(t.shape, float("nan"), dtype=dtype, device="cuda:0") for t in (lora.a, lora.b))
        G.epx.ep_lora_bwd_w(d.cfg, d.lay, x, gy, lora.c, u, gu, ga, gb)
        grads.append((ga, gb))
    xc, gc, uc, vc = x.double().cpu(), gy.double().cpu(), u.double().cpu(), gu.double().cpu()
    wa, wb = (torch.zeros(t.shape, dtype=torch.float64) for t in (lora.a, lora.b))
    for e in range(d.experts):
        on = (d.expert == e).nonzero().view(-1)
        for k, some in lora.each(on):
            rows = d.rows[on[some]]
            for row in rows:
                wa[k, e] += vc[row][:, None] * xc[row][None]
                wb[k, e] += gc[row][:, None] * uc[row][None]
    for ga, gb in grads:
        same_kinds(ga, wa, "grad_a")
        same_kinds(gb, wb, "grad_b")


# ---------------------------------------------------------------------------
# Against the calls that the block replaces
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("name", ["one-top8", "odd", "aligned", "capacity", "tall"])
@pytest.mark.parametrize("dims", [(8, 8), (136, 72), (264, 264)], ids=str)
@pytest.mark.parametrize("rank", [0, 16])
def test_the_block_is_the_product_and_the_activation(G, name, dims, rank):  # noqa: F811
    """Forward and backward against ep_expert_gemm (or its form with adapters) and
    ep_swiglu.  Those round h to bf16 in between, each of g and u by at most 2^-8 of its
    value; how far that and the sums' own roundings carry is counted as for the block
    itself, on both sides, and each result's rounding twice."""
    n_in, inter = dims
    d, e = Rows(G, name), G.epx
    x, ga = normal(1, d.R, n_in), normal(2, d.R, inter)
    w = normal(3, d.experts, 2 * inter, n_in, std=n_in ** -0.5)
    h, act, act2, gh, gh2 = (filled(d.R, n) for n in (2 * inter, inter, inter, 2 * inter, 2 * inter))
    gp, gp2 = (torch.full((d.T, d.K), float("nan"), device="cuda:0") for _ in range(2))
    kw, u_size = {}, 0
    if rank:
        lora = Lora(G, d, rank, n_in, 2 * inter)
        kw = dict(adapters=lora.c, u=words(d.R, rank))
        e.ep_lora_down(d.cfg, d.lay, x, lora.c, kw["u"])
        e.ep_expert_gemm_lora(d.cfg, d.lay, x, w, h, **kw)
        u_size = kw["u"].cpu()[d.rows].double().abs().sum(1, keepdim=True) * lora.b.double().abs().max().item()
    else:
        e.ep_expert_gemm(d.cfg, d.lay, x, w, h)
    e.ep_swiglu(d.cfg, d.lay, h, d.probs, act)
    e.ep_swiglu_bwd(d.cfg, d.lay, h, d.probs, ga, gh, gp)
    e.ep_expert_gated(d.cfg, d.lay, x, w, d.probs, act2, **kw)
    e.ep_expert_gated_bwd(d.cfg, d.lay, x, w, d.probs, ga, gh2, grad_probs=gp2,
                          workspace=e.gated_workspace_for(d.cfg, inter, "cuda:0"), **kw)
    r, p = d.rows, d.w[:, None]
    hr, gar = h.cpu()[r].double(), ga.cpu()[r].double()
    # the same sums in another order on each side: (terms + 2) roundings of their size, as
    # sum |x| |w|, at most the largest weight times sum |x|; u's as two bf16, 2^-16
    size = x.cpu()[r].double().abs().sum(1, keepdim=True) * w.double().abs().max().item()
    eh = hr.abs() * HALF_BF16 * 1.01 + 2 * size * (n_in + 4) * U32 + 2 * u_size * (2.0 ** -16 + (2 * rank + 4) * U32)
    (g, v), (eg, ev) = hr.split(inter, 1), eh.split(inter, 1)
    s, silu = silu_parts(g)
    own = 2 * (32 + g.abs()) * U32
    want = p * silu * v
    e_act = p * (1.1 * eg * (v.abs() + ev) + silu.abs() * ev) + want.abs() * own + TINY
    check(act2.cpu()[r], act.cpu()[r].double(), e_act + 2 * (want.abs() + e_act) * HALF_BF16 * 1.01, "act")
    gabs = (p * gar).abs()
    slope = s * (1 + g * torch.sigmoid(-g))
    want = torch.cat([gabs * (v * slope).abs(), gabs * silu.abs()], 1)
    e_h = torch.cat([gabs * (1.1 * ev + (v.abs() + ev) * 0.5 * eg), gabs * 1.1 * eg], 1)
    e_h = e_h + torch.cat([gabs * v.abs() * (1 + g.abs()), gabs * g.abs()], 1) * torch.cat([own, own], 1) + TINY
    check(gh2.cpu()[r], gh.cpu()[r].double(), e_h + 2 * (want + e_h) * HALF_BF16 * 1.01, "grad_h")
    terms = gar.abs() * (1.1 * eg * (v.abs() + ev) + silu.abs() * ev + (silu * v).abs() * (own + 2 * inter * U32))
    err = torch.zeros(d.T * d.cfg.kp, dtype=torch.float64)
    err[d.slots] = terms.sum(1) + TINY
    check(gp2, gp.cpu().double(), err.view(d.T, -1)[:, : d.K], "grad_probs")


# ---------------------------------------------------------------------------
# Workgroups of many tiles, and batches of many slots
# ---------------------------------------------------------------------------
GROUPS = {  # rows of each expert
    # tiles of every height: full ones and what is left over, of one height, of at most 128 and 32 rows
    "mixed": (1100, 0, 900, 300, 180, 100, 20, 1),
    # 16384 slots and more: the adapters' first products take tiles of 64 rows
    "slots": (9000, 5001, 2300, 0, 127, 3, 0, 1),
}


class Groups(Rows):
    """A layout of GROUPS, a slot a token, tokens of all experts in turn."""

    def __init__(self, G, name):  # noqa: F811
        ids = torch.cat([torch.full((n,), e, dtype=torch.int32) for e, n in enumerate(GROUPS[name])])
        ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(3))]
        self.cfg = cfg = G.epx.EpConfig(num_tokens=len(ids), hidden=16, num_experts=len(GROUPS[name]), num_segments=2,
                                        top_k=1, align=16)
        cfg.recv_rows = G.epx.ep_query(cfg).min_recv_rows + 5
        self.ids, self.lay = ids.cuda(), G.sentinel_layout(cfg)
        G.epx.ep_dispatch_layout(cfg, self.ids, G.epx.workspace_for(cfg, "cuda:0"), self.lay)
        self.T, self.K, self.R, self.experts = len(ids), 1, cfg.recv_rows, cfg.num_experts
        self.rows, self.slots = self.lay.token_row.cpu().long().view(-1), torch.arange(self.T)
        self.kept = torch.zeros(self.R, dtype=torch.bool)
        self.kept[self.rows] = True
        self.expert = ids.long()
        self.probs = torch.rand(self.T, 1, generator=torch.Generator().manual_seed(4)).cuda()
        self.w = self.probs.double().cpu().view(-1)


@pytest.fixture
def grouped(monkeypatch):
    """The block's tests on layouts of GROUPS."""
    monkeypatch.setattr(block, "Rows", Groups)
    return block


# 15 row tiles of "mixed" by 40 or 41 feature tiles: two and more of a workgroup's 256
@pytest.mark.parametrize("n_in", [8, 136, 256, 328])
@pytest.mark.parametrize("rank", [0, 8, 24])
def test_gated_block_of_many_tiles(G, grouped, n_in, rank):  # noqa: F811
    grouped.test_gated_forward_and_backward(G, "mixed", (n_in, 5128 if n_in % 64 else 5120), rank)


@pytest.mark.parametrize("dims", [(8, 10248, 8), (136, 10248, 24), (256, 10240, 64), (10248, 136, 24), (10240, 256, 64),
                                  (10248, 8, 8)], ids=str)
def test_products_of_many_tiles(G, grouped, dims):  # noqa: F811
    grouped.test_adapters_and_gradients(G, "mixed", dims)


@pytest.mark.parametrize("dims", [(136, 264, 8), (72, 136, 24), (264, 72, 64), (40, 200, 128)], ids=str)
def test_adapters_of_many_slots(G, grouped, dims):  # noqa: F811
    grouped.test_adapters_and_gradients(G, "slots", dims)


@pytest.mark.parametrize("rank", [8, 24, 64, 128])
def test_u_does_not_depend_on_the_slots(G, rank):  # noqa: F811
    """u and grad_u of a row alone, and among 16384 and more slots (tiles of 64 rows), of
    other adapters: the same bits."""
    n_in, n_out, n = 456, 328, 5
    a, b = normal(6, n, 1, rank, n_in, std=n_in ** -0.5), normal(7, n, 1, n_out, rank)
    scale = (0.5 + torch.rand(n, generator=torch.Generator().manual_seed(1))).cuda()
    x1, gy1, seen = normal(1, 1, n_in), normal(2, 1, n_out), []
    for T in (1, 16383, 16384, 17001):
        cfg = G.epx.EpConfig(num_tokens=T, hidden=16, num_experts=1, num_segments=1, top_k=1)
        cfg.recv_rows = T
        lay = G.epx.Layout.empty(cfg, "cuda:0")
        G.epx.ep_dispatch_layout(cfg, torch.zeros(T, dtype=torch.int32, device="cuda:0"), G.epx.workspace_for(cfg, "cuda:0"), lay)
        of = torch.randint(-1, n, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
        of[T // 2] = 3
        lora, at = G.epx.Adapters(of.cuda(), a, b, scale), lay.token_row.view(-1)[T // 2].item()
        x, gy = normal(T, T, n_in), normal(T + 1, T, n_out)
        x[at], gy[at] = x1[0], gy1[0]
        u, gu = words(T, rank), words(T, rank)
        G.epx.ep_lora_down(cfg, lay, x, lora, u)
        G.epx.ep_lora_bwd_u(cfg, lay, gy, lora, gu)
        seen.append((u[at].cpu(), gu[at].cpu()))
    for other in seen[1:]:
        for one, same in zip(seen[0], other):
            assert torch.equal(one, same)
