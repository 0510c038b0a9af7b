"""The expert layer's operators on the GPU against plain forms in 64 bits:
the router and its gradient, the weighted gated activation and its gradients,
the experts' products (bf16 weights, both gradients; 4-bit weights), a run of
them together with the dispatch and combine, replays of a captured run.

Tolerances: an output in bf16 is off by at most half a step, 2^-8 of its
value, on top of the fp32 error before it; that error is counted in fp32
roundings (2^-24 each) of the sum of the terms' magnitudes, as stated at each
test.  Rows that no slot owns have to stay as they were.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
FILL = 0x7A7A  # a bf16 pattern no result has: marks rows that must stay


@pytest.fixture(scope="module")
def G():
    import gpu_cases as gc

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return gc


def normal(seed, *shape, dtype=torch.bfloat16, std=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(std)).to(dtype).to("cuda:0")


def filled(*shape):
    return torch.full(shape, FILL, dtype=torch.int16, device="cuda:0").view(torch.bfloat16)


def check(got, want, err, what):
    """|got - want| <= err + half a bf16 step of what was rounded (bf16 outputs)."""
    got, want, err = got.double().cpu(), want.cpu(), err.cpu()
    assert got.shape == want.shape
    off = (got - want).abs() - err
    bad = ~(off <= 0)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst by {off[bad].max().item()}"


def rounded(want, err):
    """The allowed distance of a bf16 result whose fp32 value is within err of want."""
    return err + (want.abs() + err) * HALF_BF16 + 2.0 ** -133


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------
def plain_route(logits, bias, mask, K, r):
    """ids, q, probs (float64 numpy) from the definition; -1 where nothing is left."""
    z = logits.double().cpu().numpy()
    T, E = z.shape
    with np.errstate(all="ignore"):
        if r.score == "sigmoid":
            s = 1 / (1 + np.exp(-z))
        else:
            e = np.exp(z - z.max(1, keepdims=True))
            s = e / e.sum(1, keepdims=True)
    key = z.copy() if bias is None else s + bias.double().cpu().numpy()
    key[~(z > -np.inf)] = -np.inf
    if r.num_groups > 1:
        part = -np.sort(-key.reshape(T, r.num_groups, -1), axis=2)
        gk = part[..., 0] if bias is None or part.shape[2] == 1 else part[..., 0] + part[..., 1]
        order = np.argsort(-gk, axis=1, kind="stable")[:, r.top_groups:]
        out = np.zeros((T, r.num_groups), bool)
        np.put_along_axis(out, order, True, 1)
        key[np.repeat(out, E // r.num_groups, axis=1)] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
    none = ~(np.take_along_axis(key, ids, 1) > -np.inf)
    if mask is not None:
        none |= (mask.cpu().numpy() == 0)[:, None]
    q = np.where(none, 0.0, np.take_along_axis(s, ids, 1))
    p = r.scale * (q / (q.sum(1, keepdims=True) + 1e-20) if r.normalize else q)
    return np.where(none, -1, ids), s, q, p


def plain_route_bwd(z, s, ids, q, g, r):
    none = ids < 0
    g = np.where(none, 0.0, g)
    if r.normalize:
        Q = q.sum(1, keepdims=True) + 1e-20
        gq = np.where(none, 0.0, r.scale * (g - (g * q).sum(1, keepdims=True) / Q) / Q)
        mag = r.scale * (np.abs(g) + (np.abs(g) * q).sum(1, keepdims=True) / Q) / Q
    else:
        gq = r.scale * g
        mag = r.scale * np.abs(g)
    mag = np.where(none, 0.0, mag)
    T, E = s.shape
    gs, ms = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        for k in range(ids.shape[1]):
            if ids[t, k] >= 0:
                gs[t, ids[t, k]] += gq[t, k]
                ms[t, ids[t, k]] += mag[t, k]
    any_ = (~none).any(1, keepdims=True)
    with np.errstate(all="ignore"):
        if r.score == "sigmoid":
            rest = 1 / (1 + np.exp(z))  # 1 - s without the cancellation (2^-53 against 1 - s = 2e-16 at z = 36)
            gz, mz = gs * s * rest, ms * s * rest
        else:
            gz = s * (gs - (gq * q).sum(1, keepdims=True))
            mz = s * (ms + (mag * q).sum(1, keepdims=True))
    return np.where(any_, gz, 0.0), np.where(any_, mz, 0.0)


ROUTES = [  # T, E, K, score, biased, groups, top_groups, normalize, scale, dtype, kind of logits
    (0, 8, 2, "softmax", False, 1, 1, True, 1.0, "float32", "normal"),
    (1, 1, 1, "softmax", False, 1, 1, True, 1.0, "float32", "normal"),
    (1, 256, 8, "sigmoid", True, 8, 4, True, 2.5, "float32", "normal"),
    (3, 2, 2, "sigmoid", False, 2, 1, False, 1.0, "float32", "normal"),
    (33, 37, 5, "softmax", False, 1, 1, True, 1.0, "bfloat16", "normal"),
    (33, 37, 5, "softmax", True, 37, 9, False, 1.5, "float32", "normal"),
    (129, 64, 6, "softmax", False, 1, 1, False, 1.0, "bfloat16", "ties"),
    (129, 64, 6, "softmax", False, 8, 3, True, 1.0, "bfloat16", "ties"),
    (65, 64, 64 - 1, "sigmoid", False, 1, 1, True, 1.0, "float32", "normal"),
    (70, 96, 8, "sigmoid", True, 4, 2, True, 1.0, "bfloat16", "holes"),
    (70, 96, 8, "softmax", False, 6, 2, True, 1.0, "float32", "holes"),
    (70, 160, 8, "softmax", True, 8, 3, False, 16.0, "float32", "holes"),
    (40, 256, 8, "sigmoid", True, 8, 4, True, 2.5, "float32", "saturated"),
    (40, 256, 8, "sigmoid", True, 1, 1, False, 1.0, "float32", "close"),
    (40, 256, 8, "softmax", True, 8, 4, True, 1.0, "float32", "close"),
    (9, 2048, 16, "sigmoid", True, 64, 5, True, 1.0, "float32", "normal"),
    (9, 1000, 10, "softmax", True, 10, 4, True, 1.0, "bfloat16", "normal"),
    (5, 520, 7, "softmax", False, 1, 1, True, 1.0, "float32", "normal"),
    (300, 128, 2, "sigmoid", False, 1, 1, True, 1.0, "bfloat16", "equal"),
]


def logits_of(kind, T, E, dtype, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)).astype(np.float32) * 1.5
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    if kind == "ties":
        z = np.round(z * 2) / 2
    elif kind == "equal":
        z[:] = 0.25
    elif kind == "holes":  # masked experts, rows with few or none left, a NaN expert
        z[rng.random((T, E)) < 0.5] = -np.inf
        z[::7] = -np.inf
        z[3::7, 5:] = -np.inf
        z[4::7] = np.float32(-3e38)
    elif kind == "saturated":  # 1 / (1 + exp(-z)) of all of them is 1 in fp32
        z = (18 + np.abs(z) * 3).astype(np.float32)
        bias[:] = 0.0
    elif kind == "close":  # pairs whose keys agree to fp32 and differ in 64 bits
        z[:, 1::2] = np.nextafter(z[:, ::2], np.float32(np.inf))
        bias[:] = 0.0
    return torch.from_numpy(z).to(getattr(torch, dtype)).to("cuda:0"), torch.from_numpy(bias).to("cuda:0")


@pytest.mark.parametrize("case", ROUTES, ids=["T%d_E%d_K%d_%s_b%d_g%d-%d_%s_%s" % (*c[:7], c[9], c[10]) for c in ROUTES])
@pytest.mark.parametrize("masked", [False, True])
def test_route(G, case, masked):
    T, E, K, score, biased, groups, top, norm, scale, dtype, kind = case
    G.say(f"[gpu] route {case} masked={masked}")
    logits, bias = logits_of(kind, T, E, dtype, 7 * T + E)
    bias = bias if biased else None
    rng = np.random.default_rng(E)
    mask = torch.from_numpy((rng.random(T) < 0.7).astype(np.uint8) * 3).to("cuda:0") if masked else None
    r = G.epx.RouteConfig(score=score, normalize=norm, num_groups=groups, top_groups=top, scale=scale)
    cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K)
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda:0")
    p = torch.full((T, K), float("nan"), device="cuda:0")
    G.epx.ep_route(cfg, r, logits, ids, p, bias=bias, token_mask=mask)
    want_ids, s, q, want_p = plain_route(logits, bias, mask, K, r)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    # exp and the division: a few roundings, and exp's argument (z - max) is
    # itself rounded: its rounding is relative to |z - max|; the sums add K or E
    z = logits.double().cpu().numpy()
    fin = np.where(np.isfinite(z), z, 0.0)
    spread = np.abs(fin).max(1, keepdims=True) * 2 if T else np.zeros((0, 1))
    spread = np.minimum(spread, 200.0)  # past it the scores are zero
    rel = (32 + E + 2 * spread) * U32
    check(p, torch.from_numpy(want_p), torch.from_numpy(np.abs(want_p) * rel + 1e-37), "probs")

    g = normal(E + 1, T, K, dtype=torch.float32)
    gz = torch.full((T, E), float("nan"), dtype=logits.dtype, device="cuda:0")
    G.epx.ep_route_bwd(cfg, r, logits, ids, g, gz)
    want, mag = plain_route_bwd(z, s, want_ids, q, g.double().cpu().numpy(), r)
    err = torch.from_numpy(mag * 4 * rel + 1e-36)
    want = torch.from_numpy(want)
    check(gz, want, rounded(want, err) if logits.dtype == torch.bfloat16 else err, "grad_logits")


def test_route_gradient_against_differences(G):
    """The gradient against central differences of the weights in 64 bits (step
    1e-4 in the logits: truncation about step^2, 1e-8, against 1e-5 asked for)."""
    T, E, K = 6, 24, 4
    for score in ("softmax", "sigmoid"):
        for norm in (True, False):
            r = G.epx.RouteConfig(score=score, normalize=norm, scale=1.7)
            cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K)
            logits = normal(5, T, E, dtype=torch.float32)
            ids = torch.empty(T, K, dtype=torch.int32, device="cuda:0")
            p = torch.empty(T, K, device="cuda:0")
            G.epx.ep_route(cfg, r, logits, ids, p)
            g = normal(6, T, K, dtype=torch.float32)
            gz = torch.empty_like(logits)
            G.epx.ep_route_bwd(cfg, r, logits, ids, g, gz)
            at, z, gd = ids.long().cpu(), logits.double().cpu(), g.double().cpu()

            def weights(z):
                s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
                q = s.gather(1, at)
                return 1.7 * (q / q.sum(1, keepdim=True) if norm else q)

            for e in range(E):
                d = torch.zeros_like(z)
                d[:, e] = 1e-4
                slope = ((weights(z + d) - weights(z - d)) * gd).sum(1) / 2e-4
                assert (gz[:, e].double().cpu() - slope).abs().max() < 1e-5


def test_route_gradient_of_a_constant_weight(G):
    """One expert a token with normalized weights, or equal gradients for all of
    them: the weights do not move with the logits; what is left is the 1e-20 in
    the sum, scale g 1e-20 / Q^2 at most (Q >= 1/E here), not fp32's rounding."""
    T, E = 50, 64
    for E, K in ((64, 1), (64, 6), (512, 1), (512, 6)):
        for score in ("softmax", "sigmoid"):
            cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K)
            r = G.epx.RouteConfig(score=score, scale=2.5)
            logits = normal(8, T, E, dtype=torch.float32)
            ids, p = torch.empty(T, K, dtype=torch.int32, device="cuda:0"), torch.empty(T, K, device="cuda:0")
            G.epx.ep_route(cfg, r, logits, ids, p)
            g = normal(9, T, 1, dtype=torch.float32).expand(T, K).contiguous()
            gz = torch.empty_like(logits)
            G.epx.ep_route_bwd(cfg, r, logits, ids, g, gz)
            assert gz.abs().max().item() <= 2.5 * g.abs().max().item() * 1e-20 * E * E


def test_route_bwd_skips_invalid_ids(G):
    """Ids outside [0, E) count as unused; a repeated id gets both slots' gradients."""
    cfg = G.epx.EpConfig(num_tokens=2, hidden=8, num_experts=8, num_segments=1, top_k=4)
    logits = normal(1, 2, 8, dtype=torch.float32)
    ids = torch.tensor([[3, -1, 8, 3], [-5, 100, -1, -1]], dtype=torch.int32, device="cuda:0")
    g = torch.tensor([[0.5, float("nan"), float("inf"), 0.25], [1.0, 1.0, 1.0, 1.0]], device="cuda:0")
    for score in ("sigmoid", "softmax"):
        gz = torch.full((2, 8), float("nan"), device="cuda:0")
        G.epx.ep_route_bwd(cfg, G.epx.RouteConfig(score=score, normalize=False), logits, ids, g, gz)
        z = logits.double().cpu().requires_grad_()
        s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
        (0.75 * s[0, 3]).backward()
        check(gz, z.grad, z.grad.abs() * 64 * U32 + 64 * U32, score)
        assert (gz[1] == 0).all()


def test_route_with_nan_and_infinite_logits_keeps_ids_valid(G):
    T, E, K = 64, 96, 8
    rng = np.random.default_rng(3)
    z = rng.standard_normal((T, E)).astype(np.float32)
    z[rng.random((T, E)) < 0.2] = np.nan
    z[rng.random((T, E)) < 0.1] = np.inf
    z[5] = np.nan
    for score in ("softmax", "sigmoid"):
        for biased in (False, True):
            cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K)
            logits = torch.from_numpy(z).to("cuda:0")
            ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda:0")
            p = torch.empty(T, K, device="cuda:0")
            bias = torch.zeros(E, device="cuda:0") if biased else None
            G.epx.ep_route(cfg, G.epx.RouteConfig(score=score, num_groups=4, top_groups=2), logits, ids, p, bias=bias)
            i = ids.cpu().numpy()
            assert ((i >= -1) & (i < E)).all()
            for t in range(T):
                used = i[t][i[t] >= 0]
                assert len(set(used)) == len(used) and not np.isnan(z[t, used]).any()
            assert (i[5] == -1).all()


# ---------------------------------------------------------------------------
# Rows of a layout
# ---------------------------------------------------------------------------
LAYOUTS = {  # name: config, fraction of unused slots, expert weights (None: uniform)
    "empty": (dict(num_tokens=0, num_experts=4, num_segments=2, top_k=2, align=8), 0.0, None),
    "one": (dict(num_tokens=1, num_experts=8, num_segments=1, top_k=1, align=1), 0.0, None),
    "one-top8": (dict(num_tokens=1, num_experts=16, num_segments=4, top_k=8, align=16, shared_expert=1,
                      src_segment=2), 0.0, None),
    "all-unused": (dict(num_tokens=9, num_experts=4, num_segments=1, top_k=2, align=4), 1.0, None),
    "odd": (dict(num_tokens=77, num_experts=6, num_segments=3, top_k=3, align=1), 0.2, None),
    "aligned": (dict(num_tokens=150, num_experts=10, num_segments=2, top_k=4, align=32, shared_expert=1,
                     src_segment=1), 0.1, None),
    "skewed": (dict(num_tokens=333, num_experts=8, num_segments=2, top_k=2, align=16), 0.0, "skew"),
    "capacity": (dict(num_tokens=200, num_experts=8, num_segments=2, top_k=3, align=8, seg_capacity=217), 0.0, "skew"),
    "many-groups": (dict(num_tokens=40, num_experts=2000, num_segments=8, top_k=4, align=1), 0.0, None),
    "twenty": (dict(num_tokens=40, num_experts=4, num_segments=1, top_k=2, align=16), 0.0, None),
    "tall": (dict(num_tokens=700, num_experts=2, num_segments=1, top_k=2, align=128), 0.0, None),
}


MANY = {  # enough tiles of 64 x 64 for the wide ones: by 256 rows, by 128, unevenly
    "many-rows": (dict(num_tokens=3000, num_experts=4, num_segments=2, top_k=2, align=1, shared_expert=1), 0.02, None),
    "many-75": (dict(num_tokens=1500, num_experts=40, num_segments=4, top_k=2, align=16), 0.0, None),
    "many-skewed": (dict(num_tokens=3001, num_experts=6, num_segments=1, top_k=2, align=8), 0.1, "skew"),
}


class Rows:
    """A layout made by ep_dispatch_layout, and what the plain forms need of it."""

    def __init__(self, G, name, hidden=16, flags=0, seed=0):
        kw, unused, weights = (LAYOUTS | MANY)[name]
        cfg = G.epx.EpConfig(hidden=hidden, flags=flags, **kw)
        cfg.recv_rows = G.epx.ep_query(cfg).min_recv_rows + 5  # rows behind the last segment
        rng = np.random.default_rng(seed + 17)
        T, E, K = cfg.num_tokens, cfg.num_experts, cfg.top_k
        w = 1.0 / np.arange(1, E + 1) ** 2 if weights == "skew" else np.ones(E)
        u = rng.random((T, E)).clip(1e-300)
        ids = np.argsort(-(np.log(w) - np.log(-np.log(u))), axis=1)[:, :K].astype(np.int32)
        ids = np.where(rng.random((T, K)) < unused, -1, ids).astype(np.int32)
        self.cfg, self.ids = cfg, torch.from_numpy(np.ascontiguousarray(ids)).to("cuda:0")
        self.lay = G.sentinel_layout(cfg)
        G.epx.ep_dispatch_layout(cfg, self.ids.view(-1), G.epx.workspace_for(cfg, "cuda:0"), self.lay)
        self.T, self.K, self.R, self.experts = T, K, cfg.recv_rows, E + cfg.shared_expert
        tr = self.lay.token_row.cpu().long()
        self.slots = (tr.view(-1) >= 0).nonzero().view(-1)
        self.rows = tr.view(-1)[self.slots]
        kept = torch.zeros(self.R, dtype=torch.bool)
        kept[self.rows] = True
        self.kept = kept
        full = np.concatenate([ids, np.full((T, cfg.shared_expert), E, np.int32)], 1)
        self.expert = torch.from_numpy(full.reshape(-1)).long()[self.slots]  # of self.rows
        self.probs = torch.from_numpy(rng.random((T, K)).astype(np.float32)).to("cuda:0")
        w = torch.ones(T, cfg.kp, dtype=torch.float64)
        w[:, :K] = self.probs.double().cpu()
        self.w = w.view(-1)[self.slots]

    def untouched(self, out, zeroed=None):
        """Rows that no slot owns hold what they held (or zero, for pad rows asked for)."""
        rest = out.view(torch.int16).cpu()[~self.kept]
        ok = rest == FILL
        if zeroed is not None:
            ok = torch.where(zeroed[~self.kept][:, None], rest == 0, ok)
        assert ok.all()

    def pad_rows(self):
        """Rows [count, aligned count) of each group, below the capacity."""
        cfg, pad = self.cfg, torch.zeros(self.R, dtype=torch.bool)
        c, off, base = (getattr(self.lay, n).cpu() for n in ("counts", "row_offsets", "seg_base"))
        for s in range(cfg.num_segments):
            for g in range(cfg.groups_per_segment):
                n, o = int(c[s, g]), int(off[s, g])
                a = -(-n // cfg.align) * cfg.align
                lim = cfg.seg_capacity or (1 << 30)
                pad[int(base[s]) + min(o + n, lim):int(base[s]) + min(o + a, lim)] = True
        return pad


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("inter", [8, 520, 1416])
@pytest.mark.parametrize("weighted", [True, False])
def test_swiglu(G, name, inter, weighted):
    G.say(f"[gpu] swiglu {name} inter={inter} weighted={weighted}")
    d = Rows(G, name)
    h, ga = normal(1, d.R, 2 * inter, std=2.0), normal(2, d.R, inter)
    if d.R:
        h.view(-1)[::97] = 90.0  # exp(-a) underflows
        h.view(-1)[::89] = -95.0  # exp(-a) overflows
    probs = d.probs if weighted else None
    w = (d.w if weighted else torch.ones_like(d.w))[:, None]
    act = filled(d.R, inter)
    G.epx.ep_swiglu(d.cfg, d.lay, h, probs, act)
    a, b = h.cpu()[d.rows].double().split(inter, 1)
    g = ga.cpu()[d.rows].double()
    s = torch.sigmoid(a)
    # exp, 1 + e, the division, three products: under 16 roundings; exp's
    # own error counts for |a| (1 - s) of its argument at most.  Where exp(-a)
    # passes the largest float (a < -88.7) s is 0 instead of less than 2^-128.
    tiny = 2.0 ** -127
    want = w * a * s * b
    err = want.abs() * (16 + a.abs()) * U32 + (w * a * b).abs() * tiny + tiny
    check(act.cpu()[d.rows], want, rounded(want, err), "act")
    d.untouched(act)

    gh = filled(d.R, 2 * inter)
    gp = torch.full((d.T, d.K), float("nan"), device="cuda:0")
    G.epx.ep_swiglu_bwd(d.cfg, d.lay, h, probs, ga, gh, gp if weighted else None)
    want = torch.cat([w * g * b * s * (1 + a * torch.sigmoid(-a)), w * g * a * s], 1)
    size = torch.cat([(w * g * b).abs() * (1 + a.abs()), (w * g * a).abs()], 1)
    err = size * (torch.cat([s, s], 1) * (24 + torch.cat([a, a], 1).abs()) * U32 + tiny) + tiny
    check(gh.cpu()[d.rows], want, rounded(want, err), "grad_h")
    d.untouched(gh)
    if weighted:
        full = torch.zeros(d.T * d.cfg.kp, dtype=torch.float64)
        size = torch.zeros_like(full)
        full[d.slots] = (g * a * s * b).sum(1)
        size[d.slots] = ((g * a * b).abs() * (s * (inter + 16 + a.abs()) * U32 + tiny)).sum(1)
        full, size = (v.view(d.T, d.cfg.kp)[:, : d.K] for v in (full, size))
        check(gp, full, size + tiny, "grad_probs")


def test_swiglu_gradient_against_differences(G):
    """grad_h and grad_probs against central differences of the definition in 64
    bits (step 1e-4: 1e-8 of truncation; bf16 results are off by 2^-8 of their value)."""
    d = Rows(G, "odd")
    inter = 8
    h, ga = normal(1, d.R, 2 * inter), normal(2, d.R, inter)
    gh, gp = filled(d.R, 2 * inter), torch.empty(d.T, d.K, device="cuda:0")
    G.epx.ep_swiglu_bwd(d.cfg, d.lay, h, d.probs, ga, gh, gp)
    x, g, w = h.cpu()[d.rows].double(), ga.cpu()[d.rows].double(), d.w[:, None]

    def loss(x, w):
        a, b = x.split(inter, 1)
        return (w * a * torch.sigmoid(a) * b * g).sum(1)

    got = gh.cpu()[d.rows].double()
    for j in range(2 * inter):
        e = torch.zeros_like(x)
        e[:, j] = 1e-4
        slope = (loss(x + e, w) - loss(x - e, w)) / 2e-4
        assert ((got[:, j] - slope).abs() <= slope.abs() * HALF_BF16 * 1.01 + 1e-5).all()
    slope = (loss(x, w + 1e-4) - loss(x, w - 1e-4)) / 2e-4
    assert ((gp.cpu().view(-1).double()[d.slots] - slope).abs() <= 1e-5).all()


def expert_sums(d, f):
    for e in range(d.experts):
        on = (d.expert == e).nonzero().view(-1)
        f(e, on, d.rows[on])


# (in, out): the smallest, odd, past one tile each way, wide and flat
DIMS = [(8, 8), (40, 264), (136, 72), (264, 520), (1416, 88), (72, 1032)]


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("dims", DIMS, ids=str)
def test_expert_gemm_and_gradients(G, name, dims):
    n_in, n_out = dims
    if name == "many-groups" and n_in * n_out > 50000:
        n_in, n_out = n_in // 16 // 8 * 8 + 8, n_out // 16 // 8 * 8 + 8  # 2000 experts' weights stay small
    G.say(f"[gpu] expert_gemm {name} in={n_in} out={n_out}")
    d = Rows(G, name)
    x, gy = normal(1, d.R, n_in), normal(2, d.R, n_out)
    w = normal(3, d.experts, n_out, n_in)
    nan = torch.zeros(d.R, 1, dtype=torch.bfloat16)
    nan[~d.kept] = float("nan")  # rows that no slot owns are never read
    x, gy = x + nan.to(x), gy + nan.to(gy)
    y, gx = filled(d.R, n_out), filled(d.R, n_in)
    gw = filled(d.experts, n_out, n_in)
    gw32 = torch.full((d.experts, n_out, n_in), float("nan"), device="cuda:0")
    G.epx.ep_expert_gemm(d.cfg, d.lay, x, w, y)
    G.epx.ep_expert_gemm_bwd_x(d.cfg, d.lay, gy, w, gx)
    G.epx.ep_expert_gemm_bwd_w(d.cfg, d.lay, gy, x, gw)
    G.epx.ep_expert_gemm_bwd_w(d.cfg, d.lay, gy, x, gw32)
    acc = torch.full_like(gw32, 0.5)
    G.epx.ep_expert_gemm_bwd_w(d.cfg, d.lay, gy, x, acc, accumulate=True)
    assert torch.equal(acc, gw32 + 0.5)
    xc, gc, wc = x.double().cpu(), gy.double().cpu(), w.double().cpu()
    yc, gxc, gwc, g32c = y.cpu(), gx.cpu(), gw.cpu(), gw32.cpu()

    def one(e, on, rows):
        a, b, m = xc[rows], gc[rows], wc[e]
        # fp32 sums of exact products: one rounding a term, of the sum of magnitudes
        for got, want, size, n in ((yc[rows], a @ m.T, a.abs() @ m.abs().T, n_in),
                                   (gxc[rows], b @ m, b.abs() @ m.abs(), n_out),
                                   (gwc[e], b.T @ a, b.abs().T @ a.abs(), len(rows))):
            check(got, want, rounded(want, size * (n + 1) * U32), f"expert {e}")
        check(g32c[e], b.T @ a, (b.abs().T @ a.abs()) * (len(rows) + 1) * U32, f"expert {e} fp32")

    expert_sums(d, one)
    d.untouched(y)
    d.untouched(gx)


@pytest.mark.parametrize("name", MANY)
@pytest.mark.parametrize("dims", [(520, 584), (1032, 520)], ids=str)
def test_expert_gemm_and_gradients_of_many_rows(G, name, dims):
    test_expert_gemm_and_gradients(G, name, dims)


E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def nvfp4_weights(seed, experts, n_out, n_in):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (experts, n_out, n_in // 2)).astype(np.uint8)
    scales = rng.integers(0, 256, (experts, n_out, n_in // 16)).astype(np.uint8)
    scales[(scales & 0x7F) == 0x7F] = 0x01  # the smallest subnormal in the NaN codes' place
    rowscale = torch.from_numpy((rng.random((experts, n_out)) * 0.01).astype(np.float32)).to(torch.bfloat16)
    c = torch.from_numpy(codes).long()
    v = torch.stack([E2M1[c & 15], E2M1[c >> 4]], -1).view(experts, n_out, n_in // 16, 16)
    sc = torch.from_numpy(scales).view(torch.float8_e4m3fn).double()
    w = (v * sc[..., None]).view(experts, n_out, n_in)
    return [t.to("cuda:0") for t in (torch.from_numpy(codes), torch.from_numpy(scales), rowscale)], w, rowscale.double()


NV_DIMS = [(16, 8), (48, 264), (64, 136), (272, 72), (320, 264), (1040, 136), (528, 520), (1152, 72)]


@pytest.mark.parametrize("name", LAYOUTS)
@pytest.mark.parametrize("dims", NV_DIMS, ids=str)
def test_expert_gemm_nvfp4(G, name, dims):
    n_in, n_out = dims
    if name == "many-groups" and n_in * n_out > 50000:
        n_in, n_out = n_in // 16 // 16 * 16 + 16, n_out // 16 // 8 * 8 + 8
    G.say(f"[gpu] expert_gemm_nvfp4 {name} in={n_in} out={n_out}")
    d = Rows(G, name)
    x = normal(1, d.R, n_in)
    nan = torch.zeros(d.R, 1, dtype=torch.bfloat16)
    nan[~d.kept] = float("nan")
    x = x + nan.to(x)
    (codes, scales, rowscale), w, rs = nvfp4_weights(5, d.experts, n_out, n_in)
    y = filled(d.R, n_out)
    G.epx.ep_expert_gemm_nvfp4(d.cfg, d.lay, x, codes, scales, rowscale, y)
    xc, yc = x.double().cpu(), y.cpu()

    def one(e, on, rows):
        want, size = xc[rows] @ w[e].T * rs[e], xc[rows].abs() @ w[e].abs().T * rs[e]
        check(yc[rows], want, rounded(want, size * (n_in + 2) * U32), f"expert {e}")

    expert_sums(d, one)
    d.untouched(y)


def test_pad_rows_are_zeroed_on_request(G):
    """EP_ZERO_PAD_ROWS: pad rows of every row output are zero, rows past them stay."""
    d = Rows(G, "aligned", flags=G.epx.EP_ZERO_PAD_ROWS)
    pad = d.pad_rows()
    assert pad.any()
    inter, n_out = 24, 40
    h, ga = normal(1, d.R, 2 * inter), normal(2, d.R, inter)
    act, gh, y, gx, yq = (filled(d.R, c) for c in (inter, 2 * inter, n_out, inter, n_out))
    w = normal(3, d.experts, n_out, inter)
    G.epx.ep_swiglu(d.cfg, d.lay, h, d.probs, act)
    G.epx.ep_swiglu_bwd(d.cfg, d.lay, h, d.probs, ga, gh)
    G.epx.ep_expert_gemm(d.cfg, d.lay, ga, w, y)
    G.epx.ep_expert_gemm_bwd_x(d.cfg, d.lay, normal(4, d.R, n_out), w, gx)
    (codes, scales, rowscale), _, _ = nvfp4_weights(5, d.experts, n_out, 2 * inter)
    G.epx.ep_expert_gemm_nvfp4(d.cfg, d.lay, h, codes, scales, rowscale, yq)
    for out in (act, gh, y, gx, yq):
        d.untouched(out, zeroed=pad)
        assert (out.view(torch.int16).cpu()[d.kept] != FILL).any(1).all()


def test_infinities_and_nan_stay_in_their_rows(G):
    """A row with an infinity or a NaN spoils its own results only (and its expert's gradient)."""
    d = Rows(G, "aligned")
    x, w = normal(1, d.R, 64), normal(3, d.experts, 72, 64)
    (codes, scales, rowscale), _, _ = nvfp4_weights(5, d.experts, 72, 64)
    clean, cleanq = filled(d.R, 72), filled(d.R, 72)
    G.epx.ep_expert_gemm(d.cfg, d.lay, x, w, clean)
    G.epx.ep_expert_gemm_nvfp4(d.cfg, d.lay, x, codes, scales, rowscale, cleanq)
    bad = d.rows[::5]
    x[bad.to("cuda:0")[::2], 3] = float("inf")
    x[bad.to("cuda:0")[1::2], 60] = float("nan")
    got, gotq = filled(d.R, 72), filled(d.R, 72)
    G.epx.ep_expert_gemm(d.cfg, d.lay, x, w, got)
    G.epx.ep_expert_gemm_nvfp4(d.cfg, d.lay, x, codes, scales, rowscale, gotq)
    keep = torch.ones(d.R, dtype=torch.bool)
    keep[bad] = False
    assert torch.equal(got.view(torch.int16).cpu()[keep], clean.view(torch.int16).cpu()[keep])
    assert torch.equal(gotq.view(torch.int16).cpu()[keep], cleanq.view(torch.int16).cpu()[keep])
    assert not torch.isfinite(got.cpu()[bad].float()).all(1).any()


def test_a_rows_results_do_not_depend_on_the_batch(G):
    """The same row alone, among few and among many rows of its expert (other tile
    sizes): the same bits."""
    n_in, n_out = 448, 264
    x1, w = normal(1, 1, n_in), normal(3, 1, n_out, n_in)
    (codes, scales, rowscale), _, _ = nvfp4_weights(5, 1, n_out, n_in)
    seen = []
    for E, T in ((1, 1), (1, 20), (1, 40), (1, 100), (1, 700), (1, 15000), (160, 1600)):
        cfg = G.epx.EpConfig(num_tokens=T, hidden=16, num_experts=E, num_segments=1, top_k=1)
        cfg.recv_rows = G.epx.ep_query(cfg).min_recv_rows
        lay = G.epx.Layout.empty(cfg, "cuda:0")
        ids = torch.arange(T, dtype=torch.int32, device="cuda:0") % E
        G.epx.ep_dispatch_layout(cfg, ids, G.epx.workspace_for(cfg, "cuda:0"), lay)
        at = lay.token_row.view(-1)[T // 2].item()
        x = normal(T, T, n_in)
        x[at] = x1[0]
        y, yq, gx = filled(T, n_out), filled(T, n_out), filled(T, n_out)
        we, qe = w.repeat(E, 1, 1), [v.repeat(E, *[1] * (v.dim() - 1)) for v in (codes, scales, rowscale)]
        G.epx.ep_expert_gemm(cfg, lay, x, we, y)
        G.epx.ep_expert_gemm_nvfp4(cfg, lay, x, *qe, yq)
        G.epx.ep_expert_gemm_bwd_x(cfg, lay, x, we.transpose(1, 2).contiguous(), gx)
        seen.append([v[at].view(torch.int16).cpu() for v in (y, yq, gx)])
    for other in seen[1:]:
        for a, b in zip(seen[0], other):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(G):
    """Receive rows, weights, codes, activations and logits of more than 2^32
    bytes (and values): the last ones are right."""
    dev = "cuda:0"
    # rows: 330 000 of 7168 values
    T, n_in, n_out = 330_000, 7168, 8
    cfg = G.epx.EpConfig(num_tokens=T, hidden=16, num_experts=2, num_segments=1, top_k=1)
    cfg.recv_rows = T
    lay = G.epx.Layout.empty(cfg, dev)
    ids = torch.arange(T, device=dev, dtype=torch.int32) % 2
    G.epx.ep_dispatch_layout(cfg, ids, G.epx.workspace_for(cfg, dev), lay)
    x = torch.empty(T, n_in, dtype=torch.bfloat16, device=dev).normal_()
    w = normal(3, 2, n_out, n_in)
    y, gx = filled(T, n_out), torch.empty_like(x)
    some = torch.tensor([0, 1, T // 2 - 1, T // 2, 299_593, 299_594, T - 2, T - 1], device=dev)
    e = (some >= T // 2).long()
    G.say("[gpu] far rows")
    G.epx.ep_expert_gemm(cfg, lay, x, w, y)
    xs, ws = x[some].double().cpu(), w.double().cpu()[e.cpu()]
    want, size = torch.einsum("rh,rnh->rn", xs, ws), torch.einsum("rh,rnh->rn", xs.abs(), ws.abs())
    check(y[some], want, rounded(want, size * (n_in + 1) * U32), "far rows")
    gy = normal(4, T, n_out)
    G.epx.ep_expert_gemm_bwd_x(cfg, lay, gy, w, gx)
    gs = gy[some].double().cpu()
    want, size = torch.einsum("rn,rnh->rh", gs, ws), torch.einsum("rn,rnh->rh", gs.abs(), ws.abs())
    check(gx[some], want, rounded(want, size * (n_out + 1) * U32), "far gradients")
    act = gx.view(-1)[: T * n_in // 2].view(T, n_in // 2)
    G.epx.ep_swiglu(cfg, lay, x, None, act)
    a, b = xs.split(n_in // 2, 1)
    want = a * torch.sigmoid(a) * b
    check(act[some], want, rounded(want, want.abs() * (16 + a.abs()) * U32 + 2.0 ** -126), "far activations")
    del x, gx, act
    # weights: 70 experts of 8192 x 8192, 4-bit and bf16 (9.4 GB); one token each way
    E, n = 70, 8192
    cfg = G.epx.EpConfig(num_tokens=1, hidden=16, num_experts=E, num_segments=1, top_k=2)
    cfg.recv_rows = 2
    lay = G.epx.Layout.empty(cfg, dev)
    G.epx.ep_dispatch_layout(cfg, torch.tensor([E - 1, 0], dtype=torch.int32, device=dev), G.epx.workspace_for(cfg, dev), lay)
    x = normal(1, 2, n)
    w = torch.empty(E, n, n, dtype=torch.bfloat16, device=dev).normal_()
    y = filled(2, n)
    G.say("[gpu] far weights")
    G.epx.ep_expert_gemm(cfg, lay, x, w, y)
    for row, e in ((0, 0), (1, E - 1)):
        a, m = x[row].double(), w[e].double()
        want, size = m @ a, m.abs() @ a.abs()
        check(y[row], want, rounded(want, size * (n + 1) * U32), "far weights")
    gw = w  # the gradient of all experts, in the weights' place
    G.epx.ep_expert_gemm_bwd_w(cfg, lay, x, x, gw)
    assert (gw[1:-1] == 0).all()
    for row, e in ((0, 0), (1, E - 1)):
        a = x[row].double()
        want = torch.outer(a, a)
        check(gw[e], want, rounded(want, want.abs() * 2 * U32), "far weights' gradient")
    del w, gw
    E = 140
    cfg.num_experts = E
    lay = G.epx.Layout.empty(cfg, dev)
    G.epx.ep_dispatch_layout(cfg, torch.tensor([E - 1, 0], dtype=torch.int32, device=dev), G.epx.workspace_for(cfg, dev), lay)
    codes = torch.randint(0, 256, (E, n, n // 2), dtype=torch.uint8, device=dev)
    scales = torch.randint(0x30, 0x70, (E, n, n // 16), dtype=torch.uint8, device=dev)
    rowscale = torch.rand(E, n, device=dev).to(torch.bfloat16)
    G.say("[gpu] far codes")
    G.epx.ep_expert_gemm_nvfp4(cfg, lay, x, codes, scales, rowscale, y)
    for row, e in ((0, 0), (1, E - 1)):
        c = codes[e].long().cpu()
        v = torch.stack([E2M1[c & 15], E2M1[c >> 4]], -1).view(n, n // 16, 16)
        m = (v * scales[e].cpu().view(torch.float8_e4m3fn).double()[..., None]).view(n, n)
        a, rs = x[row].double().cpu(), rowscale[e].double().cpu()
        want, size = m @ a * rs, m.abs() @ a.abs() * rs
        check(y[row], want, rounded(want, size * (n + 2) * U32), "far codes")
    del codes, scales, rowscale
    # logits: 2.2 million tokens of 1024 experts
    T, E, K = 2_200_000, 1024, 4
    cfg = G.epx.EpConfig(num_tokens=T, hidden=8, num_experts=E, num_segments=1, top_k=K)
    logits = torch.empty(T, E, device=dev).normal_()
    ids, p = torch.empty(T, K, dtype=torch.int32, device=dev), torch.empty(T, K, device=dev)
    r = G.epx.RouteConfig(score="sigmoid")
    G.say("[gpu] far logits")
    G.epx.ep_route(cfg, r, logits, ids, p)
    some = torch.tensor([0, 1, T // 2, 2_097_152, 2_097_153, T - 1], device=dev)
    want_ids, s, q, want = plain_route(logits[some], None, None, K, r)
    np.testing.assert_array_equal(ids[some].cpu().numpy(), want_ids)
    check(p[some], torch.from_numpy(want), torch.from_numpy(want * 64 * U32), "far weights")
    gz = torch.full_like(logits, 7.0)
    G.epx.ep_route_bwd(cfg, r, logits, ids, p, gz)
    want, mag = plain_route_bwd(logits[some].double().cpu().numpy(), s, want_ids, q, p[some].double().cpu().numpy(), r)
    check(gz[some], torch.from_numpy(want), torch.from_numpy(mag * 64 * U32 + 1e-30), "far gradients")


def test_products_past_one_grid_are_refused(G):
    """2048 groups of 2^20 features: more workgroups than a launch holds."""
    E, big = 2048, 1 << 20
    cfg = G.epx.EpConfig(num_tokens=E, hidden=8, num_experts=E, num_segments=1, top_k=1)
    cfg.recv_rows = E
    lay = G.epx.Layout.empty(cfg, "cuda:0")
    ids = torch.arange(E, dtype=torch.int32, device="cuda:0")
    G.epx.ep_dispatch_layout(cfg, ids, G.epx.workspace_for(cfg, "cuda:0"), lay)
    w = torch.empty(E * big * 8, dtype=torch.bfloat16, device="cuda:0")
    rows, few = torch.empty(E, big, dtype=torch.bfloat16, device="cuda:0"), normal(1, E, 8)
    codes, scales = (torch.empty(E, big, n, dtype=torch.uint8, device="cuda:0") for n in (8, 1))
    rowscale = torch.empty(E, big, dtype=torch.bfloat16, device="cuda:0")
    calls = [
        lambda: G.epx.ep_expert_gemm(cfg, lay, few, w.view(E, big, 8), rows),
        lambda: G.epx.ep_expert_gemm_bwd_x(cfg, lay, few, w.view(E, 8, big), rows),
        lambda: G.epx.ep_expert_gemm_bwd_w(cfg, lay, rows, few, w.view(E, big, 8)),
        lambda: G.epx.ep_expert_gemm_nvfp4(cfg, lay, normal(2, E, 16), codes, scales, rowscale, rows),
    ]
    for call in calls:
        with pytest.raises(G.epx.EpError, match="status -1"):
            call()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def layer_inputs(T, H, E, inter, shared, dtype=torch.float32):
    return dict(x=normal(1, T, H), logits=normal(2, T, E, dtype=dtype),
                w1=normal(3, E + shared, 2 * inter, H, std=H ** -0.5),
                w2=normal(4, E + shared, H, inter, std=inter ** -0.5), gy=normal(5, T, H))


def layer(d, route, t, bias=None):
    ids, probs = d.gate(t["logits"], route, bias=bias)
    recv = d.dispatch(t["x"], ids)
    act = d.swiglu(d.linear(recv, t["w1"]), probs)
    return ids, d.combine(d.linear(act, t["w2"]), None)


@pytest.mark.parametrize("shared", [0, 1])
def test_layer_forward_and_backward(G, shared):
    """The whole layer through EpDispatcher against a dense form in 64 bits.  The
    layer rounds to bf16 after each of its five row operations (dispatch copies),
    each at most 2^-8 of the value: results differ by at most 5 * 2^-8 = 0.02 of
    their norm, gradients (up to eight such roundings on the way) by 0.032."""
    from combine_ep_dispatch_amd.autograd import EpDispatcher

    T, H, E, K, inter = 65, 72, 8, 3, 40
    t = layer_inputs(T, H, E, inter, shared)
    leaves = [t[n].requires_grad_() for n in ("x", "logits", "w1", "w2")]
    cfg = G.epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=2, top_k=K, align=16,
                         shared_expert=shared, src_segment=1 if shared else 0)
    route = G.epx.RouteConfig(score="sigmoid", scale=1.5)
    ids, y = layer(EpDispatcher(cfg, "cuda:0"), route, t)
    y.backward(t["gy"])
    ref = [v.detach().double().cpu().requires_grad_() for v in leaves]
    x, z, w1, w2 = ref
    s = torch.sigmoid(z).gather(1, ids.long().cpu())
    p = torch.zeros(T, E + shared, dtype=torch.float64).scatter(1, ids.long().cpu(), 1.5 * s / s.sum(1, keepdim=True))
    if shared:
        p[:, E] = 1.0
    a, b = torch.einsum("th,enh->ten", x, w1).split(inter, 2)
    want = torch.einsum("teh,te->th", torch.einsum("ten,ehn->teh", torch.nn.functional.silu(a) * b, w2), p)
    want.backward(t["gy"].double().cpu())
    off = lambda g, v: ((g.double().cpu() - v).norm() / v.norm()).item()  # noqa: E731
    assert off(y.detach(), want.detach()) < 0.02
    for name, g, v in zip(("x", "logits", "w1", "w2"), leaves, ref):
        assert off(g.grad, v.grad) < 0.032, name


def test_captured_run_replays_like_the_eager_one(G):
    """Router, layout, dispatch, products and activation captured into one graph:
    every replay gives the eager call's bits, with new inputs in between."""
    T, H, E, K, inter = 20, 64, 8, 2, 32
    cfg = G.epx.EpConfig(num_tokens=T, hidden=H, num_experts=E, num_segments=1, top_k=K, align=8)
    cfg.recv_rows = G.epx.ep_query(cfg).min_recv_rows
    t = layer_inputs(T, H, E, inter, 0)
    route = G.epx.RouteConfig(num_groups=2, top_groups=1)
    ws, lay = G.epx.workspace_for(cfg, "cuda:0"), G.epx.Layout.empty(cfg, "cuda:0")
    R = cfg.recv_rows
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    b = dict(ids=z(T, K, dtype=torch.int32), probs=z(T, K, dtype=torch.float32), recv=z(R, H), h=z(R, 2 * inter),
             act=z(R, inter), out=z(R, H), y=z(T, H), gact=z(R, inter), gh=z(R, 2 * inter),
             gp=z(T, K, dtype=torch.float32), gz=z(T, E, dtype=torch.float32), gw=z(E, H, inter))

    def step():
        e = G.epx
        e.ep_route(cfg, route, t["logits"], b["ids"], b["probs"])
        e.ep_dispatch_with_layout(cfg, b["ids"].view(-1), ws, lay, t["x"].view(-1), b["recv"].view(-1))
        e.ep_expert_gemm(cfg, lay, b["recv"], t["w1"], b["h"])
        e.ep_swiglu(cfg, lay, b["h"], b["probs"], b["act"])
        e.ep_expert_gemm(cfg, lay, b["act"], t["w2"], b["out"])
        e.ep_combine(cfg, lay, b["out"].view(-1), None, b["y"].view(-1))
        e.ep_expert_gemm_bwd_x(cfg, lay, b["out"], t["w2"], b["gact"])
        e.ep_expert_gemm_bwd_w(cfg, lay, b["out"], b["act"], b["gw"])
        e.ep_swiglu_bwd(cfg, lay, b["h"], b["probs"], b["gact"], b["gh"], b["gp"])
        e.ep_route_bwd(cfg, route, t["logits"], b["ids"], b["gp"], b["gz"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        t["logits"].copy_(normal(20 + i, T, E, dtype=torch.float32))
        t["x"].copy_(normal(40 + i, T, H))
        for v in (b["recv"], b["h"], b["act"], b["out"], b["gact"], b["gh"]):
            v.zero_()
        step()
        torch.cuda.synchronize()
        want = {n: v.clone() for n, v in b.items()}
        for v in b.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in b.items():
            assert torch.equal(v, want[n]), (i, n)


def test_calls_on_two_streams(G):
    """Two products at once on streams of their own (no workspace is shared)."""
    d = Rows(G, "tall")
    x, w = normal(1, d.R, 264), normal(2, d.experts, 136, 264)
    want = filled(d.R, 136)
    G.epx.ep_expert_gemm(d.cfg, d.lay, x, w, want)
    outs, streams = [filled(d.R, 136) for _ in range(4)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        G.epx.ep_expert_gemm(d.cfg, d.lay, x, w, o, stream=streams[i % 2])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))
