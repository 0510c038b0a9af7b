"""Cases and plain forms of the expert layer's operators: the router, the
weighted gated activation on the receive rows, the experts' products (bf16
weights, forward and backward) and the experts' products over 4-bit weights.

`run` computes a case with elementary torch operations, or, where `own` is
true, with the library's kernels; both take what `prepare` made.  Rows of a
receive-side buffer that no token owns (pad rows, rows past a segment's used
rows) are zero in the buffers `prepare` allocates and stay as they are.
"""

import math

import torch

own = False

DEV = "cuda"
TINY = 1e-20  # added to the sum that normalizes the chosen scores


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _route(name, T, E, K, score, biased, groups, top_groups, normalize, scale, dtype, train, masked=0.0):
    return {"name": name, "kind": "route", "T": T, "E": E, "K": K, "score": score, "biased": biased,
            "groups": groups, "top_groups": top_groups, "normalize": normalize, "scale": scale, "dtype": dtype,
            "train": train, "masked": masked}


def _rows(name, kind, T, E, S, K, A, shared=0, capacity=0, zipf=0.0, unused=0.0, **kw):
    return {"name": name, "kind": kind, "T": T, "E": E, "S": S, "K": K, "A": A, "shared": shared,
            "capacity": capacity, "zipf": zipf, "unused": unused, **kw}


def listed():
    return [
        # The router of a decode step: 16 sequences, sigmoid scores with a
        # selection bias, 4 of 8 expert groups (DeepSeek-V3's share: 256
        # experts, top-8).  Latency is all of it.
        _route("route_decode", 16, 256, 8, "sigmoid", True, 8, 4, True, 2.5, "float32", False),
        # The same router in a training step of 4096 tokens, with its gradient.
        _route("route_train", 4096, 256, 8, "sigmoid", True, 8, 4, True, 2.5, "float32", True, masked=0.02),
        # A long packed batch through a softmax router with bf16 logits over
        # 64 experts, top-6 (the capacity workload's experts).
        _route("route_long", 65536, 64, 6, "softmax", False, 1, 1, False, 1.0, "bfloat16", True, masked=0.05),
        # The activation of a decode step.
        _rows("swiglu_decode", "swiglu", 16, 256, 8, 8, 128, I=2048, train=False),
        # The activation of a training step at DeepSeek-V3's share, forward
        # and backward with the weights' gradient; a shared expert as well.
        _rows("swiglu_train", "swiglu", 4096, 256, 8, 8, 128, shared=1, I=2048, train=True, unused=0.03),
        # The capacity workload: skewed routing, dropped slots, rows of an
        # odd width.
        _rows("swiglu_capacity", "swiglu", 16384, 64, 4, 6, 1, capacity=27036, zipf=1.5, I=1416, train=True),
        # The first product of a decode step with bf16 weights, one of the 8
        # segments' 32 experts: bound by reading the weights.
        _rows("gemm_decode", "gemm", 16, 32, 1, 8, 128, N=4096, H=7168, train=False),
        # The first product of a training step over 32 experts (8 rows a token,
        # 1024 rows an expert): bound by the matrix cores.
        _rows("gemm_train", "gemm", 4096, 32, 1, 8, 128, N=4096, H=7168, train=False),
        # The gradients of a product over 64 unevenly loaded experts, the
        # input's and the weights', with an odd width.
        _rows("gemm_backward", "gemm", 8192, 64, 4, 6, 1, zipf=0.5, N=2048, H=1416, train=True),
        # One token through 4-bit experts (256 of them, 8 read).
        _rows("nvfp4_token", "nvfp4", 1, 256, 8, 8, 16, N=4096, H=7168),
        # A decode step of 64 sequences through 4-bit experts.
        _rows("nvfp4_decode", "nvfp4", 64, 64, 8, 8, 16, shared=1, N=4096, H=7168),
        # A short prompt through the second product's 4-bit weights.
        _rows("nvfp4_prompt", "nvfp4", 512, 32, 1, 8, 16, unused=0.05, N=7168, H=2048),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    kind = rng.choice(["route", "route", "swiglu", "gemm", "gemm", "nvfp4", "nvfp4"])
    if kind == "route":
        per, groups = rng.choice([(4, 16), (8, 8), (32, 8), (37, 1), (64, 1), (128, 1), (60, 4)])
        E = per * groups
        T = _log(rng, 1, min(65536, (1 << 22) // E))
        top_groups = rng.randint(1, groups)
        K = rng.randint(1, min(8, top_groups * per))
        score = rng.choice(["softmax", "sigmoid"])
        c = _route("", T, E, K, score, rng.random() < 0.5, groups, top_groups, rng.random() < 0.5,
                   rng.choice([1.0, 2.5]), rng.choice(["float32", "bfloat16"]), rng.random() < 0.6,
                   rng.choice([0.0, 0.04]))
        del c["name"]
        return c
    S = rng.choice([1, 2, 4])
    E = S * rng.choice([4, 8, 16])
    common = dict(E=E, S=S, K=rng.randint(1, min(8, E)), A=rng.choice([1, 16, 128]), shared=rng.choice([0, 0, 1]),
                  zipf=rng.choice([0.0, 0.0, 1.2]), unused=rng.choice([0.0, 0.05]))
    if kind == "swiglu":
        c = _rows("", kind, _log(rng, 1, 8192), I=_log(rng, 64, 2048, 8), train=rng.random() < 0.6, **common)
    else:
        step = 16 if kind == "nvfp4" else 8
        train = kind == "gemm" and rng.random() < 0.5
        T = _log(rng, 1, 512 if kind == "nvfp4" else 4096)
        N, H = _log(rng, 128, 4096, step), _log(rng, 128, 4096, step)
        while T > 1 and 2.0 * T * (common["K"] + common["shared"]) * N * H * (2 if train else 1) > 1.5e12:
            T //= 2
        c = _rows("", kind, T, N=N, H=H, **common)
        if kind == "gemm":
            c["train"] = train
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    """Normal values, rounded to dtype (drawn in it: the large weights' inputs are made many times)."""
    return torch.empty(*shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _topk_ids(case, g):
    """K distinct experts for every token, uniform or Zipf-weighted (the K
    largest of log-weights plus Gumbel noise), some slots unused (-1)."""
    T, E, K = case["T"], case["E"], case["K"]
    u = torch.rand(T, E, generator=g, device=DEV, dtype=torch.float64).clamp_min(1e-300)
    keys = -torch.log(-torch.log(u)) - case["zipf"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float64))
    ids = torch.argsort(keys, dim=1, descending=True)[:, :K]
    drop = torch.rand(T, K, generator=g, device=DEV) < case["unused"]
    return torch.where(drop, torch.full_like(ids, -1), ids)


def _layout(case, ids):
    """The receive layout of these ids: segment s holds experts [s*E/S,
    (s+1)*E/S), each group's rows in slot order and padded to a multiple of
    A; a shared expert is group 0 and gets every token's last slot in segment
    0; past `capacity` rows of a segment slots are dropped."""
    T, E, S, K, A, sh, C = (case[k] for k in ("T", "E", "S", "K", "A", "shared", "capacity"))
    G, Kp = E // S + sh, K + sh
    per = E // S
    group = torch.where(ids >= 0, (ids // per) * G + sh + ids % per, torch.full_like(ids, -1))
    expert = ids
    if sh:
        group = torch.cat([group, torch.zeros(T, 1, dtype=group.dtype, device=DEV)], 1)
        expert = torch.cat([ids, torch.full((T, 1), E, dtype=ids.dtype, device=DEV)], 1)
    group, expert = group.reshape(-1), expert.reshape(-1)
    counts = torch.bincount(group[group >= 0], minlength=S * G)
    aligned = ((counts + A - 1) // A * A).view(S, G)
    offs = torch.cat([torch.zeros(S, 1, dtype=torch.int64, device=DEV), aligned.cumsum(1)], 1)
    if C:
        base = torch.arange(S + 1, device=DEV) * C
    else:
        base = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), offs[:, -1].cumsum(0)])
    order = torch.argsort(torch.where(group >= 0, group, S * G), stable=True)
    order = order[: int(counts.sum())]
    first = torch.cumsum(counts, 0) - counts
    rank = torch.arange(order.numel(), device=DEV) - first[group[order]]
    in_seg = offs[:, :-1].reshape(-1)[group[order]] + rank
    rows = base[group[order] // G] + in_seg
    if C:
        kept = in_seg < C
        order, rows = order[kept], rows[kept]
    recv_rows = S * C if C else T * Kp + min(T * Kp, E + sh) * (A - 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    token_row = torch.full((T * Kp,), -1, **i32)
    token_row[order] = rows.int()
    expert_ids = torch.full((recv_rows,), -1, **i32)
    expert_ids[rows] = expert[order].int()
    src_info = torch.full((recv_rows, 2), -1, **i32)
    src_info[rows] = torch.stack([order // Kp, order % Kp], 1).int()
    offs = offs.clamp_max(C) if C else offs
    dropped = int(order.numel() < int(counts.sum()))
    layout = {"counts": counts.view(S, G).int(), "seg_base": base.int(), "row_offsets": offs.int(),
              "scales_offsets": offs.int(), "token_row": token_row.view(T, Kp), "expert_ids": expert_ids,
              "src_info": src_info, "flags": torch.full((1,), dropped, **i32)}
    return recv_rows, layout


def _experts(layout):
    """What the plain products go by: the experts that have rows, [U], and
    the rows of each, [U, most rows of one], -1 past its last."""
    e = layout["expert_ids"].long()
    rows = (e >= 0).nonzero().view(-1)
    rows = rows[torch.argsort(e[rows], stable=True)]
    used, slot, n = torch.unique_consecutive(e[rows], return_inverse=True, return_counts=True)
    at = torch.arange(rows.numel(), device=DEV) - (n.cumsum(0) - n)[slot]
    table = torch.full((max(1, used.numel()), max(1, int(n.max()) if n.numel() else 1)), -1, dtype=torch.int64, device=DEV)
    table[slot, at] = rows
    return (used if used.numel() else torch.zeros(1, dtype=torch.int64, device=DEV)), table


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    T, E, K = case["T"], case["E"], case["K"]
    if case["kind"] == "route":
        dt = getattr(torch, case["dtype"])
        st["logits"] = _normal(g, T, E, dtype=torch.float32, std=1.5).to(dt)
        st["bias"] = _normal(g, E, dtype=torch.float32, std=0.05) if case["biased"] else None
        st["mask"] = (torch.rand(T, generator=g, device=DEV) >= case["masked"]).to(torch.uint8) if case["masked"] else None
        st["topk_ids"] = torch.zeros(T, K, dtype=torch.int32, device=DEV)
        st["probs"] = torch.zeros(T, K, dtype=torch.float32, device=DEV)
        if case["train"]:
            st["grad_probs"] = _normal(g, T, K, dtype=torch.float32)
            st["grad_logits"] = torch.zeros(T, E, dtype=dt, device=DEV)
        return st
    R, st["layout"] = _layout(case, _topk_ids(case, g))
    experts = E + case["shared"]
    st["cfg"] = dict(num_tokens=T, hidden=case.get("H", 16), num_experts=E, num_segments=case["S"], top_k=K,
                     align=case["A"], seg_capacity=case["capacity"], shared_expert=case["shared"], recv_rows=R)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    if case["kind"] == "swiglu":
        I = case["I"]
        st["h"] = _normal(g, R, 2 * I)
        st["probs"] = torch.rand(T, K, generator=g, device=DEV)
        st["act"] = torch.zeros(R, I, **bf)
        if case["train"]:
            st["grad_act"] = _normal(g, R, I)
            st["grad_h"] = torch.zeros(R, 2 * I, **bf)
            st["grad_probs"] = torch.zeros(T, K, dtype=torch.float32, device=DEV)
        return st
    N, H = case["N"], case["H"]
    st["plan"] = _experts(st["layout"])
    if case["kind"] == "gemm":
        st["w"] = _normal(g, experts, N, H, std=H ** -0.5)
        st["x"] = _normal(g, R, H)
        if case["train"]:
            st["grad_y"] = _normal(g, R, N)
            st["grad_x"] = torch.zeros(R, H, **bf)
            st["grad_w"] = torch.zeros(experts, N, H, **bf)
        else:
            st["y"] = torch.zeros(R, N, **bf)
        return st
    # 4-bit weights: E2M1 codes of all values, E4M3 block scales in [1, 448],
    # a factor for each row that brings the outputs to about 1.
    st["codes"] = torch.randint(0, 256, (experts, N, H // 2), generator=g, device=DEV, dtype=torch.uint8)
    st["scales"] = torch.randint(0x38, 0x7F, (experts, N, H // 16), generator=g, device=DEV, dtype=torch.uint8)
    st["rowscale"] = ((0.5 + torch.rand(experts, N, generator=g, device=DEV)) * (2.5e-3 * H ** -0.5)).to(torch.bfloat16)
    st["x"] = _normal(g, R, H)
    st["y"] = torch.zeros(R, N, **bf)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _plain_route(st):
    c = st["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    low = -math.inf
    # Scores in 64 bits: the choice hangs on the order of close values.
    z = st["logits"].double()
    e = torch.exp(z - z.amax(1, keepdim=True))
    s = e / e.sum(1, keepdim=True) if c["score"] == "softmax" else 1 / (1 + torch.exp(-z))
    # Without a bias the order is the logits' own.
    key = s + st["bias"].double() if c["biased"] else z
    if G > 1:
        grouped = key.view(T, G, E // G)
        best = torch.sort(grouped, dim=2, descending=True)[0]
        of_group = best[..., :2].sum(2) if c["biased"] else best[..., 0]
        first = torch.sort(of_group, dim=1, descending=True, stable=True)[1][:, : c["top_groups"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, first, True)
        key = torch.where(kept[:, :, None], grouped, low).reshape(T, E)
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :K]
    chosen = s.gather(1, ids)
    total = chosen.sum(1, keepdim=True) + TINY
    p = c["scale"] * (chosen / total if c["normalize"] else chosen)
    out = [ids.int(), p.float()]
    on = torch.ones(T, 1, dtype=torch.bool, device=DEV) if st["mask"] is None else st["mask"].bool()[:, None]
    out = [torch.where(on, out[0], torch.full_like(out[0], -1)), torch.where(on, out[1], torch.zeros_like(out[1]))]
    if c["train"]:
        gp = st["grad_probs"].double() * c["scale"]
        if c["normalize"]:
            gp = (gp - (gp * chosen).sum(1, keepdim=True) / total) / total
        gs = torch.zeros_like(s).scatter_(1, ids, gp)
        if c["score"] == "softmax":
            gz = s * (gs - (gs * s).sum(1, keepdim=True))
        else:
            gz = gs * s * (1 - s)
        out.append(torch.where(on, gz, torch.zeros_like(gz)).to(st["logits"].dtype))
    return out


def _slots(st):
    """Rows, tokens and weights of the kept slots (weight 1 in the shared slot)."""
    token_row = st["layout"]["token_row"]
    T, Kp = token_row.shape
    w = torch.ones(T, Kp, device=DEV)
    w[:, : st["case"]["K"]] = st["probs"]
    at = (token_row.view(-1) >= 0).nonzero().view(-1)
    return token_row.view(-1)[at].long(), at, w.view(-1)[at]


def _plain_swiglu(st):
    c = st["case"]
    I, K, sh = c["I"], c["K"], c["shared"]
    rows, at, w = _slots(st)
    h = st["h"][rows].float()
    a, b = h[:, :I], h[:, I:]
    sig = 1 / (1 + torch.exp(-a))
    st["act"][rows] = (w[:, None] * (a * sig * b)).to(torch.bfloat16)
    if not c["train"]:
        return [st["act"]]
    ga = st["grad_act"][rows].float()
    gw = torch.zeros(c["T"] * (K + sh), device=DEV)
    gw[at] = (ga * (a * sig * b)).sum(1)
    st["grad_probs"].copy_(gw.view(c["T"], K + sh)[:, :K])
    ga = ga * w[:, None]
    st["grad_h"][rows] = torch.cat([ga * b * (sig * (1 + a * (1 - sig))), ga * (a * sig)], 1).to(torch.bfloat16)
    return [st["act"], st["grad_h"], st["grad_probs"]]


def _padded(rows, table):
    """rows [R, C] -> fp32 [U, M, C], zero past each expert's last row."""
    return torch.where((table >= 0)[:, :, None], rows[table.clamp_min(0)].float(), 0.0)


def _put(out, table, values):
    on = table >= 0
    out[table[on]] = values[on].to(out.dtype)
    return out


def _plain_gemm(st):
    used, table = st["plan"]
    w = st["w"][used].float()
    if not st["case"]["train"]:
        return [_put(st["y"], table, torch.bmm(_padded(st["x"], table), w.transpose(1, 2)))]
    gy = _padded(st["grad_y"], table)
    _put(st["grad_x"], table, torch.bmm(gy, w))
    st["grad_w"].zero_()
    st["grad_w"][used] = torch.bmm(gy.transpose(1, 2), _padded(st["x"], table)).to(torch.bfloat16)
    return [st["grad_x"], st["grad_w"]]


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _plain_nvfp4(st):
    used, table = st["plan"]
    N, H = st["case"]["N"], st["case"]["H"]
    value = torch.tensor(E2M1, device=DEV)
    byte = torch.arange(256, device=DEV)
    pairs = torch.stack([value[byte % 16], value[byte // 16]], 1)
    v = pairs[st["codes"][used].int()].view(-1, N, H // 16, 16)
    scale = st["scales"][used].view(torch.float8_e4m3fn).float() * st["rowscale"][used].float()[:, :, None]
    w = (v * scale[..., None]).view(-1, N, H)
    return [_put(st["y"], table, torch.bmm(_padded(st["x"], table), w.transpose(1, 2)))]


# ---------------------------------------------------------------------------
# The library's kernels
# ---------------------------------------------------------------------------
def _own(st):
    import combine_ep_dispatch_amd as epx

    c = st["case"]
    if c["kind"] == "route":
        cfg = epx.EpConfig(num_tokens=c["T"], hidden=16, num_experts=c["E"], num_segments=1, top_k=c["K"])
        route = epx.RouteConfig(score=c["score"], normalize=c["normalize"], num_groups=c["groups"],
                                top_groups=c["top_groups"], scale=c["scale"])
        epx.ep_route(cfg, route, st["logits"], st["topk_ids"], st["probs"], bias=st["bias"], token_mask=st["mask"])
        if not c["train"]:
            return [st["topk_ids"], st["probs"]]
        epx.ep_route_bwd(cfg, route, st["logits"], st["topk_ids"], st["grad_probs"], st["grad_logits"])
        return [st["topk_ids"], st["probs"], st["grad_logits"]]
    cfg, layout = epx.EpConfig(**st["cfg"]), epx.Layout(**st["layout"])
    if c["kind"] == "swiglu":
        epx.ep_swiglu(cfg, layout, st["h"], st["probs"], st["act"])
        if not c["train"]:
            return [st["act"]]
        epx.ep_swiglu_bwd(cfg, layout, st["h"], st["probs"], st["grad_act"], st["grad_h"], st["grad_probs"])
        return [st["act"], st["grad_h"], st["grad_probs"]]
    if c["kind"] == "nvfp4":
        epx.ep_expert_gemm_nvfp4(cfg, layout, st["x"], st["codes"], st["scales"], st["rowscale"], st["y"])
        return [st["y"]]
    if not c["train"]:
        epx.ep_expert_gemm(cfg, layout, st["x"], st["w"], st["y"])
        return [st["y"]]
    epx.ep_expert_gemm_bwd_x(cfg, layout, st["grad_y"], st["w"], st["grad_x"])
    epx.ep_expert_gemm_bwd_w(cfg, layout, st["grad_y"], st["x"], st["grad_w"])
    return [st["grad_x"], st["grad_w"]]


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "swiglu": _plain_swiglu, "gemm": _plain_gemm,
            "nvfp4": _plain_nvfp4}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    T, E, K = case["T"], case["E"], case["K"]
    if case["kind"] == "route":
        size = 4 if case["dtype"] == "float32" else 2
        n = T * E * size + T * K * 8
        if case["train"]:  # the gradient reads the logits again only if it runs on its own: counted once
            n += T * E * size + T * K * 4
        return {"bytes": n, "flops": T * E * 10 * (2 if case["train"] else 1)}
    rows = T * K * (1 - case["unused"]) + T * case["shared"]
    if case["capacity"]:
        rows = min(rows, case["S"] * case["capacity"])
    if case["kind"] == "swiglu":
        I = case["I"]
        n = rows * (3 * I * 2 + 8) + (rows * (3 * I * 2 + 4) if case["train"] else 0)
        return {"bytes": n, "flops": rows * I * (20 if case["train"] else 8)}
    N, H = case["N"], case["H"]
    # experts that get a row, on average, where the routing is uniform
    hit = E * (1 - (1 - K / E * (1 - case["unused"])) ** T) + case["shared"]
    weight = 0.5625 if case["kind"] == "nvfp4" else 2.0
    if case["kind"] == "gemm" and case["train"]:
        return {"bytes": hit * N * H * 4 + rows * (N + 2 * H) * 2, "flops": 4.0 * rows * N * H}
    return {"bytes": hit * N * H * weight + rows * (N + H) * 2, "flops": 2.0 * rows * N * H}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(st):
    import numpy as np

    c = st["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    z = st["logits"].double().cpu().numpy()
    if c["score"] == "softmax":
        s = np.exp(z - np.logaddexp.reduce(z, axis=1)[:, None])
    else:
        s = np.exp(-np.logaddexp(0.0, -z))
    key = z.copy()
    if c["biased"]:
        key = s + st["bias"].double().cpu().numpy()
    if G > 1:
        part = np.sort(key.reshape(T, G, -1), axis=2)
        of_group = part[..., -2:].sum(2) if c["biased"] else part[..., -1]
        order = np.argsort(-of_group, axis=1, kind="stable")[:, : c["top_groups"]]
        out = np.ones((T, G), bool)
        np.put_along_axis(out, order, False, 1)
        key[np.repeat(out, E // G, axis=1)] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :K]
    top = np.take_along_axis(s, ids, 1)
    total = top.sum(1, keepdims=True) + TINY
    p = c["scale"] * (top / total if c["normalize"] else top)
    on = np.ones((T, 1), bool) if st["mask"] is None else st["mask"].cpu().numpy()[:, None] != 0
    got = [np.where(on, ids, -1).astype(np.int32), np.where(on, p, 0.0)]
    if c["train"]:
        # d p_j / d s_i, then d s / d z
        gp = st["grad_probs"].double().cpu().numpy() * c["scale"]
        if c["normalize"]:
            gp = gp / total - (gp * top).sum(1, keepdims=True) / total ** 2
        if c["score"] == "softmax":
            gz = -s * (gp * top).sum(1, keepdims=True)
            np.put_along_axis(gz, ids, np.take_along_axis(gz, ids, 1) + gp * top, 1)
        else:
            gz = np.zeros((T, E))
            np.put_along_axis(gz, ids, gp * top * np.take_along_axis(1 / (1 + np.exp(z)), ids, 1), 1)
        got.append(np.where(on, gz, 0.0))
    return got


def _exact_swiglu(st):
    c = st["case"]
    I, T, K = c["I"], c["T"], c["K"]
    R = st["h"].shape[0]
    src = st["layout"]["src_info"].long()
    used = src[:, 0] >= 0
    w = torch.cat([st["probs"].double(), torch.ones(T, 1, dtype=torch.float64, device=DEV)], 1)
    w = torch.where(used, w[src[:, 0], src[:, 1]], 0.0)[:, None]
    gate, up = st["h"].double().chunk(2, 1)
    silu = gate * torch.sigmoid(gate)
    got = [w * silu * up]
    if c["train"]:
        ga = torch.where(used[:, None], st["grad_act"].double(), 0.0)
        slope = torch.sigmoid(gate) + silu * torch.sigmoid(-gate)
        got.append(torch.cat([w * ga * up * slope, w * ga * silu], 1))
        gw = torch.zeros(T, K + 1, dtype=torch.float64, device=DEV)
        gw[src[used, 0], src[used, 1]] = (ga * silu * up).sum(1)[used]
        got.append(gw[:, :K])
    return got


def _exact_products(st, weight):
    e = st["layout"]["expert_ids"]
    train = st["case"].get("train", False)
    if train:
        gx, gw = torch.zeros_like(st["grad_x"], dtype=torch.float64), torch.zeros_like(st["grad_w"], dtype=torch.float64)
    else:
        y = torch.zeros_like(st["y"], dtype=torch.float64)
    for i in torch.unique(e[e >= 0]).tolist():
        rows = (e == i).nonzero().view(-1)
        w, x = weight(i), st["x"][rows].double()
        if train:
            gy = st["grad_y"][rows].double()
            gx[rows] = gy @ w
            gw[i] = gy.T @ x
        else:
            y[rows] = x @ w.T
    return [gx, gw] if train else [y]


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "route":
        return _exact_route(st)
    if case["kind"] == "swiglu":
        return _exact_swiglu(st)
    if case["kind"] == "gemm":
        return _exact_products(st, lambda i: st["w"][i].double())

    def weight(i):
        c = st["codes"][i].to(torch.int64)
        c = torch.stack([c & 15, c >> 4], 2).view(case["N"], case["H"])
        ex, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((ex - 1).double())) * (1 - 2 * (c >> 3)).double()
        s = st["scales"][i].to(torch.int64)
        b = torch.where(s < 8, s.double() / 512, (1 + (s & 7).double() / 8) * torch.exp2(((s >> 3) - 7).double()))
        return v * b.repeat_interleave(16, 1) * st["rowscale"][i].double()[:, None]

    return _exact_products(st, weight)
