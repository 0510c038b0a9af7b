"""Cases and plain forms of the expert layer's gated block (both projections,
the activation and the routing weight in one product, with its backward pass)
and of the low-rank adapters of many requests beside the experts' products.

`run` computes a case with elementary torch operations, or, where `own` is
true, with the library's kernels; both take what `prepare` made.  Rows of a
receive-side buffer that no token owns (pad rows, rows past a segment's used
rows) are zero in the buffers `prepare` allocates and stay as they are.
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(name, kind, weights, T, E, S, K, A, N, H, train=False, gated=True, rank=0, adapters=0, packed=True, bare=0.0,
          shared=0, capacity=0, zipf=0.0, unused=0.0):
    """kind "gated" or "adapters"; weights "bf16" or "nvfp4"; N x H: an expert's
    weights (N = gate and up together where gated); adapters of `rank`, whose
    tokens come packed request by request or mixed, a share `bare` of them
    without an adapter."""
    return {"name": name, "kind": kind, "weights": weights, "T": T, "E": E, "S": S, "K": K, "A": A, "N": N, "H": H,
            "train": train, "gated": gated, "rank": rank, "adapters": adapters, "packed": packed, "bare": bare,
            "shared": shared, "capacity": capacity, "zipf": zipf, "unused": unused}


def listed():
    return [
        # One token through 4-bit experts' gated block (256 experts, 8 read):
        # latency, and one read of 8 experts' weights.
        _case("gated_token", "gated", "nvfp4", 1, 256, 8, 8, 16, 4096, 7168),
        # A decode step of 16 sequences, bf16 weights, one segment's 32 experts.
        _case("gated_decode", "gated", "bf16", 16, 32, 1, 8, 128, 4096, 7168),
        # A decode step of 64 sequences through 4-bit experts and a shared one.
        _case("gated_decode_nvfp4", "gated", "nvfp4", 64, 64, 8, 8, 16, 4096, 7168, shared=1),
        # A short prompt through 4-bit experts, some slots unused.
        _case("gated_prompt_nvfp4", "gated", "nvfp4", 512, 32, 1, 8, 16, 4096, 7168, unused=0.05),
        # The forward pass of a training step, or a long prompt: 1024 rows an expert.
        _case("gated_prefill", "gated", "bf16", 4096, 32, 1, 8, 128, 4096, 7168),
        # A whole training step of the block, forward and all gradients, over
        # unevenly loaded experts of an odd width.
        _case("gated_train", "gated", "bf16", 8192, 64, 4, 6, 1, 2048, 1416, train=True, zipf=0.5),
        # The capacity workload: skewed routing, dropped slots, narrow experts.
        _case("gated_capacity", "gated", "bf16", 16384, 64, 4, 6, 1, 1040, 1024, train=True, capacity=27036, zipf=1.5),
        # A decode step of 16 sequences, each with an adapter of its own among
        # 16, some without, beside the first product's bf16 weights.
        _case("adapters_decode", "adapters", "bf16", 16, 32, 1, 8, 128, 4096, 7168, gated=False, rank=16, adapters=16,
              packed=False, bare=0.1),
        # 64 sequences of 8 adapters over 4-bit experts, in the gated block.
        _case("adapters_decode_nvfp4", "adapters", "nvfp4", 64, 64, 8, 8, 16, 4096, 7168, rank=16, adapters=8,
              packed=False, bare=0.25),
        # Prompts of several requests packed behind one another, in the gated block.
        _case("adapters_prefill", "adapters", "bf16", 4096, 32, 1, 8, 128, 4096, 7168, rank=32, adapters=8, bare=0.2),
        # A batch of short prompts with every token's adapter another one, a
        # large rank and an odd width.
        _case("adapters_mixed", "adapters", "bf16", 1023, 16, 2, 4, 1, 2048, 1416, gated=False, rank=64, adapters=5,
              packed=False, bare=0.1),
        # A training step of 4 adapters over frozen experts: the product, its
        # input's gradient and the adapters'.
        _case("adapters_train", "adapters", "bf16", 4096, 32, 1, 8, 128, 2048, 2048, gated=False, train=True, rank=16,
              adapters=4, bare=0.05),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    kind = rng.choice(["gated", "gated", "adapters"])
    weights = rng.choice(["bf16", "bf16", "nvfp4"])
    gated = kind == "gated" or rng.random() < 0.5
    train = weights == "bf16" and rng.random() < 0.5 and not (kind == "adapters" and gated)
    S = rng.choice([1, 2, 4])
    E = S * rng.choice([4, 8, 16])
    K = rng.randint(1, min(8, E))
    shared = rng.choice([0, 0, 1])
    step = 16 if weights == "nvfp4" else 8
    T = _log(rng, 1, 512 if weights == "nvfp4" else 4096)
    N, H = 2 * _log(rng, 64, 2048, step), _log(rng, 128, 4096, step)
    while T > 1 and 2.0 * T * (K + shared) * N * H * (3 if train else 1) > 1.5e12:
        T //= 2
    lora = {}
    if kind == "adapters":
        lora = dict(rank=rng.choice([8, 16, 16, 24, 32, 64, 128]), adapters=rng.choice([1, 3, 8, 16]),
                    packed=rng.random() < 0.6, bare=rng.choice([0.0, 0.2]))
    c = _case("", kind, weights, T, E, S, K, rng.choice([1, 16, 128]), N, H, train=train, gated=gated, shared=shared,
              zipf=rng.choice([0.0, 0.0, 1.2]), unused=rng.choice([0.0, 0.05]), **lora)
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


def _token_adapter(case, g):
    """The adapter of every token, -1 for none: requests packed behind one
    another (of 1 to 2 T / adapters tokens), or every token by itself."""
    T, n = case["T"], case["adapters"]
    if case["packed"]:
        ends = torch.randint(1, max(2, 2 * T // n), (T,), generator=g, device=DEV).cumsum(0)
        request = torch.searchsorted(ends, torch.arange(T, device=DEV), right=True)
        of = torch.randint(0, n, (T,), generator=g, device=DEV)
        bare = torch.rand(T, generator=g, device=DEV) < case["bare"]
        return torch.where(bare, -1, of)[request].int()
    of = torch.randint(0, n, (T,), generator=g, device=DEV)
    return torch.where(torch.rand(T, generator=g, device=DEV) < case["bare"], -1, of).int()


def _grouped(keys):
    """What the plain products go by: the keys >= 0 that rows have, [U], and
    the rows of each, [U, most rows of one], -1 past its last."""
    rows = (keys >= 0).nonzero().view(-1)
    rows = rows[torch.argsort(keys[rows], stable=True)]
    used, slot, n = torch.unique_consecutive(keys[rows], return_inverse=True, return_counts=True)
    at = torch.arange(rows.numel(), device=DEV) - (n.cumsum(0) - n)[slot]
    table = torch.full((max(1, used.numel()), max(1, int(n.max()) if n.numel() else 1)), -1, dtype=torch.int64, device=DEV)
    table[slot, at] = rows
    return (used if used.numel() else torch.zeros(1, dtype=torch.int64, device=DEV)), table


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    T, E, K, N, H = (case[k] for k in ("T", "E", "K", "N", "H"))
    R, st["layout"] = _layout(case, _topk_ids(case, g))
    experts = E + case["shared"]
    st["cfg"] = dict(num_tokens=T, hidden=H, num_experts=E, num_segments=case["S"], top_k=K, align=case["A"],
                     seg_capacity=case["capacity"], shared_expert=case["shared"], recv_rows=R)
    bf, f32 = dict(dtype=torch.bfloat16, device=DEV), dict(dtype=torch.float32, device=DEV)
    expert = st["layout"]["expert_ids"].long()
    st["plan"] = _grouped(expert)
    if case["weights"] == "bf16":
        st["w"] = _normal(g, experts, N, H, std=H ** -0.5)
    else:
        # 4-bit weights: E2M1 codes of all values, E4M3 block scales in [1,
        # 448], a factor for each row that brings the outputs to about 1.
        st["codes"] = torch.randint(0, 256, (experts, N, H // 2), generator=g, device=DEV, dtype=torch.uint8)
        st["scales"] = torch.randint(0x38, 0x7F, (experts, N, H // 16), generator=g, device=DEV, dtype=torch.uint8)
        st["rowscale"] = ((0.5 + torch.rand(experts, N, generator=g, device=DEV)) * (2.5e-3 * H ** -0.5)).to(torch.bfloat16)
    st["x"] = _normal(g, R, H)
    st["probs"] = torch.rand(T, K, generator=g, device=DEV)
    out = N // 2 if case["gated"] else N
    st["out"] = torch.zeros(R, out, **bf)
    if case["rank"]:
        n, rank = case["adapters"], case["rank"]
        st["token_adapter"] = _token_adapter(case, g)
        st["a"] = _normal(g, n, experts, rank, H, std=H ** -0.5)
        st["b"] = _normal(g, n, experts, N, rank, std=0.5 * rank ** -0.5)
        st["scale"] = 0.5 + torch.rand(n, generator=g, device=DEV)
        st["u"] = torch.zeros(R, rank, **f32)
        token = st["layout"]["src_info"][:, 0].long()
        adapter = torch.where(token >= 0, st["token_adapter"].long()[token.clamp_min(0)], -1)
        st["pairs"] = _grouped(torch.where((expert >= 0) & (adapter >= 0), expert * n + adapter, -1))
    if case["train"]:
        st["grad_out"] = _normal(g, R, out)
        st["grad_x"] = torch.zeros(R, H, **bf)
        if case["rank"]:
            st["grad_u"] = torch.zeros(R, rank, **f32)
            st["grad_a"], st["grad_b"] = torch.zeros(n, experts, rank, H, **f32), torch.zeros(n, experts, N, rank, **f32)
        else:
            st["grad_h"] = torch.zeros(R, N, **bf)
            st["grad_w"] = torch.zeros(experts, N, H, **bf)
            st["grad_probs"] = torch.zeros(T, K, **f32)
            st["workspace"] = torch.zeros(T * K * (-(-out // 32)) * 4, dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _padded(rows, table):
    """rows [R, C] -> fp32 [U, M, C], zero past each key's last row."""
    return torch.where((table >= 0)[:, :, None], rows[table.clamp_min(0)].float(), 0.0)


def _weights_of(st, used):
    """The used experts' weights in fp32, [U, N, H]."""
    if "w" in st:
        return st["w"][used].float()
    N, H = st["case"]["N"], st["case"]["H"]
    value = torch.tensor(E2M1, device=DEV)
    byte = torch.arange(256, device=DEV)
    pairs = torch.stack([value[byte % 16], value[byte // 16]], 1)
    v = pairs[st["codes"][used].int()].view(-1, N, H // 16, 16)
    scale = st["scales"][used].view(torch.float8_e4m3fn).float() * st["rowscale"][used].float()[:, :, None]
    return (v * scale[..., None]).view(-1, N, H)


def _adapters_of(st):
    """Of the used pairs: A and B in fp32, the scale [U, 1, 1], and adapter and expert."""
    used, _ = st["pairs"]
    n = st["case"]["adapters"]
    ad, e = used % n, used // n
    return st["a"][ad, e].float(), st["b"][ad, e].float(), st["scale"][ad][:, None, None], ad, e


def _row_weights(st):
    """Every receive row's routing weight, [R, 1] (1 in the shared slot), its token and its slot (K: shared)."""
    T, K = st["case"]["T"], st["case"]["K"]
    token, slot = st["layout"]["src_info"].long().unbind(1)
    w = torch.cat([st["probs"], torch.ones(T, 1, device=DEV)], 1)
    return w[token.clamp_min(0), slot.clamp(0, K)][:, None], token, slot


def _plain(st):
    c = st["case"]
    used, table = st["plan"]
    on = table >= 0
    rows = table[on]
    weights = _weights_of(st, used)
    # every row's product, unrounded
    h = torch.zeros(st["x"].shape[0], c["N"], device=DEV)
    h[rows] = torch.bmm(_padded(st["x"], table), weights.transpose(1, 2))[on]
    if c["rank"]:
        pairs = st["pairs"][1]
        pon = pairs >= 0
        prows = pairs[pon]
        a, b, scale, ad, e = _adapters_of(st)
        px = _padded(st["x"], pairs)
        u = scale * torch.bmm(px, a.transpose(1, 2))
        h[prows] += torch.bmm(u, b.transpose(1, 2))[pon]
    if not c["gated"]:
        st["out"][rows] = h[rows].to(torch.bfloat16)
        if not c["train"]:
            return [st["out"]]
        gx = torch.zeros(st["x"].shape, dtype=torch.float32, device=DEV)
        gx[rows] = torch.bmm(_padded(st["grad_out"], table), weights)[on]
        pg = _padded(st["grad_out"], pairs)
        gu = scale * torch.bmm(pg, b)
        gx[prows] += torch.bmm(gu, a)[pon]
        st["grad_x"][rows] = gx[rows].to(torch.bfloat16)
        st["grad_a"].zero_()
        st["grad_b"].zero_()
        st["grad_a"][ad, e] = torch.bmm(gu.transpose(1, 2), px)
        st["grad_b"][ad, e] = torch.bmm(pg.transpose(1, 2), u)
        return [st["out"], st["grad_x"], st["grad_a"], st["grad_b"]]
    w, token, slot = _row_weights(st)
    gate, up = h[rows].chunk(2, 1)
    sig = 1 / (1 + torch.exp(-gate))
    st["out"][rows] = (w[rows] * (gate * sig * up)).to(torch.bfloat16)
    if not c["train"]:
        return [st["out"]]
    ga = st["grad_out"][rows].float()
    gw = torch.zeros(c["T"], c["K"] + 1, device=DEV)
    gw[token[rows], slot[rows]] = (ga * (gate * sig * up)).sum(1)
    st["grad_probs"].copy_(gw[:, : c["K"]])
    ga = ga * w[rows]
    h[rows] = torch.cat([ga * up * (sig * (1 + gate * (1 - sig))), ga * (gate * sig)], 1)
    gh = _padded(h, table)
    st["grad_x"][rows] = torch.bmm(gh, weights)[on].to(torch.bfloat16)
    st["grad_w"].zero_()
    st["grad_w"][used] = torch.bmm(gh.transpose(1, 2), _padded(st["x"], table)).to(torch.bfloat16)
    return [st["out"], st["grad_x"], st["grad_w"], st["grad_probs"]]


# ---------------------------------------------------------------------------
# The library's kernels
# ---------------------------------------------------------------------------
def _own(st):
    import combine_ep_dispatch_amd as epx

    c = st["case"]
    cfg, layout = epx.EpConfig(**st["cfg"]), epx.Layout(**st["layout"])
    lora = {}
    if c["rank"]:
        adapters = epx.Adapters(st["token_adapter"], st["a"], st["b"], st["scale"])
        epx.ep_lora_down(cfg, layout, st["x"], adapters, st["u"])
        lora = dict(adapters=adapters, u=st["u"])
    packed = (st["codes"], st["scales"], st["rowscale"]) if c["weights"] == "nvfp4" else None
    if c["gated"]:
        if packed:
            epx.ep_expert_gated_nvfp4(cfg, layout, st["x"], *packed, st["probs"], st["out"], **lora)
        else:
            epx.ep_expert_gated(cfg, layout, st["x"], st["w"], st["probs"], st["out"], **lora)
        if not c["train"]:
            return [st["out"]]
        epx.ep_expert_gated_bwd(cfg, layout, st["x"], st["w"], st["probs"], st["grad_out"], st["grad_h"],
                                grad_probs=st["grad_probs"], workspace=st["workspace"])
        epx.ep_expert_gemm_bwd_x(cfg, layout, st["grad_h"], st["w"], st["grad_x"])
        epx.ep_expert_gemm_bwd_w(cfg, layout, st["grad_h"], st["x"], st["grad_w"])
        return [st["out"], st["grad_x"], st["grad_w"], st["grad_probs"]]
    if packed:
        epx.ep_expert_gemm_nvfp4_lora(cfg, layout, st["x"], *packed, st["out"], **lora)
    else:
        epx.ep_expert_gemm_lora(cfg, layout, st["x"], st["w"], st["out"], **lora)
    if not c["train"]:
        return [st["out"]]
    epx.ep_lora_bwd_u(cfg, layout, st["grad_out"], adapters, st["grad_u"])
    epx.ep_expert_gemm_bwd_x_lora(cfg, layout, st["grad_out"], st["w"], st["grad_x"], adapters=adapters,
                                  grad_u=st["grad_u"])
    epx.ep_lora_bwd_w(cfg, layout, st["x"], st["grad_out"], adapters, st["u"], st["grad_u"], st["grad_a"], st["grad_b"])
    return [st["out"], st["grad_x"], st["grad_a"], st["grad_b"]]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    T, E, K, N, H = (case[k] for k in ("T", "E", "K", "N", "H"))
    rows = T * K * (1 - case["unused"]) + T * case["shared"]
    if case["capacity"]:
        rows = min(rows, case["S"] * case["capacity"])
    # experts that get a row, on average, where the routing is uniform
    hit = E * (1 - (1 - K / E * (1 - case["unused"])) ** T) + case["shared"]
    out = N // 2 if case["gated"] else N
    n = hit * N * H * (0.5625 if case["weights"] == "nvfp4" else 2.0) + rows * (H + out) * 2
    products, f = 1, 0.0
    if case["rank"]:
        with_adapter = rows * (1 - case["bare"])
        pairs = (E + case["shared"]) * case["adapters"]
        ab = pairs * (1 - math.exp(-with_adapter / pairs)) * case["rank"] * (H + N)
        n += ab * 2
        f += 2.0 * with_adapter * case["rank"] * (H + N) * (3 if case["train"] else 1)
        if case["train"]:
            n += rows * (out + H) * 2 + (E + case["shared"]) * case["adapters"] * case["rank"] * (H + N) * 4
            products = 2
    elif case["train"]:
        n += rows * (out + H) * 2 + T * K * 4 + (E + case["shared"]) * N * H * 2
        products = 3
    return {"bytes": n, "flops": f + 2.0 * products * rows * N * H}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_weights(st, i):
    if "w" in st:
        return st["w"][i].double()
    c = st["codes"][i].to(torch.int64)
    c = torch.stack([c & 15, c >> 4], 2).view(st["case"]["N"], st["case"]["H"])
    ex, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((ex - 1).double())) * (1 - 2 * (c >> 3)).double()
    s = st["scales"][i].to(torch.int64)
    b = torch.where(s < 8, s.double() / 512, (1 + (s & 7).double() / 8) * torch.exp2(((s >> 3) - 7).double()))
    return v * b.repeat_interleave(16, 1) * st["rowscale"][i].double()[:, None]


def exact(case, seed):
    st = prepare(case, seed)
    T, K, train = case["T"], case["K"], case["train"]
    f64 = dict(dtype=torch.float64, device=DEV)
    e, src = st["layout"]["expert_ids"], st["layout"]["src_info"].long()
    out = torch.zeros(st["out"].shape, **f64)
    if train:
        grad_x = torch.zeros(st["grad_x"].shape, **f64)
        sums = [torch.zeros(st[k].shape, **f64) for k in (("grad_a", "grad_b") if case["rank"] else ("grad_w", "grad_probs"))]
    for i in torch.unique(e[e >= 0]).tolist():
        rows = (e == i).nonzero().view(-1)
        weights, x = _exact_weights(st, i), st["x"][rows].double()
        h = x @ weights.T
        gy = st["grad_out"][rows].double() if train else None
        if train and case["rank"]:
            grad_x[rows] = gy @ weights
        if case["rank"]:
            of = st["token_adapter"].long()[src[rows, 0]]
            for k in torch.unique(of[of >= 0]).tolist():
                some = (of == k).nonzero().view(-1)
                a, b, s = st["a"][k, i].double(), st["b"][k, i].double(), st["scale"][k].double()
                change = s * (b @ a)
                h[some] += x[some] @ change.T
                if train:
                    grad_x[rows[some]] += gy[some] @ change
                    cross = s * (gy[some].T @ x[some])  # the gradient of the product b a
                    sums[0][k, i] = b.T @ cross
                    sums[1][k, i] = cross @ a.T
        if not case["gated"]:
            out[rows] = h
            continue
        slot = src[rows, 1]
        p = torch.where(slot < K, st["probs"].double()[src[rows, 0], slot.clamp_max(K - 1)], 1.0)[:, None]
        gate, up = h.chunk(2, 1)
        silu = gate * torch.sigmoid(gate)
        out[rows] = p * silu * up
        if train:
            slope = torch.sigmoid(gate) + silu * torch.sigmoid(-gate)
            gh = p * torch.cat([gy * up * slope, gy * silu], 1)
            grad_x[rows] = gh @ weights
            sums[0][i] = gh.T @ x
            routed = slot < K
            sums[1][src[rows, 0][routed], slot[routed]] = (gy * silu * up).sum(1)[routed]
    return [out, grad_x, *sums] if train else [out]
