"""Autograd wrappers over the C ABI, shaped after the forward/backward pairs
the NeMo AutoModel fused_a2a page documents (HybridEPDispatch: dispatch
forward, combine-of-gradients backward; HybridEPCombine: combine forward,
redispatch backward).

Marshalling only: every step runs in libepx's HIP kernels.

    d = EpDispatcher(cfg, device)            # owns layout, workspace, buffers
    recv = d.dispatch(x, topk_ids)           # [R, H] bf16, differentiable in x
    y = d.combine(expert_out, probs)         # [T, H] bf16, differentiable in
                                             # expert_out and probs
    y.backward(grad)                         # -> x.grad, expert_out.grad, probs.grad

dispatch() builds the layout (the "handle") in the same call as the
dispatch and keeps it for the combine and both backward passes; rows past a segment's used rows are left as the
buffers held them (zero for the buffers allocated here).  Every routing
gets a layout of its own, and each forward node keeps the layout it ran
with, so routing the next batch before this one's backward is safe.  The
routing is not differentiable; probs is, through the router-probability
gradient.

The expert layer around the two, on the same layout:

    topk_ids, probs = d.gate(logits, RouteConfig(...))   # differentiable in logits
    recv = d.dispatch(x, topk_ids)
    h = d.linear(recv, w1)                   # [R, 2 * inter], differentiable in both
    act = d.swiglu(h, probs)                 # weights applied to the rows; differentiable in both
    y = d.combine(d.linear(act, w2), None)

d.gated(recv, w1, probs) is d.swiglu(d.linear(recv, w1), probs) in one kernel that
keeps neither h nor act's inputs: its backward pass makes h again, which saves h's
memory and costs more time than keeping it (a step of 64 experts of 2048 x 1416, 49 152
rows: 1.57 ms, by the two 1.28 ms and 201 MB).  linear and gated
take Adapters (low-rank, a token's own each) beside the weights, differentiable in
rows, w, adapters.a and adapters.b (a scale that asks for a gradient is refused);
weights that need no gradient cost none.

A step can be captured into a graph, backward pass included, on leaves that no
eager autograd graph still holds (torch does not support capturing beside one).

The backward passes are library calls without gradients of their own: under
create_graph the first derivatives can be had, differentiating them raises.
"""

from __future__ import annotations

import functools
from typing import Optional

import torch

from . import (Adapters, EpConfig, Layout, RouteConfig, ep_combine, ep_combine_bwd, ep_combine_bwd_probs, ep_dispatch,
               ep_dispatch_bwd, ep_dispatch_layout, ep_dispatch_with_layout, ep_expert_gated, ep_expert_gated_bwd,
               ep_expert_gemm, ep_expert_gemm_bwd_w, ep_expert_gemm_bwd_x, ep_expert_gemm_bwd_x_lora,
               ep_expert_gemm_lora, ep_lora_bwd_u, ep_lora_bwd_w, ep_lora_down, ep_query, ep_route, ep_route_bwd,
               ep_swiglu, ep_swiglu_bwd, gated_workspace_for, workspace_for)

__all__ = ["EpDispatcher"]


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as the calls take it, contiguous and 16-byte aligned: itself or a copy (a
    slice of a batch, or of a flat buffer, may begin off 16 bytes)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _weights(probs: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if probs is None else probs.contiguous().float()


class _Refuse(torch.autograd.Function):
    """The first n tensors as they are, depending on all of them, with no way back."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("EpDispatcher's operators cannot be differentiated twice")


def _first_only(backward):
    """A backward pass whose results raise where they are differentiated.  They
    depend on the incoming gradients and the saved inputs, so that every path to
    a leaf meets the error (once_differentiable's leads nowhere: torch.autograd.grad
    passes it by where another term reaches the leaf)."""

    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        sources = [t for t in (*grads, *ctx.saved_tensors) if t is not None and t.requires_grad]
        if not sources:
            return out
        given = [t for t in out if t is not None]
        refusing = iter(_Refuse.apply(len(given), *given, *sources))
        return tuple(None if t is None else next(refusing) for t in out)

    return wrapped


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, cfg, layout, topk_ids=None, workspace=None):
        # with topk_ids, the layout is built in the same call (one kernel for
        # decode-sized batches)
        recv = torch.zeros(cfg.recv_rows, cfg.hidden, dtype=torch.bfloat16, device=x.device)
        if topk_ids is None:
            ep_dispatch(cfg, layout, x.view(-1), recv.view(-1))
        else:
            ep_dispatch_with_layout(cfg, topk_ids, workspace, layout, x.view(-1), recv.view(-1))
        ctx.cfg, ctx.layout = cfg, layout
        return recv

    @staticmethod
    @_first_only
    def backward(ctx, grad_recv):
        cfg = ctx.cfg
        gx = torch.empty(cfg.num_tokens, cfg.hidden, dtype=torch.bfloat16, device=grad_recv.device)
        ep_dispatch_bwd(cfg, ctx.layout, _rows(grad_recv.to(torch.bfloat16)).view(-1), gx.view(-1))
        return gx, None, None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, expert_out, probs, cfg, layout):
        y = torch.empty(cfg.num_tokens, cfg.hidden, dtype=torch.bfloat16, device=expert_out.device)
        ep_combine(cfg, layout, expert_out.view(-1), None if probs is None else probs.view(-1), y.view(-1))
        ctx.cfg, ctx.layout = cfg, layout
        ctx.has_probs = probs is not None
        ctx.save_for_backward(expert_out, probs if ctx.has_probs else torch.empty(0, device=expert_out.device))
        return y

    @staticmethod
    @_first_only
    def backward(ctx, grad_y):
        cfg, layout = ctx.cfg, ctx.layout
        eo, p = ctx.saved_tensors
        gy = _rows(grad_y.to(torch.bfloat16))
        g_out = torch.zeros(cfg.recv_rows, cfg.hidden, dtype=torch.bfloat16, device=gy.device)
        ep_combine_bwd(cfg, layout, gy.view(-1), p.view(-1) if ctx.has_probs else None, g_out.view(-1))
        g_probs = None
        if ctx.has_probs and ctx.needs_input_grad[1]:
            g_probs = torch.empty(cfg.num_tokens, cfg.top_k, dtype=torch.float32, device=gy.device)
            ep_combine_bwd_probs(cfg, layout, gy.view(-1), eo.view(-1), g_probs.view(-1))
        return g_out, g_probs, None, None


class _Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, token_mask, cfg, route):
        ids = torch.empty(cfg.num_tokens, cfg.top_k, dtype=torch.int32, device=logits.device)
        probs = torch.empty(cfg.num_tokens, cfg.top_k, dtype=torch.float32, device=logits.device)
        ep_route(cfg, route, logits, ids, probs, bias=bias, token_mask=token_mask)
        ctx.cfg, ctx.route = cfg, route
        ctx.save_for_backward(logits, ids)
        ctx.mark_non_differentiable(ids)
        return ids, probs

    @staticmethod
    @_first_only
    def backward(ctx, _, grad_probs):
        logits, ids = ctx.saved_tensors
        grad = torch.empty_like(logits)
        ep_route_bwd(ctx.cfg, ctx.route, logits, ids, grad_probs.float().contiguous(), grad)
        return grad, None, None, None, None


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, cfg, layout):
        y = torch.zeros(cfg.recv_rows, w.shape[1], dtype=torch.bfloat16, device=x.device)
        ep_expert_gemm(cfg, layout, x, w, y)
        ctx.cfg, ctx.layout = cfg, layout
        ctx.save_for_backward(x, w)
        return y

    @staticmethod
    @_first_only
    def backward(ctx, grad_y):
        x, w = ctx.saved_tensors
        gy = _rows(grad_y.to(torch.bfloat16))
        gx = gw = None
        if ctx.needs_input_grad[0]:
            gx = torch.zeros_like(x)
            ep_expert_gemm_bwd_x(ctx.cfg, ctx.layout, gy, w, gx)
        if ctx.needs_input_grad[1]:
            gw = torch.empty_like(w)
            ep_expert_gemm_bwd_w(ctx.cfg, ctx.layout, gy, x, gw)
        return gx, gw, None, None


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, probs, cfg, layout):
        act = torch.zeros(h.shape[0], h.shape[1] // 2, dtype=torch.bfloat16, device=h.device)
        ep_swiglu(cfg, layout, h, probs, act)
        ctx.cfg, ctx.layout = cfg, layout
        ctx.has_probs = probs is not None
        ctx.save_for_backward(h, probs if ctx.has_probs else torch.empty(0, device=h.device))
        return act

    @staticmethod
    @_first_only
    def backward(ctx, grad_act):
        h, p = ctx.saved_tensors
        ga = _rows(grad_act.to(torch.bfloat16))
        gh = torch.zeros_like(h)
        gp = None
        if ctx.has_probs and ctx.needs_input_grad[1]:
            gp = torch.empty(ctx.cfg.num_tokens, ctx.cfg.top_k, dtype=torch.float32, device=h.device)
        ep_swiglu_bwd(ctx.cfg, ctx.layout, h, p if ctx.has_probs else None, ga, gh, gp)
        return gh, gp, None, None


def _u(cfg, rank: int, device) -> torch.Tensor:
    return torch.empty(cfg.recv_rows, rank, dtype=torch.float32, device=device)


def _product_grads(ctx, gy, x, w, adapters, u, wanted):
    """The gradients of x, w, a and b of a product (with adapters, or None) from its
    results' gradient, those that are wanted."""
    cfg, layout = ctx.cfg, ctx.layout
    gx = gw = ga = gb = gu = None
    if adapters is not None and (wanted[0] or wanted[2] or wanted[3]):
        gu = _u(cfg, adapters.rank, gy.device)
        ep_lora_bwd_u(cfg, layout, gy, adapters, gu)
    if wanted[0]:
        gx = torch.zeros_like(x)
        if adapters is None:
            ep_expert_gemm_bwd_x(cfg, layout, gy, w, gx)
        else:
            ep_expert_gemm_bwd_x_lora(cfg, layout, gy, w, gx, adapters, gu)
    if wanted[1]:
        gw = torch.empty_like(w)
        ep_expert_gemm_bwd_w(cfg, layout, gy, x, gw)
    if wanted[2] or wanted[3]:
        ga, gb = torch.empty_like(adapters.a), torch.empty_like(adapters.b)
        ep_lora_bwd_w(cfg, layout, x, gy, adapters, u, gu, ga, gb)
    return gx, gw, ga, gb


class _LinearLora(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, a, b, token_adapter, scale, cfg, layout):
        adapters, u = Adapters(token_adapter, a, b, scale), _u(cfg, a.shape[2], x.device)
        y = torch.zeros(cfg.recv_rows, w.shape[1], dtype=torch.bfloat16, device=x.device)
        ep_lora_down(cfg, layout, x, adapters, u)
        ep_expert_gemm_lora(cfg, layout, x, w, y, adapters, u)
        ctx.cfg, ctx.layout = cfg, layout
        ctx.save_for_backward(x, w, a, b, u, token_adapter, scale)
        return y

    @staticmethod
    @_first_only
    def backward(ctx, grad_y):
        x, w, a, b, u, token_adapter, scale = ctx.saved_tensors
        adapters = Adapters(token_adapter, a, b, scale)
        grads = _product_grads(ctx, _rows(grad_y.to(torch.bfloat16)), x, w, adapters, u, ctx.needs_input_grad)
        return (*grads, None, None, None, None)


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, a, b, probs, token_adapter, scale, cfg, layout):
        adapters = u = None
        if a is not None:
            adapters, u = Adapters(token_adapter, a, b, scale), _u(cfg, a.shape[2], x.device)
            ep_lora_down(cfg, layout, x, adapters, u)
        act = torch.zeros(cfg.recv_rows, w.shape[1] // 2, dtype=torch.bfloat16, device=x.device)
        ep_expert_gated(cfg, layout, x, w, probs, act, adapters, u)
        ctx.cfg, ctx.layout = cfg, layout
        ctx.save_for_backward(x, w, a, b, probs, u, token_adapter, scale)
        return act

    @staticmethod
    @_first_only
    def backward(ctx, grad_act):
        x, w, a, b, probs, u, token_adapter, scale = ctx.saved_tensors
        cfg, layout = ctx.cfg, ctx.layout
        adapters = None if a is None else Adapters(token_adapter, a, b, scale)
        ga = _rows(grad_act.to(torch.bfloat16))
        gh = torch.zeros(cfg.recv_rows, w.shape[1], dtype=torch.bfloat16, device=x.device)
        gp = ws = None
        if probs is not None and ctx.needs_input_grad[4]:
            gp = torch.empty(cfg.num_tokens, cfg.top_k, dtype=torch.float32, device=x.device)
            ws = gated_workspace_for(cfg, ga.shape[1], x.device)
        ep_expert_gated_bwd(cfg, layout, x, w, probs, ga, gh, grad_probs=gp, workspace=ws, adapters=adapters, u=u)
        return (*_product_grads(ctx, gh, x, w, adapters, u, ctx.needs_input_grad), gp, None, None, None, None)


def _parts(adapters: Optional[Adapters]):
    """a, b, token_adapter and scale of adapters as the calls take them."""
    if adapters is None:
        return None, None, None, None
    if adapters.scale is not None and adapters.scale.requires_grad and torch.is_grad_enabled():
        raise ValueError("adapters.scale gets no gradient: detach it")
    return (_rows(adapters.a), _rows(adapters.b), adapters.token_adapter.to(torch.int32).contiguous(),
            None if adapters.scale is None else adapters.scale.detach().float().contiguous())


class EpDispatcher:
    """Dispatch / combine with autograd for one configuration on one device."""

    def __init__(self, cfg: EpConfig, device, recv_rows: Optional[int] = None):
        q = ep_query(cfg)
        cfg.recv_rows = q.min_recv_rows if recv_rows is None else recv_rows
        self.cfg = cfg
        self.device = torch.device(device)
        self.layout = Layout.empty(cfg, self.device)
        self.workspace = workspace_for(cfg, self.device)

    def route(self, topk_ids: torch.Tensor) -> Layout:
        """Build a new layout (counts, offsets, token_row, expert_ids, src_info,
        flags) for these ids; later dispatch/combine calls use it.  Nodes
        already recorded keep the layout they ran with."""
        layout = Layout.empty(self.cfg, self.device)
        ep_dispatch_layout(self.cfg, topk_ids.to(torch.int32).contiguous().view(-1), self.workspace, layout)
        self.layout = layout
        return layout

    def dispatch(self, x: torch.Tensor, topk_ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """[T, H] bf16 -> [R, H] bf16 receive rows.  With topk_ids, routes in
        the same call (ep_dispatch_with_layout) into a new layout that later
        calls use, as route() would."""
        if topk_ids is None:
            return _Dispatch.apply(_rows(x), self.cfg, self.layout)
        layout = Layout.empty(self.cfg, self.device)
        ids = topk_ids.to(torch.int32).contiguous().view(-1)
        recv = _Dispatch.apply(_rows(x), self.cfg, layout, ids, self.workspace)
        self.layout = layout
        return recv

    def combine(self, expert_out: torch.Tensor, probs: Optional[torch.Tensor]) -> torch.Tensor:
        """[R, H] bf16 expert outputs -> [T, H] bf16, weighted by probs [T, K] (or 1)."""
        return _Combine.apply(_rows(expert_out), _weights(probs), self.cfg, self.layout)

    def gate(self, logits: torch.Tensor, route: RouteConfig, bias: Optional[torch.Tensor] = None,
             token_mask: Optional[torch.Tensor] = None):
        """[T, E] logits (float32 or bfloat16) -> topk_ids int32 [T, K] and probs
        float32 [T, K], differentiable in the logits."""
        return _Gate.apply(_rows(logits), bias, token_mask, self.cfg, route)

    def linear(self, rows: torch.Tensor, w: torch.Tensor, adapters: Optional[Adapters] = None) -> torch.Tensor:
        """[R, in] bf16 receive rows times their experts' weights bf16
        [E (+1 shared), out, in] (and their tokens' adapters) -> [R, out]; rows no
        slot owns are zero."""
        if adapters is None:
            return _Linear.apply(_rows(rows), _rows(w), self.cfg, self.layout)
        a, b, of, scale = _parts(adapters)
        return _LinearLora.apply(_rows(rows), _rows(w), a, b, of, scale, self.cfg, self.layout)

    def gated(self, rows: torch.Tensor, w: torch.Tensor, probs: Optional[torch.Tensor],
              adapters: Optional[Adapters] = None) -> torch.Tensor:
        """swiglu(linear(rows, w, adapters), probs) in one kernel: rows [R, in], w bf16
        [E (+1 shared), 2*inter, in] (gate rows, then up rows) -> [R, inter].  Faster
        forward; with gradients the two calls are, where h fits beside the rest."""
        a, b, of, scale = _parts(adapters)
        return _Gated.apply(_rows(rows), _rows(w), a, b, _weights(probs), of, scale, self.cfg, self.layout)

    def swiglu(self, h: torch.Tensor, probs: Optional[torch.Tensor]) -> torch.Tensor:
        """[R, 2*inter] bf16 (gate, then up) -> [R, inter], each row times its
        slot's probs [T, K] (or 1); rows no slot owns are zero."""
        return _Swiglu.apply(_rows(h), _weights(probs), self.cfg, self.layout)

    def tokens_per_expert(self) -> torch.Tensor:
        """Routed rows per group [S, G] (the shared group included)."""
        return self.layout.counts
