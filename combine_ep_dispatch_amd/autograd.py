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

A step can be captured into a graph, backward pass included, on leaves that no
eager autograd graph still holds (torch does not support capturing beside one).

The backward passes are library calls without gradients of their own: under
create_graph the first derivatives can be had, differentiating them raises.
"""

from __future__ import annotations

import functools
from typing import Optional

import torch

from . import (EpConfig, Layout, RouteConfig, ep_combine, ep_combine_bwd, ep_combine_bwd_probs, ep_dispatch,
               ep_dispatch_bwd, ep_dispatch_layout, ep_dispatch_with_layout, ep_expert_gemm, ep_expert_gemm_bwd_w,
               ep_expert_gemm_bwd_x, ep_query, ep_route, ep_route_bwd, ep_swiglu, ep_swiglu_bwd, workspace_for)

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

    def linear(self, rows: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
        """[R, in] bf16 receive rows times their experts' weights bf16
        [E (+1 shared), out, in] -> [R, out]; rows no slot owns are zero."""
        return _Linear.apply(_rows(rows), _rows(w), self.cfg, self.layout)

    def swiglu(self, h: torch.Tensor, probs: Optional[torch.Tensor]) -> torch.Tensor:
        """[R, 2*inter] bf16 (gate, then up) -> [R, inter], each row times its
        slot's probs [T, K] (or 1); rows no slot owns are zero."""
        return _Swiglu.apply(_rows(h), _weights(probs), self.cfg, self.layout)

    def tokens_per_expert(self) -> torch.Tensor:
        """Routed rows per group [S, G] (the shared group included)."""
        return self.layout.counts
