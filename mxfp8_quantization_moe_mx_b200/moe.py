"""The operators of a mixture-of-experts layer as a model calls them: they allocate their
results, and the ones that a model trains through are differentiable.

    n = moe.rmsnorm(x, weight, residual=stream)        # n.y, n.res, and n.q, n.s in MXFP8
    weights, ids = moe.route(n.y.float() @ router.T, k, renorm=True)
    p = moe.plan(ids, E)                               # p.offs, p.rows, p.src
    rows = n.y[p.src.long() // k]                      # the experts' rows, sorted
    out = experts(rows, p.offs)                        # moe.Mxfp4Experts, for serving
    slots = out[p.rows.clamp(min=0).long()].float().masked_fill(p.rows[:, :, None] < 0, 0.0)
    y = (slots * weights[:, :, None]).sum(1)

A slot that is routed nowhere (its id is -1) has row -1 and weight 0.  Rows at and past the
last offset belong to no expert, and the products leave them unwritten: what lies there may be
NaN, which a weight of 0 does not remove, so the slots are masked.  Their source is -1 as well
(the gather above takes the last token for them); where gradients pass through the gather and
a product that leaves those rows' gradients unwritten, mask `rows` by p.src < 0 alike.

Everything runs in this library's kernels on the tensors' device and its current stream;
there is no CPU path.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import (SOFTMAX, MxqError, moe_plan, moe_plan_workspace_bytes, moe_route, moe_route_backward,
               mx_scales_blocked_bytes, mxfp4_grouped_gemm, mxfp4_quantize, rmsnorm_backward,
               rmsnorm_backward_workspace_bytes, rmsnorm_mx_quantize)


def _new(like: torch.Tensor, dtype, *shape) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=like.device)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, k, score, n_groups, top_groups, group_top, renorm, scale):
        logits = logits.contiguous()
        T = logits.shape[0]
        weights, ids = _new(logits, torch.float32, T, k), _new(logits, torch.int32, T, k)
        moe_route(logits, weights, ids, bias=bias, score=score, n_groups=n_groups, top_groups=top_groups,
                  group_top=group_top, renorm=renorm, scale=scale)
        ctx.save_for_backward(logits, ids)
        ctx.how = (score, renorm, scale)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_weights, _):
        logits, ids = ctx.saved_tensors
        score, renorm, scale = ctx.how
        grad = torch.empty_like(logits)
        moe_route_backward(logits, ids, grad_weights.float().contiguous(), grad, score=score, renorm=renorm,
                           scale=scale)
        return (grad,) + (None,) * 8


def route(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, score: int = SOFTMAX, n_groups: int = 1,
          top_groups: int = 1, group_top: int = 1, renorm: bool = False,
          scale: float = 1.0) -> tuple[torch.Tensor, torch.Tensor]:
    """logits bf16 or fp32 (T, E) -> (weights fp32 (T, k), ids int32 (T, k)), as moe_route.
    Differentiable in the logits; the bias shapes the choice alone and takes no gradient."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise MxqError("logits must be (T, E)")
    if bias is not None:
        bias = bias.detach().contiguous()
    return _Route.apply(logits, bias, int(k), score, n_groups, top_groups, group_top, bool(renorm), float(scale))


class Plan(NamedTuple):
    offs: torch.Tensor  # int32 (E,): expert e's rows are offs[e - 1] .. offs[e] - 1
    rows: torch.Tensor  # int32, the ids' shape: the row of each slot, or -1
    src: torch.Tensor   # int32 (n,): the slot of each row, or -1 past the last


def plan(ids: torch.Tensor, n_experts: int) -> Plan:
    """The rows of the routed slots, sorted by expert and stable within one (moe_plan)."""
    ids = ids.contiguous()
    n = ids.numel()
    p = Plan(_new(ids, torch.int32, n_experts), torch.empty_like(ids), _new(ids, torch.int32, n))
    need = moe_plan_workspace_bytes(n, n_experts)
    moe_plan(ids, p.offs, p.rows, p.src, _new(ids, torch.uint8, need) if need else None)
    return p


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        x, weight = x.contiguous(), weight.contiguous()
        M, D = x.shape
        y, rstd = torch.empty_like(x), _new(x, torch.float32, M)
        q, s = _new(x, torch.uint8, M, D), _new(x, torch.uint8, M, D // 32)
        res = None
        if residual is not None:
            residual, res = residual.contiguous(), torch.empty_like(x)
        rmsnorm_mx_quantize(x, weight, eps, q, s, residual=residual, res_out=res, y=y, rstd=rstd)
        ctx.save_for_backward(x if res is None else res, weight, rstd)
        ctx.with_residual = res is not None
        ctx.mark_non_differentiable(q, s)
        ctx.set_materialize_grads(False)
        return (y, q, s) if res is None else (y, q, s, res)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, _q, _s, grad_res=None):
        h, weight, rstd = ctx.saved_tensors
        if grad_y is None:  # only the stream was used: the norm itself has no part in it
            g = grad_res
            return g, g if ctx.with_residual else None, None, None
        M, D = h.shape
        grad_x, grad_w = torch.empty_like(h), _new(h, torch.float32, D)
        ws = _new(h, torch.uint8, rmsnorm_backward_workspace_bytes(M, D))
        rmsnorm_backward(grad_y.contiguous(), h, weight, rstd, grad_x, grad_w, ws,
                         grad_res=None if grad_res is None else grad_res.contiguous())
        return grad_x, grad_x if ctx.with_residual else None, grad_w.to(weight.dtype), None


class Norm(NamedTuple):
    y: torch.Tensor    # bf16 (M, D), the norm
    q: torch.Tensor    # uint8 (M, D), its E4M3 codes
    s: torch.Tensor    # uint8 (M, D/32), their E8M0 scales
    res: torch.Tensor  # bf16 (M, D), x + residual (x itself without one)


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None) -> Norm:
    """The RMS norm of x (+ residual), bf16 (M, D), in bf16 and in MXFP8 (rmsnorm_mx_quantize).
    Differentiable in x, residual and weight through y and res; the codes take no gradient
    (a product with them passes its own through to y)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise MxqError("x must be (M, D)")
    if residual is not None and residual.shape != x.shape:
        raise MxqError("residual must have the shape of x")
    out = _RmsNorm.apply(x, residual, weight, float(eps))
    return Norm(out[0], out[1], out[2], x if residual is None else out[3])


class Mxfp4Experts:
    """Expert matrices held in MXFP4, for serving: quantized and laid out once, then applied to
    the rows of a plan.

    weights: bf16 (G, N, K), N a multiple of 256 and K of 128; experts(x, offs) is
    x[rows of g] @ weights[g].T for every group g of the end offsets, with x bf16 (M, K)
    quantized to MXFP4 on the way.  Rows in no group come back unwritten (mask them when they
    are combined, as above).  No gradient."""

    def __init__(self, weights: torch.Tensor):
        if not isinstance(weights, torch.Tensor) or weights.dim() != 3:
            raise MxqError("weights must be (G, N, K)")
        G, N, K = weights.shape
        if N % 256 or K % 128:
            raise MxqError("N must be a multiple of 256 and K of 128")
        self.shape = (G, N, K)
        self.codes = _new(weights, torch.uint8, G, N, K // 2)
        self.scales = _new(weights, torch.uint8, mx_scales_blocked_bytes(G, N, K // 32))
        mxfp4_quantize(weights.detach().contiguous(), self.codes, sf_blocked=self.scales)

    def __call__(self, x: torch.Tensor, offs: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        G, N, K = self.shape
        if x.dim() != 2 or x.shape[1] != K or offs.numel() != G:
            raise MxqError(f"x must be (M, {K}) and offs ({G},)")
        if torch.is_grad_enabled() and x.requires_grad:
            raise MxqError("the MXFP4 experts have no gradient: call them under torch.no_grad()")
        M = x.shape[0]
        codes = _new(x, torch.uint8, M, K // 2)
        scales = _new(x, torch.uint8, mx_scales_blocked_bytes(1, M, K // 32, G))
        if out is None:
            out = _new(x, torch.bfloat16, M, N)
        mxfp4_quantize(x.contiguous(), codes, sf_blocked=scales, offs=offs)
        mxfp4_grouped_gemm(codes, scales, self.codes, self.scales, offs, out)
        return out
