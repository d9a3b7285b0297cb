"""The expert layer at any number of tokens, from the calls in ``moeq``.

``Mx4MoeLayer`` serves: router, sort by expert, gate_up and down products with
MXFP4 weights, and the weighted combine with the shared expert, for one token
or a prompt.  ``moeq.moeq_moe_layer`` is its FP8 counterpart for up to 16
tokens in one kernel.

``route``, ``dispatch`` and ``combine`` train: the same routing and movement
as autograd functions, around whatever experts the caller's program has, to any order.
"""
from __future__ import annotations

import torch

from . import moeq


class Dispatch:
    """Where each (token, slot) pair goes: rows of expert e are
    offs[e] .. offs[e + 1] - 1; pair_row [T, k] and row_pair [T * k] map
    between the two orders (-1: no row)."""

    def __init__(self, topk_id: torch.Tensor, E: int):
        T, k = topk_id.shape
        new = lambda *s: torch.empty(s, dtype=torch.int32, device=topk_id.device)
        self.E, self.offs, self.pair_row, self.row_pair = E, new(E + 1), new(T, k), new(T * k)
        moeq.moeq_expert_sort(topk_id, E, self.offs, self.pair_row, self.row_pair)


# ------------------------------------------------------------------ training
# Every backward pass is a function of its own with a backward pass, so that a
# second differentiation (a gradient penalty, a Hessian-vector product) sees
# the first one's dependence on what was saved: the kernels read and write
# through pointers, and a graph would take their results for constants.
# (torch's once_differentiable would not refuse it: it looks at the incoming
# gradients alone, and d_y = w d_out depends on w for a constant d_out.)
# Indices are saved as tensors, so that autograd notices when one is
# overwritten in place.
def _route_grad(dw, ids, w, E):
    dl = torch.empty((ids.shape[0], E), dtype=w.dtype, device=w.device)
    moeq.moeq_route_rows_grad(dw, ids, w, dl)
    return dl


def _gather(x, offs, pair_row):
    xs = torch.empty((pair_row.numel(), x.shape[1]), dtype=x.dtype, device=x.device)
    moeq.moeq_gather_rows(x, offs, pair_row, xs)
    return xs


def _gather_grad(dxs, offs, pair_row):
    dx = torch.empty((pair_row.shape[0], dxs.shape[1]), dtype=dxs.dtype, device=dxs.device)
    moeq.moeq_gather_rows_grad(dxs, pair_row, dx)
    return dx


def _combine_grad(dout, y, w, offs, pair_row):
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    moeq.moeq_combine_rows_grad(dout, y, offs, pair_row, w, dy, dw)
    return dy, dw


def _grad(function, plain):
    """The autograd function where its result may be differentiated again, the plain call where it cannot."""
    return function.apply if torch.is_grad_enabled() else plain


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k):
        T = logits.shape[0]
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, k), dtype=logits.dtype, device=logits.device)
        moeq.moeq_route_rows(logits, ids, w)
        ctx.save_for_backward(ids, w)
        ctx.E = logits.shape[1]
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, dw):
        ids, w = ctx.saved_tensors
        return _grad(_RouteGrad, _route_grad)(dw.contiguous(), ids, w, ctx.E), None


class _RouteGrad(torch.autograd.Function):
    """F = sum_j g_j w_j (dw_j - s), s = sum_i w_i dw_i, for a gradient g of d_logits at the picks:
    dF/d(dw_j) = w_j (g_j - t) and dF/dw_j = g_j (dw_j - s) - dw_j t, t = sum_i w_i g_i."""

    @staticmethod
    def forward(ctx, dw, ids, w, E):
        ctx.save_for_backward(dw, ids, w)
        return _route_grad(dw, ids, w, E)

    @staticmethod
    def backward(ctx, g):
        dw, ids, w = ctx.saved_tensors
        live = ids >= 0
        zero = torch.zeros((), dtype=w.dtype, device=w.device)
        g = torch.where(live, g.gather(1, ids.clamp(min=0).long()), zero)
        dw = torch.where(live, dw, zero)
        s, t = (w * dw).sum(1, keepdim=True), (w * g).sum(1, keepdim=True)
        return w * (g - t), None, g * (dw - s) - dw * t, None


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offs, pair_row):
        ctx.save_for_backward(offs, pair_row)
        return _gather(x, offs, pair_row)

    @staticmethod
    def backward(ctx, dxs):
        return _grad(_DispatchGrad, _gather_grad)(dxs.contiguous(), *ctx.saved_tensors), None, None


class _DispatchGrad(torch.autograd.Function):
    """Dispatch's adjoint, so its own is dispatch."""

    @staticmethod
    def forward(ctx, dxs, offs, pair_row):
        ctx.save_for_backward(offs, pair_row)
        return _gather_grad(dxs, offs, pair_row)

    @staticmethod
    def backward(ctx, g):
        return _grad(_Dispatch, _gather)(g.contiguous(), *ctx.saved_tensors), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, w, base, offs, pair_row):
        ctx.has_base = base is not None
        ctx.save_for_backward(y, w, offs, pair_row)
        out = torch.empty((w.shape[0], y.shape[1]), dtype=y.dtype if base is None else base.dtype, device=y.device)
        moeq.moeq_combine_rows(y, pair_row, w, out, base=base)
        return out

    @staticmethod
    def backward(ctx, dout):
        dout = dout.contiguous()
        dy, dw = _grad(_CombineGrad, _combine_grad)(dout, *ctx.saved_tensors)
        return dy, dw, dout if ctx.has_base else None, None, None


class _CombineGrad(torch.autograd.Function):
    """dy = w dout and dw = <dout, y> at the slots' rows.  For gradients gy and gw of them, dout gets
    sum_j w_j gy + gw_j y, y gets gw dout, and w gets <dout, gy>: combine and this function again."""

    @staticmethod
    def forward(ctx, dout, y, w, offs, pair_row):
        ctx.save_for_backward(dout, y, w, offs, pair_row)
        return _combine_grad(dout, y, w, offs, pair_row)

    @staticmethod
    def backward(ctx, gy, gw):
        dout, y, w, *plan = ctx.saved_tensors
        gy, gw = gy.contiguous(), gw.contiguous()
        d_dout = _Combine.apply(y, gw, _Combine.apply(gy, w, torch.zeros_like(dout), *plan), *plan)
        dy, dw = _grad(_CombineGrad, _combine_grad)(dout, gy, gw, *plan)
        return d_dout, dy, dw, None, None


def route(logits: torch.Tensor, k: int):
    """topk_id [T, k] int32 and topk_w [T, k] fp32 of logits [T, E] fp32; the weights carry the gradient."""
    return _Route.apply(logits, k)


def dispatch(x: torch.Tensor, d: Dispatch) -> torch.Tensor:
    """Rows of x [T, H] in expert order: [T * k, H], zero rows after the last."""
    return _Dispatch.apply(x, d.offs, d.pair_row)


def combine(y: torch.Tensor, w: torch.Tensor, d: Dispatch, base: torch.Tensor | None = None) -> torch.Tensor:
    """base[t] + sum_j w[t, j] * y[row of (t, j)]."""
    return _Combine.apply(y.contiguous(), w.contiguous(), base, d.offs, d.pair_row)


# ------------------------------------------------------------------- serving
class Mx4Weights:
    """Expert matrices w [E, N, K] (bf16 or fp32, on the device) quantised to MXFP4 tiles."""

    def __init__(self, w: torch.Tensor):
        self.E, self.N, self.K = w.shape
        self.tiles, self.scales = moeq.mx4_weight_buffers(self.E, self.N, self.K, device=w.device)
        moeq.moeq_mx4_quant_weight(w, self.tiles, self.scales)


class Mx4MoeLayer:
    """out = shared(x) + sum_j w_j * expert_j(x), every expert down(silu(gate x) * up x).

    w_gu [E, 2I, H] (gate rows, then up rows), w_d [E, H, I]; shared_gu
    [1, 2I, H] and shared_d [1, H, I], or None for a layer without a shared
    expert.  Buffers are kept for the number of tokens last seen; one instance
    is not to be used by two streams at once."""

    def __init__(self, w_gu, w_d, top_k: int, shared_gu=None, shared_d=None):
        self.gu, self.d = Mx4Weights(w_gu), Mx4Weights(w_d)
        self.s_gu = None if shared_gu is None else Mx4Weights(shared_gu)
        self.s_d = None if shared_d is None else Mx4Weights(shared_d)
        if (self.s_gu is None) != (self.s_d is None):
            raise ValueError("Mx4MoeLayer: shared_gu and shared_d come together")
        self.top_k, self.T = top_k, -1

    def _buffers(self, T: int, device):
        if T == self.T:
            return
        H, I, E, k, R = self.gu.K, self.d.K, self.gu.E, self.top_k, T * self.top_k
        new = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=device)
        self.ids, self.w = new(T, k, dt=torch.int32), new(T, k, dt=torch.float32)
        self.offs, self.pair_row, self.row_pair = new(E + 1, dt=torch.int32), new(T, k, dt=torch.int32), new(R, dt=torch.int32)
        self.h, self.y = new(R, 2 * I), new(R, H)
        sizes = [moeq.moeq_mx4_expert_gemm_workspace_size(T, H, 2 * I, E, R),
                 moeq.moeq_mx4_expert_gemm_workspace_size(R, I, H, E, R)]
        if self.s_gu is not None:
            self.sh, self.sy = new(T, 2 * self.s_d.K), new(T, H)
            self.s_offs = torch.tensor([0, T], dtype=torch.int32, device=device)
            sizes += [moeq.moeq_mx4_expert_gemm_workspace_size(T, H, 2 * self.s_d.K, 1, T),
                      moeq.moeq_mx4_expert_gemm_workspace_size(T, self.s_d.K, H, 1, T)]
        self.ws = moeq.Workspace(max(sizes), device=device)   # the products run one after another
        self.T = T

    def __call__(self, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """x [T, H] bf16, logits [T, E] fp32 -> out [T, H] bf16."""
        T = x.shape[0]
        if out is None:
            out = torch.empty_like(x)
        if T == 0:
            return out
        self._buffers(T, x.device)
        base = None
        if self.s_gu is not None:
            self._ffn(x, self.s_gu, self.s_d, self.s_offs, self.sh, self.sy, None, 1)
            base = self.sy
        moeq.moeq_route_rows(logits, self.ids, self.w)
        moeq.moeq_expert_sort(self.ids, self.gu.E, self.offs, self.pair_row, self.row_pair)
        self._ffn(x, self.gu, self.d, self.offs, self.h, self.y, self.row_pair, self.top_k)
        moeq.moeq_combine_rows(self.y, self.pair_row, self.w, out, base=base)
        return out

    def _ffn(self, x, gu, d, offs, h, y, row_pair, top_k):
        moeq.moeq_mx4_expert_gemm(x, gu.tiles, gu.scales, offs, h, self.ws, row_pair=row_pair, top_k=top_k)
        moeq.moeq_mx4_expert_gemm(h, d.tiles, d.scales, offs, y, self.ws, act=moeq.MOEQ_ACT_SWIGLU)
