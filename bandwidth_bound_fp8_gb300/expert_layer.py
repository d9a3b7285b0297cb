"""The expert layer at any number of tokens, from the calls in ``moeq``.

``Mx4MoeLayer`` serves: router, sort by expert, gate_up and down products with
MXFP4 weights, and the weighted combine with the shared expert, for one token
or a prompt.  ``moeq.moeq_moe_layer`` is its FP8 counterpart for up to 16
tokens in one kernel.

``route``, ``dispatch`` and ``combine`` train: the same routing and movement
as autograd functions, around whatever experts the caller's program has, to any
order (in reverse mode: a tangent raises).  ``expert_product`` is the product of
bf16 experts for it, to any order too; ``swiglu`` and ``expert_mlp`` (the experts
between dispatch and combine as one function) keep what their backward pass
needs in 8 bits.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import moeq


_words: dict = {}   # status words that no plan has yet, by the stream that they were zeroed on


def _status_word(device: torch.device) -> torch.Tensor:
    """An int32 [1] that is 0 on the current stream.  Many are zeroed at once: a fill for each would double a plan's time on
    the host.  Inside a capture the fill belongs to the graph, so that every replay starts with 0."""
    if device.type != "cuda" or torch.cuda.is_current_stream_capturing():
        return torch.zeros(1, dtype=torch.int32, device=device)
    of = device.index, moeq.current_stream_handle()
    words = _words.get(of)
    if not words:
        words = _words[of] = list(torch.zeros(256, dtype=torch.int32, device=device).split(1))
    return words.pop()


class Dispatch:
    """Where each (token, slot) pair goes: rows of expert e are
    offs[e] .. offs[e + 1] - 1; pair_row [T, k] and row_pair [T * k] map
    between the two orders (-1: no row).  status [1] is 0, or what a product
    with this plan (or its gradient) reported: ``check`` asks."""

    def __init__(self, topk_id: torch.Tensor, E: int):
        T, k = topk_id.shape
        new = lambda *s: torch.empty(s, dtype=torch.int32, device=topk_id.device)
        self.E, self.offs, self.pair_row, self.row_pair = E, new(E + 1), new(T, k), new(T * k)
        moeq.moeq_expert_sort(topk_id, E, self.offs, self.pair_row, self.row_pair)
        self.status = _status_word(topk_id.device)

    def check(self) -> None:
        """Raises MoeqError where a product with this plan gave up a wait inside its kernel: its results are then not
        valid.  (Waits for the device; a training step asks where it reads its loss.)"""
        status = int(self.status)
        if status:
            raise moeq.MoeqError("a product of the experts", status)


# ------------------------------------------------------------------ training
# Every backward pass is a function of its own with a backward pass, so that a
# second differentiation (a gradient penalty, a Hessian-vector product) sees
# the first one's dependence on what was saved: the kernels read and write
# through pointers, and a graph would take their results for constants.
# (torch's once_differentiable would not refuse it: it looks at the incoming
# gradients alone, and d_y = w d_out depends on w for a constant d_out.)
# Indices are saved as tensors, so that autograd notices when one is
# overwritten in place.
# A step that is captured into a CUDA graph has to be the only one that holds
# the leaves' gradients: torch's engine ends a capture that meets a node of an
# eager graph of the same leaves, so drop that graph first.
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


def _differentiated(args) -> bool:
    """Whether a result of args may be differentiated again, or one of them has a tangent."""
    if torch.is_grad_enabled():
        return True
    # (outside a dual_level, the module's level -1, there are no tangents: 1 us a tensor saved)
    return getattr(forward_ad, "_current_level", 0) >= 0 and any(
        isinstance(t, torch.Tensor) and t.is_floating_point() and forward_ad.unpack_dual(t).tangent is not None for t in args)


def _grad(function, plain, *args):
    """The autograd function where its result is differentiated further (in forward mode it raises: it has no rule), the
    plain call where it is not."""
    return (function.apply if _differentiated(args) else plain)(*args)


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
        return _grad(_RouteGrad, _route_grad, dw.contiguous(), ids, w, ctx.E), None


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
        return _grad(_DispatchGrad, _gather_grad, dxs.contiguous(), *ctx.saved_tensors), None, None


class _DispatchGrad(torch.autograd.Function):
    """Dispatch's adjoint, so its own is dispatch."""

    @staticmethod
    def forward(ctx, dxs, offs, pair_row):
        ctx.save_for_backward(offs, pair_row)
        return _gather_grad(dxs, offs, pair_row)

    @staticmethod
    def backward(ctx, g):
        return _grad(_Dispatch, _gather, g.contiguous(), *ctx.saved_tensors), None, None


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
        dy, dw = _grad(_CombineGrad, _combine_grad, dout, *ctx.saved_tensors)
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
        dy, dw = _grad(_CombineGrad, _combine_grad, dout, gy, gw, *plan)
        return d_dout, dy, dw, None, None


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy where its rows are not contiguous or lie over each other (a transpose, an expanded bias)."""
    fits = t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1) and (t.stride(0) >= t.shape[1] or t.shape[0] <= 1)
    return t if fits else t.contiguous()


def route(logits: torch.Tensor, k: int):
    """topk_id [T, k] int32 and topk_w [T, k] fp32 of logits [T, E] fp32; the weights carry the gradient."""
    return _Route.apply(_rows(logits), k)


def dispatch(x: torch.Tensor, d: Dispatch) -> torch.Tensor:
    """Rows of x [T, H] in expert order: [T * k, H], zero rows after the last."""
    return _Dispatch.apply(_rows(x), d.offs, d.pair_row)


def combine(y: torch.Tensor, w: torch.Tensor, d: Dispatch, base: torch.Tensor | None = None) -> torch.Tensor:
    """base[t] + sum_j w[t, j] * y[row of (t, j)]."""
    return _Combine.apply(y.contiguous(), w.contiguous(), None if base is None else _rows(base), d.offs, d.pair_row)


# ------------------------------------------------------- training: experts
def _product(x, w, offs, status):
    y = torch.empty((x.shape[0], w.shape[1]), dtype=x.dtype, device=x.device)
    moeq.moeq_expert_product(x, w, offs, y, status=status)
    return y


def _product_grad_x(dy, w, offs, status):
    dx = torch.empty((dy.shape[0], w.shape[2]), dtype=dy.dtype, device=dy.device)
    moeq.moeq_expert_product_grad_x(dy, w, offs, dx, status=status)
    return dx


def _product_grad_w(dy, x, offs, status):
    dw = torch.empty((offs.shape[0] - 1, dy.shape[1], x.shape[1]), dtype=x.dtype, device=x.device)
    moeq.moeq_expert_product_grad_w(dy, x, offs, dw, status=status)
    return dw


def _copied(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy where tensor copies cannot read its rows: they start and step on 16 bytes."""
    t = _rows(t)
    fits = t.data_ptr() % 16 == 0 and (t.stride(0) % 8 == 0 or t.shape[0] <= 1)
    return t if fits else t.clone(memory_format=torch.contiguous_format)


def _weights(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy where it is not contiguous or starts off 16 bytes (a slice of a flat buffer)."""
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


# y = W x, dx = W^T dy and dW = dy x^T are linear in either argument, and each
# one's derivatives are the other two.  (The status word is written, and so not
# among what autograd watches.)
class _Product(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offs, status):
        ctx.status = status
        ctx.save_for_backward(x, w, offs)
        return _product(x, w, offs, status)

    @staticmethod
    def backward(ctx, dy):
        x, w, offs = ctx.saved_tensors
        dy, need = _copied(dy), ctx.needs_input_grad
        return (_grad(_ProductGradX, _product_grad_x, dy, w, offs, ctx.status) if need[0] else None,
                _grad(_ProductGradW, _product_grad_w, dy, x, offs, ctx.status) if need[1] else None, None, None)


class _ProductGradX(torch.autograd.Function):
    @staticmethod
    def forward(ctx, dy, w, offs, status):
        ctx.status = status
        ctx.save_for_backward(dy, w, offs)
        return _product_grad_x(dy, w, offs, status)

    @staticmethod
    def backward(ctx, g):
        dy, w, offs = ctx.saved_tensors
        g, need = _copied(g), ctx.needs_input_grad
        return (_grad(_Product, _product, g, w, offs, ctx.status) if need[0] else None,
                _grad(_ProductGradW, _product_grad_w, dy, g, offs, ctx.status) if need[1] else None, None, None)


class _ProductGradW(torch.autograd.Function):
    @staticmethod
    def forward(ctx, dy, x, offs, status):
        ctx.status = status
        ctx.save_for_backward(dy, x, offs)
        return _product_grad_w(dy, x, offs, status)

    @staticmethod
    def backward(ctx, g):
        dy, x, offs = ctx.saved_tensors
        g, need = _weights(g), ctx.needs_input_grad
        return (_grad(_Product, _product, x, g, offs, ctx.status) if need[0] else None,
                _grad(_ProductGradX, _product_grad_x, dy, g, offs, ctx.status) if need[1] else None, None, None)


class _Once(torch.autograd.Function):
    """Ties gradients to what they depend on, so that a second differentiation raises instead of taking them for
    constants."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(None if t is None else t.detach() for t in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("swiglu and expert_mlp keep their inputs in 8 bits: they are differentiable once")


# What was quantised is not kept, and the gradients depend on it: its place in
# the graph is held by a second output, empty, whose node is the function's own.
def _mark(ctx, t, keep):
    ctx.set_materialize_grads(False)   # (the mark's own gradient would be made each time)
    return t.new_empty(0) if keep else None


def _once(grads, *of):
    """Gradients as a backward pass returns them; `of`: the tensors they depend on."""
    return _Once.apply(len(grads), *grads, *of) if _differentiated(of) else grads


def _keep8(x):
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty((x.shape[0], moeq.fp8_groups(x.shape[1])), dtype=torch.float32, device=x.device)
    moeq.moeq_fp8_quant_rows(x, codes, scales)
    return codes, scales


def _swiglu(gu, w, row_pair, keep):
    """h, and gate and up in 8 bits where they are kept."""
    R, I = gu.shape[0], gu.shape[1] // 2
    h = torch.empty((R, I), dtype=gu.dtype, device=gu.device)
    if not keep:
        moeq.moeq_swiglu_rows(gu, h, row_pair=row_pair, topk_w=w)
        return h, None, None
    codes = torch.empty(gu.shape, dtype=torch.uint8, device=gu.device)
    scales = torch.empty((R, 2 * moeq.fp8_groups(I)), dtype=torch.float32, device=gu.device)
    moeq.moeq_swiglu_rows(gu, h, row_pair=row_pair, topk_w=w, codes=codes, scales=scales)
    return h, codes, scales


def _swiglu_grad(dh, codes, scales, w, pair_row, row_pair, need_w, again):
    """d_gu, d_w where it is needed, and h where it is asked for again."""
    dgu = torch.empty(codes.shape, dtype=dh.dtype, device=dh.device)
    dw = torch.empty_like(w) if need_w else None
    h = torch.empty_like(dh, memory_format=torch.contiguous_format) if again else None
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, dgu, h=h, row_pair=row_pair, topk_w=w, pair_row=pair_row, d_topk_w=dw)
    return dgu, dw, h


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gu, w, pair_row, row_pair, keep):
        h, codes, scales = _swiglu(gu, w, row_pair, keep)
        mark = _mark(ctx, gu, keep)
        ctx.save_for_backward(codes, scales, w, pair_row, row_pair, mark)
        return h, mark

    @staticmethod
    def backward(ctx, dh, _):
        codes, scales, w, pair_row, row_pair, mark = ctx.saved_tensors
        if dh is None:
            dh = mark.new_zeros((codes.shape[0], codes.shape[1] // 2))
        dgu, dw, _ = _swiglu_grad(_rows(dh), codes, scales, w, pair_row, row_pair, ctx.needs_input_grad[1], False)
        return (*_once((dgu, dw), dh, w, mark), None, None, None)


class _ExpertMlp(torch.autograd.Function):
    """The routing weight is part of h, so that the rows of y add up to out, and its gradient is <d_h, h / w>: neither y
    nor h is kept, and x and its gate and up rows are in 8 bits."""

    @staticmethod
    def forward(ctx, x, w, w_gu, w_d, offs, pair_row, row_pair, status, keep):
        ctx.status = status
        gu = _product(_gather(x, offs, pair_row), w_gu, offs, status)
        h, codes, scales = _swiglu(gu, w, row_pair, keep)
        del gu
        x8 = _keep8(x) if keep and ctx.needs_input_grad[2] else (None, None)
        mark = _mark(ctx, x, keep)
        ctx.save_for_backward(*x8, codes, scales, w, w_gu, w_d, offs, pair_row, row_pair, mark)
        return _gather_grad(_product(h, w_d, offs, status), offs, pair_row), mark

    @staticmethod
    def backward(ctx, dout, _):
        x_codes, x_scales, codes, scales, w, w_gu, w_d, offs, pair_row, row_pair, mark = ctx.saved_tensors
        need_x, need_w, need_gu, need_d = ctx.needs_input_grad[:4]
        if dout is None:
            dout = mark.new_zeros((pair_row.shape[0], w_gu.shape[2]))
        with torch.no_grad():
            dy = _gather(_rows(dout), offs, pair_row)
            dh = _product_grad_x(dy, w_d, offs, ctx.status)
            dgu, dw, h = _swiglu_grad(dh, codes, scales, w, pair_row, row_pair, need_w, need_d)
            del dh
            dw_d = _product_grad_w(dy, h, offs, ctx.status) if need_d else None
            del dy, h
            dx = _gather_grad(_product_grad_x(dgu, w_gu, offs, ctx.status), offs, pair_row) if need_x else None
            dw_gu = None
            if need_gu:
                xs = torch.empty((dgu.shape[0], w_gu.shape[2]), dtype=dgu.dtype, device=dgu.device)
                moeq.moeq_fp8_gather_rows(x_codes, x_scales, offs, pair_row, xs)
                dw_gu = _product_grad_w(dgu, xs, offs, ctx.status)
        return (*_once((dx, dw, dw_gu, dw_d), dout, w, w_gu, w_d, mark), None, None, None, None, None)


def _experts_fit(what: str, w: torch.Tensor, d: Dispatch, width: int, name: str = "w") -> None:
    if w.dim() != 3 or w.shape[0] != d.E or w.shape[2] != width:
        raise ValueError(f"{what}: {name} [{d.E}, N, {width}] is wanted, got {tuple(w.shape)}")


def _weights_fit(what: str, w: torch.Tensor, d: Dispatch) -> None:
    if w.shape != d.pair_row.shape or w.dtype is not torch.float32:
        raise ValueError(f"{what}: weights {tuple(d.pair_row.shape)} fp32 are wanted, got {w.dtype} {tuple(w.shape)}")


def expert_product(x: torch.Tensor, w: torch.Tensor, d: Dispatch) -> torch.Tensor:
    """w[e] x[r] for the rows [T * k, K] of dispatch, bf16, and w [E, N, K] bf16: [T * k, N], zero rows after the last.
    K and N are multiples of 8; rows and weights that do not start on 16 bytes are copied."""
    if x.dim() != 2 or x.shape[0] != d.row_pair.shape[0]:
        raise ValueError(f"expert_product: x [{d.row_pair.shape[0]}, K] is wanted, got {tuple(x.shape)}")
    _experts_fit("expert_product", w, d, x.shape[1])
    return _Product.apply(_copied(x), _weights(w), d.offs, d.status)


def swiglu(gu: torch.Tensor, d: Dispatch, w: torch.Tensor | None = None) -> torch.Tensor:
    """w silu(gate) up for the rows gu [T * k, 2I] (gate, then up; bf16 or fp32), w [T, k] a pair's weight (None: 1).
    The backward pass sees gate and up in 8 bits (groups of 128, moeq_fp8_quant_rows): half to a quarter of the bytes.
    Differentiable once: a second derivative raises."""
    if gu.dim() != 2 or gu.shape[0] != d.row_pair.shape[0] or gu.shape[1] % 2:
        raise ValueError(f"swiglu: gu [{d.row_pair.shape[0]}, 2I] is wanted, got {tuple(gu.shape)}")
    if w is not None:
        _weights_fit("swiglu", w, d)
        w = w.contiguous()
    keep = torch.is_grad_enabled() and (gu.requires_grad or w is not None and w.requires_grad)
    return _Swiglu.apply(_rows(gu), w, d.pair_row, d.row_pair, keep)[0]


def expert_mlp(x: torch.Tensor, w: torch.Tensor, w_gu: torch.Tensor, w_d: torch.Tensor, d: Dispatch) -> torch.Tensor:
    """out[t] = sum_j w[t, j] expert_j(x[t]), expert = down(silu(gate x) * up x): x [T, H] bf16, w [T, k] fp32 as route
    gives it, w_gu [E, 2I, H] (gate rows, then up rows) and w_d [E, H, I] bf16, H and I multiples of 8.  As
    combine(expert_product(swiglu(expert_product(dispatch(x)))), w), with less kept for the backward pass: x [T, H] and
    the gate and up rows [T * k, 2I] in 8 bits, and nothing else of its size.  Differentiable once, as swiglu is."""
    if x.dim() != 2 or x.shape[0] != d.pair_row.shape[0] or x.dtype is not torch.bfloat16:
        raise ValueError(f"expert_mlp: x [{d.pair_row.shape[0]}, H] bf16 is wanted, got {x.dtype} {tuple(x.shape)}")
    _weights_fit("expert_mlp", w, d)
    H = x.shape[1]
    _experts_fit("expert_mlp", w_gu, d, H, "w_gu")
    if w_gu.shape[1] % 2 or w_d.shape != (d.E, H, w_gu.shape[1] // 2):
        raise ValueError(f"expert_mlp: w_gu [{d.E}, 2I, {H}] and w_d [{d.E}, {H}, I] are wanted, got {tuple(w_gu.shape)} "
                         f"and {tuple(w_d.shape)}")
    keep = torch.is_grad_enabled() and any(t.requires_grad for t in (x, w, w_gu, w_d))
    return _ExpertMlp.apply(_rows(x), w.contiguous(), _weights(w_gu), _weights(w_d), d.offs, d.pair_row, d.row_pair,
                            d.status, keep)[0]


# ------------------------------------------------------------------- serving
class Mx4Weights:
    """Expert matrices w [E, N, K] (bf16 or fp32, on the device) quantised to MXFP4 tiles."""

    def __init__(self, w: torch.Tensor):
        self._make(w.shape, w.device)
        moeq.moeq_mx4_quant_weight(w, self.tiles, self.scales)

    @classmethod
    def from_codes(cls, codes: torch.Tensor, scales: torch.Tensor) -> Mx4Weights:
        """From row-major MXFP4 codes [E, N, K/2] and scales [E, N, K/32] (uint8), as a checkpoint holds them."""
        self = cls.__new__(cls)
        E, N, half = codes.shape
        self._make((E, N, 2 * half), codes.device)
        moeq.moeq_mx4_pack_weight(codes, scales, self.tiles, self.scales)
        return self

    def _make(self, shape, device):
        self.E, self.N, self.K = self.shape = tuple(shape)
        self.device = device
        self.tiles, self.scales = moeq.mx4_weight_buffers(self.E, self.N, self.K, device=device)


class _Serve(torch.autograd.Function):
    """Ties the layer's output to inputs that require a gradient, so that a backward pass raises instead of leaving
    them without one."""

    @staticmethod
    def forward(ctx, out, x, logits):
        # a caller's own buffer gathers no history, and the result may be added to in place (a view might not)
        return out.detach()

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("Mx4MoeLayer has no backward pass (route, dispatch and combine train)")


class _Buffers:
    """The buffers of an Mx4MoeLayer call of up to T tokens, and a workspace of ws_bytes."""

    def __init__(self, layer: Mx4MoeLayer, T: int, ws_bytes: int):
        H, I, E, k, device = layer.gu.K, layer.d.K, layer.gu.E, layer.top_k, layer.gu.tiles.device
        new = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=device)
        i32 = torch.int32
        self.T, self.captured = T, False
        self.t = dict(ids=new(T, k, dt=i32), w=new(T, k, dt=torch.float32), offs=new(E + 1, dt=i32),
                      pair_row=new(T, k, dt=i32), row_pair=new(T * k, dt=i32), h=new(T * k, 2 * I), y=new(T * k, H))
        if layer.s_gu is not None:
            # row n of s_offs is {0, n}: rows of another T are not overwritten
            s_offs = torch.zeros((T + 1, 2), dtype=i32, device=device)
            s_offs[:, 1] = torch.arange(T + 1, dtype=i32, device=device)
            self.t.update(sh=new(T, 2 * layer.s_d.K), sy=new(T, H), s_offs=s_offs)
        self.ws = moeq.Workspace(ws_bytes, device=device)   # the products run one after another
        self.streams = {moeq.current_stream_handle()}

    def views(self, T: int, k: int) -> dict:
        n = dict(ids=T, w=T, pair_row=T, row_pair=T * k, h=T * k, y=T * k, sh=T, sy=T)
        v = {name: t[:n[name]] if name in n else t for name, t in self.t.items()}
        if "s_offs" in v:
            v["s_offs"] = v["s_offs"][T]
        return dict(v, ws=self.ws)

    def used(self, capturing: bool) -> None:
        """Notes a call's stream: memory in use there is not given to another's tensors when it is freed."""
        if capturing:
            self.captured = True
            return
        stream = moeq.current_stream_handle()
        if stream not in self.streams:
            for t in (*self.t.values(), self.ws.t):
                t.record_stream(torch.cuda.current_stream())
            self.streams.add(stream)


class Mx4MoeLayer:
    """out = shared(x) + sum_j w_j * expert_j(x), every expert down(silu(gate x) * up x).

    w_gu [E, 2I, H] (gate rows, then up rows), w_d [E, H, I]; shared_gu
    [1, 2I, H] and shared_d [1, H, I], or None for a layer without a shared
    expert.  Each is a tensor or Mx4Weights.

    Buffers are kept for the most tokens seen (``reserve`` makes them
    beforehand), and those that a CUDA graph was captured with for as long as
    the layer lives, so a graph stays valid whatever calls follow.  All calls
    and graphs of one instance share them: they follow one another, on one
    stream or ordered by events."""

    _VIEWS = ("ids", "w", "offs", "pair_row", "row_pair", "h", "y", "sh", "sy", "s_offs", "ws")

    def __init__(self, w_gu, w_d, top_k: int, shared_gu=None, shared_d=None):
        if (shared_gu is None) != (shared_d is None):
            raise ValueError("Mx4MoeLayer: shared_gu and shared_d come together")
        # the products know their weights by the size of their tiles, which is rounded up: other widths are seen here
        H = w_gu.shape[-1]
        for gu, d, what in ((w_gu, w_d, "w"), (shared_gu, shared_d, "shared")):
            if gu is None:
                continue
            E = w_gu.shape[0] if what == "w" else 1
            if len(d.shape) != 3 or gu.shape != (E, 2 * d.shape[2], H) or d.shape != (E, H, d.shape[2]):
                raise ValueError(f"Mx4MoeLayer: {what}_gu [{E}, 2I, {H}] and {what}_d [{E}, {H}, I] are wanted, got "
                                 f"{tuple(gu.shape)} and {tuple(d.shape)}")
            if gu.device != w_gu.device or d.device != w_gu.device:
                raise ValueError("Mx4MoeLayer: the weights lie on different devices")
        tiled = lambda w: w if w is None or isinstance(w, Mx4Weights) else Mx4Weights(w)
        self.gu, self.d, self.s_gu, self.s_d = (tiled(w) for w in (w_gu, w_d, shared_gu, shared_d))
        self.top_k, self.T = top_k, -1   # T: the tokens that the views below are for
        self._kept, self._of_graphs = None, []

    def _ws_bytes(self, T: int) -> int:
        H, I, E, R = self.gu.K, self.d.K, self.gu.E, T * self.top_k
        shapes = [(T, H, 2 * I, E, R), (R, I, H, E, R)]
        if self.s_gu is not None:
            shapes += [(T, H, 2 * self.s_d.K, 1, T), (T, self.s_d.K, H, 1, T)]
        return max(moeq.moeq_mx4_expert_gemm_workspace_size(*s) for s in shapes)

    def reserve(self, T: int) -> None:
        """Makes the buffers for up to T tokens now (not inside a capture: a graph's memory is its own)."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("Mx4MoeLayer.reserve: a CUDA graph is being captured")
        if self._kept is None or T > self._kept.T:
            self._grow(T, self._ws_bytes(T))

    def _grow(self, T: int, ws_bytes: int) -> None:
        old = self._kept
        if old is not None:
            T, ws_bytes = max(T, old.T), max(ws_bytes, old.ws.nbytes)
            if old.captured:
                self._of_graphs.append(old)
        self._kept, self.T, old = None, -1, None   # what no graph uses makes room first
        for name in self._VIEWS:
            self.__dict__.pop(name, None)
        # Fewer tokens, in narrower tiles, may need a little more workspace
        # than T; what a tile's rows (224) more need covers them.
        self._kept = _Buffers(self, T, max(ws_bytes, self._ws_bytes(T), self._ws_bytes(T + 224 // self.top_k + 1)))

    def _buffers(self, T: int) -> None:
        capturing = torch.cuda.is_current_stream_capturing()
        if T != self.T:
            need = self._ws_bytes(T)
            fits = self._kept is not None and T <= self._kept.T and need <= self._kept.ws.nbytes
            if not fits and not capturing:
                self._grow(T, need)
                fits = True
            # Inside a capture, memory and its zeroing belong to the graph: new
            # buffers serve this call alone.
            b = self._kept if fits else _Buffers(self, T, need)
            for name, v in b.views(T, self.top_k).items():
                setattr(self, name, v)
            self.T = T if fits else -1
        if self.T == T:
            self._kept.used(capturing)

    def __call__(self, x: torch.Tensor, logits: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        """x [T, H] bf16, logits [T, E] fp32 -> out [T, H] bf16."""
        # (that all tensors lie on the weights' device, the current one, the calls check)
        shape = x.shape
        T = shape[0]
        if shape != (T, self.gu.K) or logits.shape != (T, self.gu.E):
            raise ValueError(f"x [T, {self.gu.K}] and logits [T, {self.gu.E}] are wanted, got {tuple(shape)} and "
                             f"{tuple(logits.shape)}")
        if out is None:
            out = torch.empty_like(x)
        elif out.shape != shape:
            raise ValueError(f"out: x's shape is wanted, got {tuple(out.shape)}")
        if T == 0:
            return out
        self._buffers(T)
        base = None
        if self.s_gu is not None:
            self._ffn(x, self.s_gu, self.s_d, self.s_offs, self.sh, self.sy, None, 1)
            base = self.sy
        moeq.moeq_route_rows(logits, self.ids, self.w)
        moeq.moeq_expert_sort(self.ids, self.gu.E, self.offs, self.pair_row, self.row_pair)
        self._ffn(x, self.gu, self.d, self.offs, self.h, self.y, self.row_pair, self.top_k)
        moeq.moeq_combine_rows(self.y, self.pair_row, self.w, out, base=base)
        if torch.is_grad_enabled() and (x.requires_grad or logits.requires_grad):
            return _Serve.apply(out.detach(), x, logits)
        return out

    def _ffn(self, x, gu, d, offs, h, y, row_pair, top_k):
        moeq.moeq_mx4_expert_gemm(x, gu.tiles, gu.scales, offs, h, self.ws, row_pair=row_pair, top_k=top_k)
        moeq.moeq_mx4_expert_gemm(h, d.tiles, d.scales, offs, y, self.ws, act=moeq.MOEQ_ACT_SWIGLU)
