"""The calls that expert_layer makes, in torch operations on the CPU: for
tests of what the Python layer itself does with them.  They write through
.data, as the kernels write through pointers: autograd sees none of it."""
from __future__ import annotations

import torch


def _matrix(*tensors):
    """The rows that the binding accepts."""
    for t in tensors:
        if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
            raise ValueError(f"shape {tuple(t.shape)}, strides {t.stride()}")


def route_rows(logits, ids, w, stream=None):
    _matrix(logits)
    k = ids.shape[1]
    v, i = torch.sort(logits.data, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    live = v > -torch.inf
    p = torch.where(live, torch.exp(v - torch.where(live[:, :1], v[:, :1], torch.zeros_like(v[:, :1]))), torch.zeros_like(v))
    ids.data.copy_(torch.where(live, i, torch.full_like(i, -1)))
    w.data.copy_(p / p.sum(1, keepdim=True).clamp(min=1e-30))


def route_rows_grad(dw, ids, w, dl, stream=None):
    live = ids >= 0
    d = torch.where(live, dw.data, torch.zeros_like(dw)) * w.data
    d = d - w.data * d.sum(1, keepdim=True)
    dl.data.zero_().scatter_add_(1, ids.clamp(min=0).long(), torch.where(live, d, torch.zeros_like(d)))


def expert_sort(ids, E, offs, pair_row, row_pair, stream=None):
    flat = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E)).reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    kept = flat[order] < E
    at = torch.arange(flat.numel())
    offs.data[0] = 0
    offs.data[1:] = torch.cumsum(torch.bincount(flat, minlength=E + 1)[:E], 0)
    row_pair.data.copy_(torch.where(kept, order, -1))
    pr = torch.empty_like(at)
    pr[order] = torch.where(kept, at, -1)
    pair_row.data.copy_(pr.view(ids.shape))


def _rows(y, pair_row):
    live = (pair_row >= 0).unsqueeze(2)
    return torch.where(live, y.data[pair_row.clamp(min=0).long()], torch.zeros((), dtype=y.dtype))


def _scatter(out, pair_row, rows):
    live = pair_row >= 0
    out.data.zero_()
    out.data[pair_row[live].long()] = rows[live].to(out.dtype)


def gather_rows(x, offs, pair_row, xs, stream=None):
    _matrix(x, xs)
    _scatter(xs, pair_row, x.data.unsqueeze(1).expand(-1, pair_row.shape[1], -1))


def gather_rows_grad(dxs, pair_row, dx, stream=None):
    _matrix(dxs, dx)
    dx.data.copy_(_rows(dxs, pair_row).sum(1))


def combine_rows(y, pair_row, w, out, base=None, stream=None):
    _matrix(y, out, *([] if base is None else [base]))
    v = (w.data.unsqueeze(2) * _rows(y, pair_row)).sum(1)
    out.data.copy_(v if base is None else v + base.data)


def combine_rows_grad(dout, y, offs, pair_row, w, dy, dw, stream=None):
    _matrix(dout, y, dy)
    _scatter(dy, pair_row, w.data.unsqueeze(2) * dout.data.unsqueeze(1))
    dw.data.copy_((_rows(y, pair_row) * dout.data.unsqueeze(1)).sum(2))


def expert_gemm(x, w, w_scales, offs, y, ws, row_pair=None, top_k=1, act=0, x_scales=None, stream=None):
    R = y.shape[0]
    assert ws.nbytes >= workspace_size(x.shape[0], w.shape[2], w.shape[1], w.shape[0], R)
    rows = torch.arange(R) if row_pair is None else torch.div(row_pair, top_k, rounding_mode="floor")
    a = x.float()
    if act:
        a = torch.nn.functional.silu(a[:, :a.shape[1] // 2]) * a[:, a.shape[1] // 2:]
    y.data.zero_()
    for e in range(w.shape[0]):
        lo, hi = int(offs[e]), int(offs[e + 1])
        y.data[lo:hi] = (a[rows[lo:hi].long()] @ w[e].t()).to(y.dtype)


def weight_buffers(E, N, K, device=None):
    return torch.empty((E, N, K)), torch.empty(0)


def pack_weight(codes, scales, tiles, stiles, stream=None):
    import rows_plain as rp
    E, N, K = tiles.shape
    code = torch.stack((codes & 15, codes >> 4), -1).reshape(E * N, K)
    tiles.copy_(torch.from_numpy(rp.mx4_values(code.numpy(), scales.reshape(E * N, -1).numpy())).reshape(E, N, K))


def workspace_size(rows, K, N, E, R):
    """Any size that does not rise with the rows, as the library's does not where tiles widen."""
    return 4096 + 64 * (R + (16 if R % 3 else 40))


class Workspace:
    def __init__(self, nbytes, device=None, stream=None):
        self.nbytes, self.t = nbytes, torch.zeros(nbytes, dtype=torch.uint8)


def use(monkeypatch):
    """Replaces the calls; returns what the test may set: whether a graph is being captured, and the current stream."""
    import types
    from bandwidth_bound_fp8_gb300 import moeq
    state = types.SimpleNamespace(capturing=False, stream=0)
    for f in (route_rows, route_rows_grad, expert_sort, gather_rows, gather_rows_grad, combine_rows, combine_rows_grad):
        monkeypatch.setattr(moeq, "moeq_" + f.__name__, f)
    monkeypatch.setattr(moeq, "moeq_mx4_expert_gemm", expert_gemm)
    monkeypatch.setattr(moeq, "moeq_mx4_expert_gemm_workspace_size", workspace_size)
    monkeypatch.setattr(moeq, "mx4_weight_buffers", weight_buffers)
    monkeypatch.setattr(moeq, "moeq_mx4_quant_weight", lambda w, tiles, scales, stream=None: tiles.copy_(w))
    monkeypatch.setattr(moeq, "moeq_mx4_pack_weight", pack_weight)
    monkeypatch.setattr(moeq, "Workspace", Workspace)
    monkeypatch.setattr(moeq, "current_stream_handle", lambda: state.stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    return state
