"""The MXFP4 product's ways through its launcher: tokens quantised once and
their codes gathered (4096 rows or more), quantised while they are
gathered, codes given with an index, SwiGLU in front of any of them, and row
counts around the widths of a token tile.  Tolerances as in test_gpu_mx4."""
import numpy as np
import pytest
import torch

import rows_plain as rp
from rows_plain import to64
from test_gpu_mx4 import BF, F32, Weights, _close, _offs, _quant, _rand, _ref, moeq  # noqa: F401

pytestmark = pytest.mark.gpu


def _routed(moeq, T, k, E, drop, seed):  # noqa: F811
    r = np.random.default_rng(seed)
    ids = np.argsort(r.random((T, E)), 1)[:, :k].astype(np.int32) if E >= k else r.integers(0, E, (T, k)).astype(np.int32)
    ids[r.random((T, k)) < drop] = -1
    i32 = dict(dtype=torch.int32, device="cuda")
    offs, pr, rr = torch.empty(E + 1, **i32), torch.empty((T, k), **i32), torch.empty(T * k, **i32)
    moeq.moeq_expert_sort(torch.from_numpy(ids).cuda(), E, offs, pr, rr)
    return offs, rr


# T * k below 4096 rows, at it, above; odd K blocks; one row's width off 16 bytes (strided)
GATHERED = [  # T, k, E, N, K, drop, x type, y type, swiglu, strided
    (1365, 3, 12, 200, 288, 0.0, BF, F32, False, False),      # 4095 rows: quantised while gathered
    (512, 8, 32, 200, 288, 0.0, BF, F32, False, False),       # 4096: once
    (512, 8, 32, 136, 1056, 0.25, F32, BF, False, False),
    (2048, 2, 3, 128, 96, 0.0, F32, F32, False, True),
    (1025, 4, 60, 257, 544, 0.5, BF, BF, False, True),
    (900, 8, 256, 100, 320, 0.0, BF, BF, True, False),
    (2500, 2, 5, 128, 160, 0.3, F32, F32, True, True),
    (4096, 2, 1, 64, 64, 0.9, BF, F32, False, False),         # most slots without an expert
    (37, 4, 8, 200, 288, 0.2, F32, F32, True, False),         # few rows, SwiGLU in fp32 while gathered
    (41, 3, 4, 129, 1056, 0.0, BF, BF, True, True),
    (2100, 2, 4, 64, 32, 1.0, BF, BF, False, False),          # no rows at all
]


@pytest.mark.parametrize("T,k,E,N,K,drop,xt,yt,swiglu,strided", GATHERED)
def test_gathered_product(moeq, T, k, E, N, K, drop, xt, yt, swiglu, strided):  # noqa: F811
    offs, rr = _routed(moeq, T, k, E, drop, T + K)
    W = Weights(moeq, E, N, K, 5)
    width = K * (2 if swiglu else 1)
    x = (1.5 * _rand((T, width + 13), 6, 0.5 if swiglu else 2)).to(xt).cuda()[:, 3:3 + width]
    if not strided:
        x = x.contiguous()
    act = moeq.MOEQ_ACT_SWIGLU if swiglu else moeq.MOEQ_ACT_NONE
    R, kept = T * k, int(offs[-1])
    y = torch.full((R, N), float("nan"), dtype=yt, device="cuda")
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(T, K, N, E, R))
    for _ in range(2):
        y.fill_(float("nan"))
        moeq.moeq_mx4_expert_gemm(x, W.t, W.s, offs, y, ws, row_pair=rr, top_k=k, act=act)
    # the values of the quantiser, which has its own tests (bit for bit without SwiGLU)
    q, s = _quant(moeq, x, act=act)
    v = torch.empty((T, K), device="cuda")
    moeq.moeq_mx4_dequant_act(q, s, v)
    if not swiglu:
        assert np.array_equal(to64(v), rp.mx4_values(*rp.mx4_codes(to64(x))))
    tokens = rr.cpu().numpy()[:kept] // k
    ref, terms = _ref(to64(v), W, np.diff(offs.cpu().numpy()), tokens)
    _close(y[:kept], ref, terms, K)
    assert (y[kept:] == 0).all()
    # codes given with the same index: the same bits
    y2 = torch.full((R, N), float("nan"), dtype=yt, device="cuda")
    moeq.moeq_mx4_expert_gemm(q, W.t, W.s, offs, y2, ws, row_pair=rr, top_k=k, x_scales=s)
    assert torch.equal(y, y2)
    # and the rows laid out by the caller, without an index
    rows = torch.zeros(R, dtype=torch.long, device="cuda")
    rows[:kept] = torch.from_numpy(tokens).long().cuda()
    big = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, E, R))
    moeq.moeq_mx4_expert_gemm(x[rows], W.t, W.s, offs, y2, big, act=act)
    assert torch.equal(y, y2)
    assert moeq.moeq_read_device_status(ws.t, ws.nbytes) == 0 and moeq.moeq_read_device_status(big.t, big.nbytes) == 0


@pytest.mark.parametrize("rows", [199, 200, 207, 208, 209, 223, 224, 225, 416, 417, 448, 449])
@pytest.mark.parametrize("E", [1, 3])
def test_rows_around_a_tiles_width(moeq, rows, E):  # noqa: F811
    """One CTA a tile up to 199 rows, pairs from 200, two tiles from 225 (one expert; more where the average is less)."""
    N, K = 300, 544
    counts = [rows] if E == 1 else [rows, 1, rows // 2]
    R = sum(counts)
    W = Weights(moeq, E, N, K, rows)
    x = _rand((R, K), rows, 2).to(BF).cuda()
    ref, terms = _ref(rp.mx4_values(*rp.mx4_codes(to64(x))), W, counts, np.arange(R))
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, E, R))
    for yt in (BF, F32):
        y = torch.full((R, N), float("nan"), dtype=yt, device="cuda")
        moeq.moeq_mx4_expert_gemm(x, W.t, W.s, _offs(counts), y, ws)
        _close(y, ref, terms, K)
    assert moeq.moeq_read_device_status(ws.t, ws.nbytes) == 0


@pytest.mark.parametrize("R,K,N,xt", [(1, 2048, 6144, BF), (19, 2048, 6144, F32), (250, 1408, 640, F32), (3, 16384, 128, F32)])
def test_down_product_with_swiglu(moeq, R, K, N, xt):  # noqa: F811
    """A layer's second product: SwiGLU in front, rows in order, several experts; the last one is cut along K."""
    counts = [R // 2, 0, R - R // 2]
    W = Weights(moeq, 3, N, K, 11)
    x = (1.5 * _rand((R, 2 * K), 12)).to(xt).cuda()
    q, s = _quant(moeq, x, act=moeq.MOEQ_ACT_SWIGLU)
    v = torch.empty((R, K), device="cuda")
    moeq.moeq_mx4_dequant_act(q, s, v)
    ref, terms = _ref(to64(v), W, counts, np.arange(R))
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, 3, R))
    y = torch.full((R, N), float("nan"), device="cuda")
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, _offs(counts), y, ws, act=moeq.MOEQ_ACT_SWIGLU)
    _close(y, ref, terms, K)
    assert moeq.moeq_read_device_status(ws.t, ws.nbytes) == 0


def test_dequant_of_the_largest_scales(moeq):  # noqa: F811
    """Scales 2^126 and 2^127, which the quantiser does not make: values past the type's largest are infinities."""
    scale = np.array([[253], [254]], np.uint8)
    code = np.tile(np.arange(16, dtype=np.uint8), (2, 2))
    q, s = torch.from_numpy(rp.pack_codes(code)).cuda(), torch.from_numpy(rp.pad_scales(scale, 8)).cuda()
    ref = rp.mx4_values(code, scale)
    for dt in (BF, F32):
        v = torch.empty((2, 32), dtype=dt, device="cuda")
        moeq.moeq_mx4_dequant_act(q, s, v)
        with np.errstate(over="ignore"):
            want = np.where(np.abs(ref) > np.finfo(np.float32).max, np.copysign(np.inf, ref), ref)
        assert np.array_equal(to64(v), want)
