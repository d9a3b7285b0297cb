"""GPU parity of the MXFP4 operators: quantisation bit for bit, products
against 64-bit sums of the same quantised operands.

Product tolerance.  Codes times powers of two multiply exactly; the tensor
core adds the 64 products of one MMA and the running sum, each MMA with at
most one truncation of its sum (2^-22 of the terms' magnitude T covers an
aligner that keeps two bits fewer than fp32), K/64 MMAs in a row, plus the
fp32 additions of a cut unit's parts (fewer than 8): (K/64 + 8) 2^-22 T, and
half an ulp of y's type."""
import numpy as np
import pytest
import torch

import rows_plain as rp
from rows_plain import TINY, to64, type_half_ulp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moeq():
    from bandwidth_bound_fp8_gb300 import moeq
    moeq.load()
    return moeq


def _rand(shape, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x = x * torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g))
    return x


def _quant(moeq, x, act=0):
    rows, K = x.shape[0], x.shape[1] // (2 if act else 1)
    q = torch.full((rows, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, moeq.moeq_mx4_scale_pitch(K)), 0xEE, dtype=torch.uint8, device="cuda")
    moeq.moeq_mx4_quant_act(x, q, s, act=act)
    torch.cuda.synchronize()
    return q, s


def _check_quant(moeq, x):
    q, s = _quant(moeq, x)
    code, scale = rp.mx4_codes(to64(x))
    assert np.array_equal(s.cpu().numpy(), rp.pad_scales(scale, s.shape[1]))
    assert np.array_equal(q.cpu().numpy(), rp.pack_codes(code))
    return q, s, code, scale


@pytest.mark.parametrize("rows,K,dtype,spread", [(1, 32, BF, 0), (1, 6144, BF, 4), (3, 96, F32, 4), (17, 160, F32, 20),
                                                 (5, 992, BF, 20), (16, 256, F32, 0), (129, 2048, BF, 2), (2, 32768, F32, 1)])
def test_quant_act_bit_exact(moeq, rows, K, dtype, spread):
    x = _rand((rows, K), rows + K, spread).to(dtype).cuda()
    q, s, code, scale = _check_quant(moeq, x)
    for dt in (BF, F32):
        v = torch.full((rows, K), float("nan"), dtype=dt, device="cuda")
        moeq.moeq_mx4_dequant_act(q, s, v)
        assert np.array_equal(to64(v), rp.mx4_values(code, scale))


def test_quant_act_strided(moeq):
    for dt in (BF, F32):
        wide = _rand((9, 1003), 4, 3).to(dt).cuda()
        x = wide[:, 3:3 + 992]
        _check_quant(moeq, x)
        q, s = _quant(moeq, x)
        out = torch.full((9, 1003), 7.0, dtype=dt, device="cuda")
        moeq.moeq_mx4_dequant_act(q, s, out[:, 3:3 + 992])
        code, scale = rp.mx4_codes(to64(x))
        assert np.array_equal(to64(out[:, 3:3 + 992]), rp.mx4_values(code, scale))
        assert (out[:, :3] == 7).all() and (out[:, 995:] == 7).all()


def test_quant_act_edges(moeq):
    """Ties, powers of two, zeros and negative zeros, saturation, subnormals, the largest numbers, NaN, infinities."""
    x = np.zeros((12, 64), np.float32)
    x[0, :13] = [0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7.9375, -0.25, -0.75, -5]
    x[1, :32] = -np.float32(0)
    x[2] = np.float32(2.0) ** np.arange(-32, 32)
    x[3, :32] = np.float32(1e-40) * np.arange(-16, 16)
    x[3, 32:] = np.float32(1e-45)
    x[4] = np.float32(3.4e38) * np.linspace(-1, 1, 64, dtype=np.float32)
    x[5, 7] = np.nan
    x[5, 32:] = 1
    x[6, 40] = np.inf
    x[6, :32] = -3
    x[7, 0] = -np.inf
    x[8] = np.float32(1.1754944e-38) * np.linspace(0.1, 9, 64, dtype=np.float32)
    x[9, 5] = np.float32(8.0) - np.float32(2.0) ** -21     # rounds to 8 only if x is rounded before
    x[10] = np.float32(4.0)
    x[11, :2] = [np.float32(-6), np.float32(6)]
    q, s, code, scale = _check_quant(moeq, torch.from_numpy(x).cuda())
    assert scale[5].tolist() == [255, 125] and scale[6, 1] == 255 and scale[7, 0] == 255 and scale[1, 0] == 0
    v = torch.empty((12, 64), device="cuda")
    moeq.moeq_mx4_dequant_act(q, s, v)
    ref = rp.mx4_values(code, scale)
    assert np.array_equal(to64(v), ref, equal_nan=True)
    xb = torch.from_numpy(x).to(BF).cuda()
    _check_quant(moeq, xb)


def test_dequant_every_code_and_scale(moeq):
    scale = np.repeat(np.concatenate([np.arange(0, 253), [255]]).astype(np.uint8)[:, None], 1, 1)
    code = np.tile(np.arange(16, dtype=np.uint8), (254, 2))
    q = torch.from_numpy(rp.pack_codes(code)).cuda()
    s = torch.from_numpy(rp.pad_scales(scale, 8)).cuda()
    for dt in (BF, F32):
        v = torch.empty((254, 32), dtype=dt, device="cuda")
        moeq.moeq_mx4_dequant_act(q, s, v)
        assert np.array_equal(to64(v), rp.mx4_values(code, scale), equal_nan=True)


@pytest.mark.parametrize("rows,K,dtype", [(1, 2048, BF), (7, 96, F32), (33, 1408, BF)])
def test_quant_swiglu(moeq, rows, K, dtype):
    """h = silu(g) * u is computed in fp32 within 1e-5 (the fast exponential is within 2 + 1.2 |g| ulp, |g| < 20, the
    fast division within 2): codes and scales must be those of some h in that range."""
    x = (3 * _rand((rows, 2 * K), K)).to(dtype).cuda()
    q, s = _quant(moeq, x, act=moeq.MOEQ_ACT_SWIGLU)
    g, u = to64(x)[:, :K], to64(x)[:, K:]
    h = g / (1 + np.exp(-g)) * u
    lo_s, hi_s = rp.mx4_codes(h * (1 - 1e-5))[1], rp.mx4_codes(h * (1 + 1e-5))[1]
    got_s = s.cpu().numpy()[:, :K // 32]
    assert ((got_s == lo_s) | (got_s == hi_s)).all()
    v = torch.empty((rows, K), device="cuda")
    moeq.moeq_mx4_dequant_act(q, s, v)
    unit = np.repeat(np.exp2(got_s.astype(np.float64) - 127), 32, 1)

    def nearest(a):  # magnitudes, scaled; ties to the even code
        c = np.zeros(a.shape, int)
        for n in range(7):
            mid = (rp.E2M1[n] + rp.E2M1[n + 1]) / 2
            c = np.where(a > mid if n % 2 == 0 else a >= mid, n + 1, c)
        return rp.E2M1[c]

    a = np.abs(h) / unit
    got = np.abs(to64(v)) / unit
    assert ((got >= nearest(a * (1 - 1e-5))) & (got <= nearest(a * (1 + 1e-5)))).all()
    assert ((np.sign(to64(v)) == np.sign(h)) | (got == 0)).all()


@pytest.mark.parametrize("E,N,K,dtype", [(1, 128, 256, F32), (3, 100, 160, BF), (2, 257, 1056, F32), (1, 1, 32, F32)])
def test_weight_tiles(moeq, E, N, K, dtype):
    w = (0.02 * _rand((E, N, K), N + K)).to(dtype).cuda()
    t, st = moeq.mx4_weight_buffers(E, N, K)
    t.fill_(0xEE), st.fill_(0xEE)
    moeq.moeq_mx4_quant_weight(w, t, st)
    code, scale = rp.mx4_codes(to64(w).reshape(E * N, K))
    codes, scale = rp.pack_codes(code).reshape(E, N, K // 2), scale.reshape(E, N, K // 32)
    rt, rs = rp.tiles(codes, scale)
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(st.cpu().numpy(), rs)
    t.fill_(0xEE), st.fill_(0xEE)
    moeq.moeq_mx4_pack_weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(), t, st)
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(st.cpu().numpy(), rs)


# ------------------------------------------------------------------ product
class Weights:
    def __init__(self, moeq, E, N, K, seed):
        w = (0.02 * _rand((E, N, K), seed)).cuda()
        self.t, self.s = moeq.mx4_weight_buffers(E, N, K)
        moeq.moeq_mx4_quant_weight(w, self.t, self.s)
        code, scale = rp.mx4_codes(to64(w).reshape(E * N, K))
        self.v = torch.from_numpy(rp.mx4_values(code, scale).reshape(E, N, K)).cuda()


def _ref(xv, W, counts, rows):
    """y and sum of |terms| in 64 bits; rows: the activation row of each sorted row."""
    R, N = len(rows), W.v.shape[1]
    y, T = torch.zeros((R, N), dtype=torch.float64), torch.zeros((R, N), dtype=torch.float64)
    xv, at = torch.from_numpy(xv).cuda(), 0
    for e, c in enumerate(counts):
        if c:
            a = xv[torch.from_numpy(np.asarray(rows[at:at + c])).long().cuda()]
            y[at:at + c] = (a @ W.v[e].t()).cpu()
            T[at:at + c] = (a.abs() @ W.v[e].abs().t()).cpu()
        at += c
    return y.numpy(), T.numpy()


def _offs(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()


def _close(y, ref, T, K):
    got = to64(y)
    bound = (K / 64 + 8) * 2.0 ** -22 * T + type_half_ulp(y.dtype) * np.abs(ref) * 1.01 + TINY
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"{(err > bound).sum()} outside, worst {np.max(err / (T + 1e-30))} of T"


PRODUCTS = [  # counts per expert, N, K, x type, y type
    ([1], 128, 256, BF, F32),
    ([3], 1, 32, F32, F32),
    ([15], 100, 96, BF, BF),
    ([16], 128, 512, BF, F32),
    ([17], 1000, 1056, F32, BF),
    ([240], 256, 256, BF, BF),
    ([241], 129, 288, BF, F32),
    ([500], 384, 2048, BF, BF),
    ([1, 0, 2, 0, 0, 5, 1, 1], 512, 6144, BF, F32),
    ([0, 0, 130, 1, 0, 33], 300, 1408, F32, BF),
    ([2] * 64, 256, 512, BF, BF),
    ([0, 0, 0], 128, 256, BF, F32),
    ([700, 3, 0, 900, 1100, 260, 17, 1500], 1280, 256, BF, F32),     # many units: whole ones
    ([1500, 700], 2048, 544, BF, BF),
    ([3], 128, 32768, BF, F32),                                      # few units of long K: cut in four
    ([2, 0, 40], 200, 16384, BF, BF),
    ([240], 300, 32768, F32, BF),                                    # cut, by pairs of CTAs
    ([300, 200], 640, 1024, BF, BF),                                 # an odd weight block of a pair
    ([1, 0, 3, 2] * 256, 128, 96, BF, F32),                          # as many experts as there may be
    ([0] * 1022 + [260, 1], 130, 64, BF, BF),
]


@pytest.mark.parametrize("counts,N,K,xt,yt", PRODUCTS)
def test_expert_gemm(moeq, counts, N, K, xt, yt):
    E, R = len(counts), max(sum(counts), 4)
    W = Weights(moeq, E, N, K, N + K)
    x = _rand((R, K), 7, 2).to(xt).cuda()
    y = torch.full((R, N), float("nan"), dtype=yt, device="cuda")
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, E, R))
    code, scale = rp.mx4_codes(to64(x))
    ref, T = _ref(rp.mx4_values(code, scale), W, counts, np.arange(sum(counts)))
    ref = np.concatenate([ref, np.zeros((R - len(ref), N))])
    T = np.concatenate([T, np.zeros((R - len(T), N))])
    first = None
    for _ in range(2):   # the workspace is reusable, and the result the same
        moeq.moeq_mx4_expert_gemm(x, W.t, W.s, _offs(counts), y, ws)
        assert moeq.moeq_read_device_status(ws.t, ws.nbytes) == 0
        _close(y, ref, T, K)
        if first is not None:
            assert torch.equal(first, y)
        first = y.clone()
        y.fill_(float("nan"))
    # codes made beforehand give the same bits
    q, s = _quant(moeq, x)
    moeq.moeq_mx4_expert_gemm(q, W.t, W.s, _offs(counts), y, ws, x_scales=s)
    assert torch.equal(first, y)


@pytest.mark.parametrize("T,k,E,N,K,drop", [(1, 8, 32, 256, 1024, 0), (61, 8, 64, 384, 512, 0.3), (300, 4, 8, 200, 288, 0),
                                            (2, 2, 4, 128, 256, 1.0)])
def test_expert_gemm_gathers_tokens(moeq, T, k, E, N, K, drop):
    """Routed rows: row r reads the token of its pair; slots without an expert leave zero rows at the end."""
    r = np.random.default_rng(T)
    ids = r.integers(0, E, (T, k)).astype(np.int32)
    ids[r.random((T, k)) < drop] = -1
    i32 = dict(dtype=torch.int32, device="cuda")
    offs, pr, rr = torch.empty(E + 1, **i32), torch.empty((T, k), **i32), torch.empty(T * k, **i32)
    moeq.moeq_expert_sort(torch.from_numpy(ids).cuda(), E, offs, pr, rr)
    W = Weights(moeq, E, N, K, 5)
    wide = _rand((T, K + 24), 6, 2).to(BF).cuda()
    x = wide[:, 8:8 + K]
    yw = torch.full((T * k, N + 7), float("nan"), device="cuda")
    y = yw[:, 3:3 + N]
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(T, K, N, E, T * k))
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, offs, y, ws, row_pair=rr, top_k=k)
    kept = int(offs[-1])
    counts = np.diff(offs.cpu().numpy())
    ref, Tm = _ref(rp.mx4_values(*rp.mx4_codes(to64(x))), W, counts, rr.cpu().numpy()[:kept] // k)
    _close(y[:kept], ref, Tm, K)
    assert (y[kept:] == 0).all() and torch.isnan(yw[:, :3]).all() and torch.isnan(yw[:, 3 + N:]).all()
    assert moeq.moeq_read_device_status(ws.t, ws.nbytes) == 0


def test_expert_gemm_swiglu(moeq):
    """The SwiGLU in front gives the bits of the quantiser's own."""
    K, N, R = 288, 200, 37
    W = Weights(moeq, 1, N, K, 3)
    x = (2 * _rand((R, 2 * K), 1)).to(BF).cuda()
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, 1, R))
    y, y2 = torch.empty((R, N), device="cuda"), torch.empty((R, N), device="cuda")
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, _offs([R]), y, ws, act=moeq.MOEQ_ACT_SWIGLU)
    q, s = _quant(moeq, x, act=moeq.MOEQ_ACT_SWIGLU)
    moeq.moeq_mx4_expert_gemm(q, W.t, W.s, _offs([R]), y2, ws, x_scales=s)
    assert torch.equal(y, y2) and torch.isfinite(y).all()


def test_expert_gemm_nan_stays_in_its_row(moeq):
    K, N, R = 256, 128, 20
    W = Weights(moeq, 1, N, K, 4)
    x = _rand((R, K), 2).cuda()
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, 1, R))
    y0, y1 = torch.empty((R, N), device="cuda"), torch.empty((R, N), device="cuda")
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, _offs([R]), y0, ws)
    x[11, 77] = float("inf")
    x[3, 0] = float("nan")
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, _offs([R]), y1, ws)
    torch.cuda.synchronize()
    bad = torch.zeros(R, dtype=torch.bool, device="cuda")
    bad[[3, 11]] = True
    assert torch.isnan(y1[bad]).all() and torch.equal(y1[~bad], y0[~bad])


def test_expert_gemm_bad_plan_stays_in_bounds(moeq):
    """Offsets out of range or order are clamped to [0, R] and pairs to the tokens: no access leaves the buffers,
    the rows between are still the experts'."""
    K, N, R = 256, 128, 10
    W = Weights(moeq, 3, N, K, 4)
    x = _rand((R, K), 2).cuda()
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, 3, R))
    y = torch.zeros((R + 4, N), device="cuda")
    offs = torch.tensor([-3, 4, 2, 1000], dtype=torch.int32, device="cuda")
    rr = torch.tensor([0, 1, 2, 3, 10 ** 6, -1, -2 ** 31, 2 ** 31 - 1, 4, 5], dtype=torch.int32, device="cuda")
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, offs, y[:R], ws, row_pair=rr)
    torch.cuda.synchronize()
    assert (y[R:] == 0).all() and torch.isfinite(y).all()
    assert moeq.moeq_read_device_status(ws.t, ws.nbytes) == 0


def test_expert_gemm_on_another_stream_and_in_a_graph(moeq):
    K, N, R = 512, 256, 5
    W = Weights(moeq, 1, N, K, 9)
    x = _rand((R, K), 2).to(BF).cuda()
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(R, K, N, 1, R))
    y, offs = torch.empty((R, N), device="cuda"), _offs([R])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, offs, y, ws, stream=s)
    s.synchronize()
    want = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moeq.moeq_mx4_expert_gemm(x, W.t, W.s, offs, y, ws)
    y.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_offsets_past_32_bits(moeq):
    """Rows 2^27 elements apart: the last start past 2^32 elements."""
    rows, K, N, ld = 40, 512, 256, 1 << 27
    x0 = _rand((rows, K), 3, 2).to(BF).cuda()
    x = torch.empty(rows * ld, dtype=BF, device="cuda").as_strided((rows, K), (ld, 1))
    x.copy_(x0)
    for a, b in zip(_quant(moeq, x0), _quant(moeq, x)):
        assert torch.equal(a, b)
    W = Weights(moeq, 2, N, K, 8)
    y0 = torch.empty((rows, N), dtype=BF, device="cuda")
    y = torch.empty(rows * ld, dtype=BF, device="cuda").as_strided((rows, N), (ld, 1))
    ws = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(rows, K, N, 2, rows))
    moeq.moeq_mx4_expert_gemm(x0, W.t, W.s, _offs([33, 7]), y0, ws)
    moeq.moeq_mx4_expert_gemm(x, W.t, W.s, _offs([33, 7]), y, ws)
    assert torch.equal(y0, y)
    q, s = _quant(moeq, x0)
    v0 = torch.empty((rows, K), dtype=BF, device="cuda")
    moeq.moeq_mx4_dequant_act(q, s, v0)
    moeq.moeq_mx4_dequant_act(q, s, x)
    assert torch.equal(v0, x)
