"""GPU parity of the operators on any number of tokens that move and route:
moeq_route_rows, moeq_expert_sort, moeq_gather_rows, moeq_combine_rows and
their gradients, against plain 64-bit forms.  Indices must match exactly.

Tolerances, from the operators' roundings (U24 = 2^-24, half an fp32 ulp):
  * weights: w = p / sum p, p = expf(l - l0).  The subtraction rounds an
    argument of size d (d U24 relative in p), expf is within 2 ulp (4 U24), the
    sum takes at most 5 additions and the division rounds once; numerator and
    denominator carry the first two: (2 (d + 4) + 6) U24, relative.
  * combine: k + 1 fused multiply-adds and the final rounding.
  * dw: a thread adds ceil(H/256) + 8 products at most in one chain, then 5
    shuffles and 8 warps: (ceil(H/256) + 24) U24 of the sum of |terms|.
"""
import numpy as np
import pytest
import torch

import rows_plain as rp
from rows_plain import TINY, U24, to64, type_half_ulp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moeq():
    from bandwidth_bound_fp8_gb300 import moeq
    moeq.load()
    return moeq


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _poison(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _within(got, ref, bound, what):
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), f"{what}: {(err > bound).sum()} outside, worst {np.max(err - bound)}"


# ------------------------------------------------------------------ routing
def _route(moeq, logits, k):
    T = logits.shape[0]
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = _poison((T, k), F32)
    moeq.moeq_route_rows(logits, ids, w)
    torch.cuda.synchronize()
    return ids, w


def _check_route(moeq, logits, k):
    ids, w = _route(moeq, logits, k)
    lg = to64(logits)
    ref_id, ref_w = rp.route(lg, k)
    assert np.array_equal(ids.cpu().numpy(), ref_id)
    top = np.minimum(np.where(np.isnan(lg), -np.inf, lg), np.finfo(np.float32).max)
    picked = np.take_along_axis(top, np.maximum(ref_id, 0), 1)
    d = np.where(ref_id >= 0, np.abs(picked - picked[:, :1]), 0.0)
    d = np.minimum(np.nan_to_num(d), 110.0).max(1, keepdims=True)
    _within(to64(w), ref_w, (2 * (d + 4) + 6) * U24 * ref_w + TINY, "weights")
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (16, 256, 8), (1, 1, 1), (7, 8, 8), (33, 60, 4), (130, 1000, 16),
                                   (65, 384, 1), (5, 64, 6), (513, 65, 3), (9, 1024, 8)])
def test_route_rows(moeq, T, E, k):
    lg = (2 * torch.randn((T, E), generator=_gen(T * 7 + E))).to(BF).float()   # bf16 values: ties occur
    _check_route(moeq, lg.cuda(), k)


def test_route_rows_masks(moeq):
    """Rows that a mask leaves empty or short, NaN, infinities, the type's lowest value, ties over everything."""
    E, k = 40, 4
    lg = torch.randn((10, E), generator=_gen(5))
    low = torch.finfo(F32).min
    lg[0] = float("-inf")
    lg[1] = float("-inf")
    lg[1, 37] = 0.5
    lg[2, ::2] = float("nan")
    lg[3] = float("nan")
    lg[4] = low
    lg[5, 3:] = low
    lg[6, 11] = float("inf")
    lg[6, 12] = float("inf")
    lg[7] = 0.0
    lg[7, 1::2] = -0.0
    lg[8] = low
    lg[8, 20] = 1e38
    ids, w = _check_route(moeq, lg.cuda(), k)
    assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[3] == -1).all()
    assert ids[1].tolist() == [37, -1, -1, -1] and w[1].tolist() == [1, 0, 0, 0]
    assert ids[4].tolist() == [0, 1, 2, 3] and ids[7].tolist() == [0, 1, 2, 3]


def test_route_rows_strided_and_other_stream(moeq):
    wide = torch.randn((37, 300), generator=_gen(8)).cuda()
    lg = wide[:, 13:13 + 200]
    _check_route(moeq, lg, 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids = torch.empty((37, 5), dtype=torch.int32, device="cuda")
    w = torch.empty((37, 5), device="cuda")
    moeq.moeq_route_rows(lg, ids, w, stream=s)
    s.synchronize()
    assert np.array_equal(ids.cpu().numpy(), rp.route(to64(lg), 5)[0])


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (19, 60, 4), (40, 1001, 16), (3, 1, 1)])
def test_route_rows_grad(moeq, T, E, k):
    lg = torch.randn((T, E), generator=_gen(T + E))
    if E > 8:
        lg[0, 3:] = float("-inf")   # three picks are left to row 0
    lg = lg.cuda()
    ids, w = _route(moeq, lg, k)
    dw = torch.randn((T, k), generator=_gen(3)).cuda()
    wide = _poison((T, E + 5), F32)
    for dl in (_poison((T, E), F32), wide[:, 2:2 + E]):
        moeq.moeq_route_rows_grad(dw, ids, w, dl)
        torch.cuda.synchronize()
        w64, g64, i = to64(w), to64(dw), ids.cpu().numpy()
        live = i >= 0
        d = w64 * (g64 - (w64 * g64).sum(1, keepdims=True))
        mag = w64 * (np.abs(g64) + (w64 * np.abs(g64)).sum(1, keepdims=True))
        ref, bound = np.zeros((T, E)), np.zeros((T, E))
        for t in range(T):
            ref[t, i[t][live[t]]] = d[t][live[t]]
            bound[t, i[t][live[t]]] = mag[t][live[t]] * (k + 4) * U24
        _within(to64(dl), ref, bound + TINY, "d_logits")
    assert torch.isnan(wide[:, :2]).all() and torch.isnan(wide[:, 2 + E:]).all()


def test_route_rows_grad_is_the_derivative(moeq):
    """Central differences of the 64-bit forward: h^2 |f'''| / 6 with h = 1e-4 and third derivatives below 10 gives
    2e-8; the kernel's own roundings are below 20 U24 of values below 10."""
    T, E, k, h = 6, 12, 4, 1e-4
    lg = torch.randn((T, E), generator=_gen(11))
    dw = torch.randn((T, k), generator=_gen(12))
    ids, w = _route(moeq, lg.cuda(), k)
    dl = torch.empty((T, E), device="cuda")
    moeq.moeq_route_rows_grad(dw.cuda(), ids, w, dl)
    got, base, g = to64(dl), to64(lg), to64(dw)
    i = ids.cpu().numpy()

    def loss(z):
        v = np.take_along_axis(z, i, 1)
        p = np.exp(v - v.max(1, keepdims=True))
        return ((p / p.sum(1, keepdims=True)) * g).sum()

    for t in range(T):
        for e in range(E):
            up, dn = base.copy(), base.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((loss(up) - loss(dn)) / (2 * h) - got[t, e]) <= 2e-8 + 200 * U24


# --------------------------------------------------------------------- sort
def _ids(T, k, E, drop, seed):
    r = np.random.default_rng(seed)
    ids = r.integers(0, E, (T, k)).astype(np.int32)
    if drop:
        out = r.random((T, k)) < drop
        ids[out] = r.choice(np.array([-1, E, -2 ** 31, 2 ** 31 - 1, E + 1], np.int64), (T, k))[out].astype(np.int32)
    return ids


def _sort(moeq, ids, E):
    T, k = ids.shape
    full = lambda *s: torch.full(s, -99, dtype=torch.int32, device="cuda")
    o, pr, rr = full(E + 1), full(T, k), full(T * k)
    moeq.moeq_expert_sort(torch.from_numpy(ids).cuda(), E, o, pr, rr)
    torch.cuda.synchronize()
    return o, pr, rr


@pytest.mark.parametrize("T,k,E,drop", [(0, 2, 8, 0), (1, 1, 1, 0), (1, 8, 256, 0), (16, 8, 256, 0), (256, 8, 60, 0.3),
                                        (257, 8, 60, 0.3), (4096, 8, 256, 0), (33001, 8, 1024, 0.1),
                                        (2049, 16, 1000, 0.9), (700, 3, 5, 1.0), (1000, 2, 1, 0)])
def test_expert_sort(moeq, T, k, E, drop):
    ids = _ids(T, k, E, drop, T + E)
    got = _sort(moeq, ids, E)
    for g, ref in zip(got, rp.sort_pairs(ids, E)):
        assert np.array_equal(g.cpu().numpy(), ref)


def test_expert_sort_one_expert_takes_all(moeq):
    ids = np.full((3000, 4), 7, np.int32)
    o, pr, rr = _sort(moeq, ids, 9)
    assert np.array_equal(rr.cpu().numpy(), np.arange(12000)) and np.array_equal(pr.cpu().numpy().reshape(-1), np.arange(12000))
    assert o.tolist() == [0] * 8 + [12000, 12000]


# ---------------------------------------------------------------- movement
def _matrix(rows, H, dtype, strided, seed):
    x = torch.randn((rows, H), generator=_gen(seed)).to(dtype).cuda()
    if not strided:
        return x
    wide = torch.full((rows, H + 13), 3.0, dtype=dtype, device="cuda")
    wide[:, 5:5 + H] = x
    return wide[:, 5:5 + H]


CASES = [  # T, H, k, E, y type, out type, base, drop, strided
    (1, 6144, 8, 256, BF, BF, True, 0, False),
    (16, 6144, 8, 256, F32, BF, True, 0.2, False),
    (33, 1001, 4, 60, BF, BF, False, 0.2, False),
    (33, 1000, 4, 60, BF, F32, True, 0.5, True),
    (5, 1, 16, 20, F32, F32, True, 0.2, False),
    (9, 7, 16, 20, BF, F32, False, 0, True),
    (300, 136, 9, 31, F32, F32, True, 0.1, False),
    (300, 2048, 2, 8, BF, BF, False, 1.0, False),   # no slot has a row
    (130, 5120, 1, 3, BF, BF, False, 0, False),
]


@pytest.mark.parametrize("T,H,k,E,yt,ot,base,drop,strided", CASES)
def test_rows_move_and_come_back(moeq, T, H, k, E, yt, ot, base, drop, strided):
    ids = _ids(T, k, E, drop, T * H)
    offs, pair_row, row_pair = _sort(moeq, ids, E)
    pr, kept = pair_row.cpu().numpy(), int(offs[-1])
    R, live = T * k, pr >= 0
    out_like = lambda rows, dt: (_poison((rows, H + 13), dt)[:, 5:5 + H] if strided else _poison((rows, H), dt))

    x, xs = _matrix(T, H, yt, strided, 1), out_like(R, yt)
    moeq.moeq_gather_rows(x, offs, pair_row, xs)
    ref = np.zeros((R, H))
    for j in range(k):
        ref[pr[live[:, j], j]] = to64(x)[live[:, j]]
    assert np.array_equal(to64(xs), ref)

    # rows past the kept ones hold garbage that must not be read
    y, w = _matrix(R, H, yt, strided, 2), torch.randn((T, k), generator=_gen(3)).cuda()
    y[kept:] = float("nan")
    b = _matrix(T, H, ot, strided, 4) if base else None
    out = out_like(T, ot)
    moeq.moeq_combine_rows(y, pair_row, w, out, base=b)
    y64, w64 = np.nan_to_num(to64(y)), to64(w)
    yj = np.where(live[..., None], y64[np.maximum(pr, 0)], 0.0)
    ref = (w64[..., None] * yj).sum(1) + (to64(b) if base else 0)
    mag = (np.abs(w64)[..., None] * np.abs(yj)).sum(1) + (np.abs(to64(b)) if base else 0)
    _within(to64(out), ref, (k + 1) * U24 * mag * 1.01 + type_half_ulp(ot) * np.abs(ref) * 1.01 + TINY, "out")

    dxs, dx = _matrix(R, H, yt, strided, 5), out_like(T, yt)
    dxs[kept:] = float("nan")
    moeq.moeq_gather_rows_grad(dxs, pair_row, dx)
    dj = np.where(live[..., None], np.nan_to_num(to64(dxs))[np.maximum(pr, 0)], 0.0)
    ref, mag = dj.sum(1), np.abs(dj).sum(1)
    _within(to64(dx), ref, k * U24 * mag * 1.01 + type_half_ulp(yt) * np.abs(ref) * 1.01 + TINY, "dx")

    do = _matrix(T, H, ot, strided, 6)
    dy, dw = out_like(R, yt), _poison((T, k), F32)
    moeq.moeq_combine_rows_grad(do, y, offs, pair_row, w, dy, dw)
    do64 = to64(do)
    ref = np.zeros((R, H))
    for j in range(k):
        t = live[:, j]
        ref[pr[t, j]] = w64[t, j, None] * do64[t]
    _within(to64(dy), ref, (U24 + type_half_ulp(yt)) * np.abs(ref) * 1.01 + TINY, "dy")
    assert (to64(dy)[kept:] == 0).all()
    ref, mag = (yj * do64[:, None]).sum(2), (np.abs(yj) * np.abs(do64)[:, None]).sum(2)
    _within(to64(dw), ref, (-(-H // 256) + 24) * U24 * mag + TINY, "dw")
    assert (to64(dw)[~live] == 0).all()


def test_movement_grads_are_derivatives(moeq):
    """The movement is linear, so a central difference of any step is its derivative: <dL, delta> against
    (L(+delta) - L(-delta)) / 2 of the kernels' own forward passes, in fp32 with sums in 64 bits.  Each output is
    within (k + 2) U24 of its terms, on either side of the difference."""
    T, H, k, E = 21, 264, 5, 7
    ids = _ids(T, k, E, 0.2, 9)
    offs, pair_row, _ = _sort(moeq, ids, E)
    pr = pair_row.cpu().numpy()
    kept, R = int(offs[-1]), T * k
    rnd = lambda s, *shape: torch.randn(shape, generator=_gen(s)).cuda()
    y, w, do, x, dxs = rnd(1, R, H), rnd(2, T, k), rnd(3, T, H), rnd(4, T, H), rnd(5, R, H)
    dy, dw, dx = torch.empty_like(y), torch.empty_like(w), torch.empty_like(x)
    moeq.moeq_combine_rows_grad(do, y, offs, pair_row, w, dy, dw)
    moeq.moeq_gather_rows_grad(dxs, pair_row, dx)

    def combined(yy, ww):
        out = torch.empty((T, H), device="cuda")
        moeq.moeq_combine_rows(yy, pair_row, ww, out)
        return (to64(out) * to64(do)).sum()

    def gathered(xx):
        xs = torch.empty((R, H), device="cuda")
        moeq.moeq_gather_rows(xx, offs, pair_row, xs)
        return (to64(xs) * to64(dxs))[:kept].sum()

    # every product below has factors under 6 (normal draws), T * H * k of them
    bound = 4 * (k + 2) * U24 * 6 * 6 * 6 * T * H * k
    d = rnd(6, R, H)
    got = (to64(dy) * to64(d)).sum()
    assert abs((combined(y + d, w) - combined(y - d, w)) / 2 - got) <= bound
    d = rnd(7, T, k)
    d[torch.from_numpy(pr < 0).cuda()] = 0
    assert abs((combined(y, w + d) - combined(y, w - d)) / 2 - (to64(dw) * to64(d)).sum()) <= bound
    d = rnd(8, T, H)
    assert abs((gathered(x + d) - gathered(x - d)) / 2 - (to64(dx) * to64(d)).sum()) <= bound


def test_zero_tokens(moeq):
    e = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")
    i32 = torch.int32
    moeq.moeq_route_rows(e(0, 8), e(0, 2, dt=i32), e(0, 2))
    moeq.moeq_route_rows_grad(e(0, 2), e(0, 2, dt=i32), e(0, 2), e(0, 8))
    offs = torch.full((9,), 5, dtype=i32, device="cuda")
    moeq.moeq_expert_sort(e(0, 2, dt=i32), 8, offs, e(0, 2, dt=i32), e(0, dt=i32))
    moeq.moeq_gather_rows(e(0, 16), offs, e(0, 2, dt=i32), e(0, 16))
    moeq.moeq_combine_rows(e(0, 16), e(0, 2, dt=i32), e(0, 2), e(0, 16))
    moeq.moeq_gather_rows_grad(e(0, 16), e(0, 2, dt=i32), e(0, 16))
    moeq.moeq_combine_rows_grad(e(0, 16), e(0, 16), offs, e(0, 2, dt=i32), e(0, 2), e(0, 16), e(0, 2))
    torch.cuda.synchronize()
    assert (offs == 0).all()


def test_bad_indices_stay_in_bounds(moeq):
    """Row numbers out of range name no row: nothing is read or written for them."""
    T, H, k = 4, 64, 2
    pr = torch.tensor([[0, 99], [-5, 3], [2 ** 31 - 1, 1], [-2 ** 31, 8]], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    x, w = torch.randn((T, H)).cuda(), torch.ones((T, k), device="cuda")
    xs = torch.zeros((T * k, H), device="cuda")
    moeq.moeq_gather_rows(x, offs, pr, xs)
    out = torch.empty((T, H), device="cuda")
    moeq.moeq_combine_rows(xs, pr, w, out)
    torch.cuda.synchronize()
    assert torch.equal(xs[0], x[0]) and torch.equal(xs[3], x[1]) and torch.equal(xs[1], x[2]) and (xs[4:] == 0).all()
    assert torch.equal(out[:3], x[:3]) and (out[3] == 0).all()


def test_offsets_past_32_bits(moeq):
    """Rows 2^27 elements apart: the last start past 2^32 elements.  Results are those of packed rows, bit for bit."""
    T, k, H, E, ld = 20, 2, 136, 5, 1 << 27
    ids = _ids(T, k, E, 0.1, 4)
    offs, pr, _ = _sort(moeq, ids, E)
    w = torch.rand((T, k), generator=_gen(1)).cuda()
    x0, y0, do0 = (_matrix(n, H, BF, False, s) for n, s in ((T, 2), (T * k, 3), (T, 4)))
    far = [torch.empty(T * k * ld, dtype=BF, device="cuda") for _ in range(2)]
    rows = lambda i, n: far[i].as_strided((n, H), (ld, 1))

    def run(x, y, do, new):
        res = []
        xs = new(T * k)
        moeq.moeq_gather_rows(x, offs, pr, xs)
        res.append(xs.clone())
        dx = torch.empty((T, H), dtype=BF, device="cuda")
        moeq.moeq_gather_rows_grad(xs, pr, dx)
        out = torch.empty((T, H), dtype=BF, device="cuda")
        moeq.moeq_combine_rows(y, pr, w, out, base=do)
        dy, dw = new(T * k), torch.empty((T, k), device="cuda")
        moeq.moeq_combine_rows_grad(do, y, offs, pr, w, dy, dw)
        return res + [dx, out, dy.clone(), dw]

    near = run(x0, y0, do0, lambda n: torch.empty((n, H), dtype=BF, device="cuda"))
    y = rows(1, T * k)
    y.copy_(y0)
    for a, b in zip(near, run(x0, y, do0, lambda n: rows(0, n))):
        assert torch.equal(a, b)
