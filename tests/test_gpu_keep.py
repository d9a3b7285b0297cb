"""Activations in 8 bits, and SwiGLU from them: codes and scales bit for bit
against the definition, values and gradients against 64 bits.

Tolerances in steps u = 2^-24 (half a step of fp32): the sigmoid is an
exponential (2 steps), a sum, and a reciprocal (1 step), 4 steps = 8 u; for bf16
rows the exponent g log2 e is a rounded product with a rounded constant, u |g|
each.  Every product or sum after it adds u.  A dot product of n terms adds at
most (n/8 + 40) u of the sum of |terms| (a lane's run of additions, then a
tree).  At the end half a step of the output's type."""
import numpy as np
import pytest
import torch

import keep_plain as kp
import rows_plain as rp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = rp.U24


def _rand(seed, *shape, dt=F32, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dt).cuda()


def _kept(rows, K, halves=1):
    from bandwidth_bound_fp8_gb300 import moeq
    return (torch.full((rows, halves * K), 255, dtype=torch.uint8, device="cuda"),
            torch.full((rows, halves * moeq.fp8_groups(K)), -1.0, device="cuda"))


def _quant(x):
    from bandwidth_bound_fp8_gb300 import moeq
    codes, scales = _kept(*x.shape)
    moeq.moeq_fp8_quant_rows(x, codes, scales)
    return codes, scales


def _same_codes(x, codes, scales):
    c, s = kp.keep(kp.to_np(x))
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    got = codes.cpu().numpy()
    assert np.array_equal(got, c), f"{(got != c).sum()} codes differ, first at {np.argwhere(got != c)[0]}"


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (1, 8), (5, 100), (2, 128), (7, 129), (33, 136), (4, 1001), (17, 2048),
                                    (9, 6144), (300, 384), (2, 40000)])
def test_codes_and_values(rows, K, dt):
    from bandwidth_bound_fp8_gb300 import moeq
    x = _rand(rows + K, rows, K, dt=dt)
    x[:, ::97] *= 30
    codes, scales = _quant(x)
    _same_codes(x, codes, scales)
    v = kp.values(codes.cpu().numpy(), scales.cpu().numpy())
    for out_dt in (BF, F32):
        out = torch.full((rows, K), float("nan"), dtype=out_dt, device="cuda")
        moeq.moeq_fp8_dequant_rows(codes, scales, out)
        assert torch.equal(out.cpu(), torch.from_numpy(v).to(out_dt))
    # half a step: 2^-4 of what has a normal code, 2^-10 of the scale below
    err = np.abs(v.astype(np.float64) - rp.to64(x))
    s = np.repeat(scales.cpu().numpy().astype(np.float64), 128, axis=1)[:, :K]
    assert (err <= (2.0 ** -4 * np.abs(rp.to64(x)) + 2.0 ** -10 * s) * (1 + 4 * U)).all()


@pytest.mark.parametrize("seed", range(4))
def test_codes_at_the_borders(seed):
    """Quotients at every midpoint between two codes, and up to six steps of fp32 beside it."""
    g = np.random.default_rng(seed)
    mids = np.concatenate([(kp.E4M3[:-1] + kp.E4M3[1:]) / 2, kp.E4M3])
    rows = []
    for top in g.uniform(0.1, 1000, 60).astype(np.float32):
        s = np.float32(top / np.float32(448))
        x = (mids * float(s)).astype(np.float32)
        x = x[x < top]
        x = (x.view(np.int32) + g.integers(-6, 7, len(x)).astype(np.int32) * (x > 0)).view(np.float32)
        x = np.abs(x) * np.where(g.random(len(x)) < 0.5, -1, 1).astype(np.float32)
        x = np.where(np.abs(x) > top, top, x)
        for i in range(0, len(x), 127):
            b = np.zeros(128, np.float32)
            b[0] = top
            b[1:1 + len(x[i:i + 127])] = x[i:i + 127]
            rows.append(b)
    x = torch.from_numpy(np.stack(rows)).cuda()
    _same_codes(x, *_quant(x))


def test_ties_of_bf16():
    """Every bf16 significand over every amax significand: quotients that are ties between two codes are common."""
    tops = torch.arange(128, 256, dtype=torch.float32)
    x = torch.zeros((128, 1024))
    for i in range(8):
        x[:, 128 * i:128 * (i + 1)] = torch.arange(128, 256, dtype=torch.float32) * 2.0 ** -(i + 1) * torch.tensor([1.0, -1.0]).repeat(64)
        x[:, 128 * i] = tops
    x = x.to(BF).cuda()
    codes, scales = _quant(x)
    _same_codes(x, codes, scales)
    q = (x.float().cpu() / scales.cpu().repeat_interleave(128, 1)).double().abs()
    mids = torch.from_numpy((kp.E4M3[:-1] + kp.E4M3[1:]) / 2)
    assert torch.isin(q, mids).sum() > 500


def test_extreme_groups():
    """Zeros of both signs, the smallest and the largest numbers, and groups that are not finite."""
    x = torch.zeros((12, 300))
    x[1] = -0.0
    x[2, 5], x[2, 200] = 1e-45, -3e-43
    x[3] = 1.1e-38 * torch.arange(300)
    x[4] = 3.4e38
    x[5, 0], x[5, 299] = 3.4e38, -1e-30
    x[6] = torch.randn(300, generator=torch.Generator().manual_seed(1)) * 1e-36
    x[7, 3] = float("nan")
    x[8, 130] = float("inf")
    x[9, 299] = -float("inf")
    x[10] = torch.randn(300, generator=torch.Generator().manual_seed(2)) * 1e-42
    x = x.cuda()
    codes, scales = _quant(x)
    _same_codes(x, codes, scales)
    from bandwidth_bound_fp8_gb300 import moeq
    out = torch.empty_like(x)
    moeq.moeq_fp8_dequant_rows(codes, scales, out)
    bad = torch.isnan(out).cpu()
    want = torch.zeros_like(bad)
    want[7, :128], want[8, 128:256], want[9, 256:] = True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K,off,gap", [(136, 8, 8), (136, 3, 0), (101, 1, 6)])
def test_strided_rows(K, off, gap, dt):
    from bandwidth_bound_fp8_gb300 import moeq
    rows = 11
    big = _rand(1, rows + 1, off + K + gap, dt=dt)
    x = big[1:, off:off + K]
    codes, scales = _quant(x)
    _same_codes(x, codes, scales)
    back = torch.full_like(big, 7.0)
    moeq.moeq_fp8_dequant_rows(codes, scales, back[1:, off:off + K])
    want = torch.full_like(big, 7.0)
    want[1:, off:off + K] = torch.from_numpy(kp.values(codes.cpu().numpy(), scales.cpu().numpy())).to(dt)
    assert torch.equal(back, want)


def _pairs(seed, T, k, E, drop):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[g.random((T, k)) < drop] = -1
    offs, pair_row, row_pair = rp.sort_pairs(ids, E)
    return [torch.from_numpy(a).cuda() for a in (offs, pair_row, row_pair)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,H,k,drop", [(1, 8, 1, 0), (1, 128, 8, 0.3), (37, 1001, 3, 0.3), (64, 6144, 8, 0.0), (5, 264, 12, 1.0),
                                        (130, 40, 2, 0.5)])
def test_gather(T, H, k, drop, dt):
    from bandwidth_bound_fp8_gb300 import moeq
    E = 16
    offs, pair_row, row_pair = _pairs(T, T, k, E, drop)
    x = _rand(3, T, H, dt=dt)
    codes, scales = _quant(x)
    v = torch.empty_like(x)
    moeq.moeq_fp8_dequant_rows(codes, scales, v)
    want, xs = (torch.full((T * k, H), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    moeq.moeq_gather_rows(v, offs, pair_row, want)
    moeq.moeq_fp8_gather_rows(codes, scales, offs, pair_row, xs)
    assert torch.equal(xs, want)
    # indices and offsets out of range write nothing out of range
    big = torch.full((T * k + 2, H), 7.0, dtype=dt, device="cuda")
    wild = pair_row.clone()
    wild[0, 0] = T * k
    wild[-1, -1] = 2 ** 31 - 1
    moeq.moeq_fp8_gather_rows(codes, scales, torch.full_like(offs, -9), wild, big[1:-1])
    assert (big[0] == 7).all() and (big[-1] == 7).all()


def _within(got, ref, bound, what):
    got, bound = rp.to64(got), np.broadcast_to(bound, ref.shape)
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}"


def _steps(dt, gate, n=12, m=2):
    """Relative error of n steps, and of m |gate| more for bf16 rows."""
    return (n + m * np.abs(gate) * (dt == BF)) * U


def _swiglu_case(T, k, I, dt, drop, weighted, seed=5):
    offs, pair_row, row_pair = _pairs(seed, T, k, 16, drop)
    R = T * k
    gu, dh = _rand(seed, R, 2 * I, dt=dt, scale=2.0), _rand(seed + 1, R, I, dt=dt)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(seed + 2)).cuda() if weighted else None
    kept = int(offs[-1])
    gu[kept:], dh[kept:] = float("nan"), float("nan")     # nobody's rows
    rows = row_pair[:kept].long().cpu()
    wr = np.ones(kept) if w is None else rp.to64(w).reshape(-1)[rows.numpy()]
    return offs, pair_row, row_pair, gu, dh, w, wr, kept, rows.numpy()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,I,drop", [(1, 1, 1, 0), (1, 8, 64, 0), (3, 2, 128, 0.4), (9, 3, 129, 0.2), (40, 4, 200, 0.3),
                                        (6, 2, 1001, 0.5), (16, 8, 2048, 0.1), (2, 1, 5000, 0), (4, 3, 72, 1.0)])
def test_swiglu_and_its_gradient(T, k, I, drop, dt, weighted):
    from bandwidth_bound_fp8_gb300 import moeq
    offs, pair_row, row_pair, gu, dh, w, wr, kept, pairs = _swiglu_case(T, k, I, dt, drop, weighted)
    R = T * k
    half = rp.type_half_ulp(dt)
    h = torch.full((R, I), float("nan"), dtype=dt, device="cuda")
    codes, scales = _kept(R, I, 2)
    moeq.moeq_swiglu_rows(gu, h, row_pair=row_pair, topk_w=w, codes=codes, scales=scales)
    plain = torch.empty_like(h)
    moeq.moeq_swiglu_rows(gu, plain, row_pair=row_pair, topk_w=w)
    assert torch.equal(plain, h)
    z = rp.to64(gu[:kept])
    ref = kp.swiglu(z[:, :I], z[:, I:], wr)
    _within(h[:kept], ref, (_steps(dt, z[:, :I]) + half) * np.abs(ref) + rp.TINY, "h")
    assert (h[kept:] == 0).all() and (codes[kept:] == 0).all() and (scales[kept:] == 0).all()
    c, s = kp.keep_gate_up(kp.to_np(gu[:kept]))
    assert np.array_equal(codes[:kept].cpu().numpy(), c) and np.array_equal(scales[:kept].cpu().numpy(), s)

    gate, up = (v.astype(np.float64) for v in kp.values_gate_up(c, s))
    d = rp.to64(dh[:kept])
    dgate, dup, again, dw = kp.swiglu_grad(d, gate, up, wr)
    sig = 1 / (1 + np.exp(-gate))
    dgu, hh = torch.full((R, 2 * I), float("nan"), dtype=dt, device="cuda"), torch.full_like(h, float("nan"))
    d_w = torch.full((T, k), float("nan"), device="cuda") if weighted else None
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, dgu, h=hh, row_pair=row_pair, topk_w=w, pair_row=pair_row, d_topk_w=d_w)
    # 1 - sig and 1 + x (1 - sig) are sums: their errors are steps of their terms
    parts = np.abs(wr[:, None] * d * up) * sig * (1 + np.abs(gate) * (1 - sig) + np.abs(gate) * sig)
    _within(dgu[:kept, :I], dgate, _steps(dt, gate, 30, 6) * parts + half * np.abs(dgate) + rp.TINY, "d_gate")
    _within(dgu[:kept, I:], dup, (_steps(dt, gate) + half) * np.abs(dup) + rp.TINY, "d_up")
    _within(hh[:kept], again, (_steps(dt, gate) + half) * np.abs(again) + rp.TINY, "h again")
    assert (dgu[kept:] == 0).all() and (hh[kept:] == 0).all()
    if weighted:
        ref, size = np.zeros(R), np.zeros(R)
        ref[pairs], size[pairs] = dw, (np.abs(d * gate * sig * up) * ((I / 8 + 40) * U + _steps(dt, gate))).sum(1)
        _within(d_w.reshape(-1), ref, size + rp.TINY, "d_topk_w")
    only = torch.empty_like(dgu)
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, only, row_pair=row_pair, topk_w=w)
    assert torch.equal(only, dgu)


@pytest.mark.parametrize("dt", [BF, F32])
def test_swiglu_of_every_row(dt):
    """Without a sort: all rows are live, weights are 1; strided rows, what lies between them stays."""
    from bandwidth_bound_fp8_gb300 import moeq
    for I, off in ((136, 8), (101, 3)):
        R = 13
        big = _rand(1, R, 2 * I + 16, dt=dt)
        gu = big[:, off:off + 2 * I]
        hb = torch.full((R, I + 24), 7.0, dtype=dt, device="cuda")
        h = hb[:, off:off + I]
        codes, scales = _kept(R, I, 2)
        moeq.moeq_swiglu_rows(gu, h, codes=codes, scales=scales)
        z = rp.to64(gu)
        ref = kp.swiglu(z[:, :I], z[:, I:], np.ones(R))
        half = rp.type_half_ulp(dt)
        _within(h, ref, (_steps(dt, z[:, :I]) + half) * np.abs(ref) + rp.TINY, "h")
        hb[:, off:off + I] = 7.0
        assert (hb == 7).all()
        db = torch.full((R, 2 * I + 16), 7.0, dtype=dt, device="cuda")
        dh = _rand(2, R, I + 24, dt=dt)[:, off:off + I]
        moeq.moeq_swiglu_rows_grad(dh, codes, scales, db[:, off:off + 2 * I], h=h)
        gate, up = (v.astype(np.float64) for v in kp.values_gate_up(codes.cpu().numpy(), scales.cpu().numpy()))
        _, dup, again, _ = kp.swiglu_grad(rp.to64(dh), gate, up, np.ones(R))
        _within(db[:, off + I:off + 2 * I], dup, (_steps(dt, gate) + half) * np.abs(dup) + rp.TINY, "d_up")
        _within(h, again, (_steps(dt, gate) + half) * np.abs(again) + rp.TINY, "h again")
        db[:, off:off + 2 * I] = 7.0
        assert (db == 7).all()


def test_swiglu_far_out():
    """Gates where exp overflows or vanishes: finite, and as the formula says."""
    from bandwidth_bound_fp8_gb300 import moeq
    g = torch.tensor([-1e38, -1000.0, -104.0, -90.0, -88.5, -50.0, -20.0, -0.0, 0.0, 1e-30, 20.0, 90.0, 1000.0, 1e30]).cuda()
    I = len(g)
    gu = torch.stack([torch.cat((g, torch.full_like(g, u))) for u in (1.0, -3.0, 0.0)])
    h = torch.empty((3, I), device="cuda")
    moeq.moeq_swiglu_rows(gu, h)
    ref = kp.swiglu(rp.to64(gu[:, :I]), rp.to64(gu[:, I:]), np.ones(3))
    _within(h, ref, 13 * U * np.abs(ref) + 400 * rp.TINY, "h")   # (a sigmoid below 2^-126 may be rounded there)


def test_gradient_against_differences():
    """Gate and up on the 8-bit grid (so that they are kept exactly): the gradient is that of h, by central differences
    in 64 bits, whose own error is of the order of the step's square."""
    from bandwidth_bound_fp8_gb300 import moeq
    R, I = 6, 128
    rng = np.random.default_rng(3)
    gu = kp.E4M3[rng.integers(0, 127, (R, 2 * I))] * rng.choice([-1, 1], (R, 2 * I)) * 2.0 ** -7
    gu[:, 0], gu[:, I] = 3.5, -3.5           # 448 * 2^-7: the scale is 2^-7
    x = torch.from_numpy(gu).float().cuda()
    dh = _rand(4, R, I)
    h, dgu = torch.empty((R, I), device="cuda"), torch.empty_like(x)
    codes, scales = _kept(R, I, 2)
    moeq.moeq_swiglu_rows(x, h, codes=codes, scales=scales)
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, dgu)
    d, ones, eps = rp.to64(dh), np.ones(R), 1e-5
    up = lambda z: d * kp.swiglu(z[:, :I], z[:, I:], ones)
    for half in (0, 1):
        step = np.zeros_like(gu)
        step[:, half * I:(half + 1) * I] = eps
        num = (up(gu + step) - up(gu - step)) / (2 * eps)
        _within(dgu[:, half * I:(half + 1) * I], num, 1e-6 * (1 + np.abs(d)) * 4, "differences")


def test_one_bad_group():
    """A NaN in a gate: its row's group comes back as NaN in d_gu, its pair's weight gradient too, and nothing else."""
    from bandwidth_bound_fp8_gb300 import moeq
    T, k, I = 5, 2, 300
    offs, pair_row, row_pair, gu, dh, w, *_ = _swiglu_case(T, k, I, BF, 0.0, True)
    gu[3, 140] = float("nan")
    h = torch.empty((T * k, I), dtype=BF, device="cuda")
    codes, scales = _kept(T * k, I, 2)
    moeq.moeq_swiglu_rows(gu, h, row_pair=row_pair, topk_w=w, codes=codes, scales=scales)
    bad = torch.isnan(h)
    assert bad[3, 140] and bad.sum() == 1
    dgu, d_w = torch.empty_like(gu), torch.empty_like(w)
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, dgu, row_pair=row_pair, topk_w=w, pair_row=pair_row, d_topk_w=d_w)
    want = torch.zeros_like(dgu, dtype=torch.bool)
    want[3, 128:256], want[3, I + 128:I + 256] = True, True
    assert torch.equal(torch.isnan(dgu), want)
    assert torch.isnan(d_w).sum() == 1 and torch.isnan(d_w.reshape(-1)[int(row_pair[3])])


def test_wild_pairs_stay_inside():
    """row_pair out of range: such rows are not live."""
    from bandwidth_bound_fp8_gb300 import moeq
    R, I = 8, 64
    gu, dh, w = _rand(1, R, 2 * I), _rand(2, R, I), torch.ones((R, 1), device="cuda")
    rp_ = torch.tensor([0, -7, 2, 2 ** 31 - 1, 8, 5, 6, 7], dtype=torch.int32, device="cuda")
    h, dgu, d_w = torch.empty((R, I), device="cuda"), torch.empty_like(gu), torch.full((3, R), 7.0, device="cuda")
    codes, scales = _kept(R, I, 2)
    moeq.moeq_swiglu_rows(gu, h, row_pair=rp_, topk_w=w, codes=codes, scales=scales)
    assert (h[[1, 3, 4]] == 0).all() and (h[[0, 2, 5, 6, 7]].abs().sum(1) > 0).all()
    pr = torch.tensor([0, -1, 2, -1, -1, 5, 6, 7], dtype=torch.int32, device="cuda")
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, dgu, row_pair=rp_, topk_w=w, pair_row=pr, d_topk_w=d_w[1].view(R, 1))
    assert (dgu[[1, 3, 4]] == 0).all() and (d_w[1, [1, 3, 4]] == 0).all()
    assert (d_w[0] == 7).all() and (d_w[2] == 7).all()


def test_no_rows():
    from bandwidth_bound_fp8_gb300 import moeq
    e = lambda *s, dt=F32: torch.empty(s, dtype=dt, device="cuda")
    moeq.moeq_fp8_quant_rows(e(0, 64), e(0, 64, dt=torch.uint8), e(0, 1))
    moeq.moeq_fp8_dequant_rows(e(0, 64, dt=torch.uint8), e(0, 1), e(0, 64))
    moeq.moeq_swiglu_rows(e(0, 64), e(0, 32))
    moeq.moeq_swiglu_rows_grad(e(0, 32), e(0, 64, dt=torch.uint8), e(0, 2), e(0, 64))


def test_captured_and_replayed():
    from bandwidth_bound_fp8_gb300 import moeq
    T, k, I = 33, 4, 520
    offs, pair_row, row_pair, gu, dh, w, wr, kept, pairs = _swiglu_case(T, k, I, BF, 0.2, True)
    gu[kept:], dh[kept:] = 0, 0
    outs = lambda: dict(h=torch.empty_like(dh), dgu=torch.empty_like(gu), again=torch.empty_like(dh), dw=torch.empty_like(w))
    codes, scales = _kept(T * k, I, 2)

    def step(o):
        moeq.moeq_swiglu_rows(gu, o["h"], row_pair=row_pair, topk_w=w, codes=codes, scales=scales)
        moeq.moeq_swiglu_rows_grad(dh, codes, scales, o["dgu"], h=o["again"], row_pair=row_pair, topk_w=w, pair_row=pair_row,
                                   d_topk_w=o["dw"])
    a, b = outs(), outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(a)
    torch.cuda.synchronize()
    gu.copy_(_rand(91, *gu.shape, dt=BF))
    dh.copy_(_rand(92, *dh.shape, dt=BF))
    w.copy_(torch.rand(w.shape, generator=torch.Generator().manual_seed(93)))
    graph.replay()
    torch.cuda.synchronize()
    step(b)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_offsets_past_32_bits():
    from bandwidth_bound_fp8_gb300 import moeq
    R, I = 300_000, 8192          # gu: 4.9e9 elements
    gu = torch.zeros((R, 2 * I), dtype=BF, device="cuda")
    gu[-1] = _rand(1, 2 * I, dt=BF)
    h = torch.empty((R, I), dtype=BF, device="cuda")
    codes, scales = _kept(R, I, 2)
    moeq.moeq_swiglu_rows(gu, h, codes=codes, scales=scales)
    z = rp.to64(gu[-1:])
    ref = kp.swiglu(z[:, :I], z[:, I:], np.ones(1))
    _within(h[-1:], ref, (_steps(BF, z[:, :I]) + 2.0 ** -8) * np.abs(ref) + rp.TINY, "h")
    c, _ = kp.keep_gate_up(kp.to_np(gu[-1:]))
    assert np.array_equal(codes[-1:].cpu().numpy(), c)
    dh = torch.ones((R, I), dtype=BF, device="cuda")
    gu.fill_(7)
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, gu)
    gate, up = (v.astype(np.float64) for v in kp.values_gate_up(c, scales[-1:].cpu().numpy()))
    dup = kp.swiglu_grad(np.ones((1, I)), gate, up, np.ones(1))[1]
    _within(gu[-1:, I:], dup, (_steps(BF, gate) + 2.0 ** -8) * np.abs(dup) + rp.TINY, "d_up")
    out = torch.empty((R, 2 * I), dtype=BF, device="cuda")
    moeq.moeq_fp8_dequant_rows(codes, scales, out)
    assert torch.equal(out[-1].cpu(), torch.from_numpy(kp.values(c, scales[-1:].cpu().numpy())[0]).to(BF))


def test_refusals():
    """On the device: shapes and types that do not fit each other, and nothing is written."""
    from bandwidth_bound_fp8_gb300 import moeq
    z = lambda *s, dt=F32: torch.zeros(s, dtype=dt, device="cuda")
    u8, i32 = torch.uint8, torch.int32
    offs, pr, rp_ = z(4, dt=i32), z(4, 2, dt=i32), z(8, dt=i32)
    with pytest.raises(ValueError, match="xs"):
        moeq.moeq_fp8_gather_rows(z(4, 64, dt=u8), z(4, 1), offs, pr, z(7, 64))
    with pytest.raises(ValueError, match="codes"):
        moeq.moeq_fp8_gather_rows(z(5, 64, dt=u8), z(4, 1), offs, pr, z(8, 64))
    with pytest.raises(ValueError, match="scales"):
        moeq.moeq_fp8_quant_rows(z(4, 129), z(4, 129, dt=u8), z(4, 1))
    with pytest.raises(TypeError):
        moeq.moeq_fp8_quant_rows(z(4, 64, dt=torch.float16), z(4, 64, dt=u8), z(4, 1))
    with pytest.raises(ValueError, match="row_pair"):
        moeq.moeq_swiglu_rows(z(8, 64), z(8, 32), row_pair=rp_[:7], topk_w=z(4, 2))
    with pytest.raises(ValueError, match="topk_w"):
        moeq.moeq_swiglu_rows(z(8, 64), z(8, 32), row_pair=rp_, topk_w=z(4, 3))
    with pytest.raises(ValueError, match="d_topk_w"):
        moeq.moeq_swiglu_rows_grad(z(8, 32), z(8, 64, dt=u8), z(8, 2), z(8, 64), row_pair=rp_, topk_w=z(4, 2), pair_row=pr,
                                   d_topk_w=z(2, 4))
    with pytest.raises(moeq.MoeqError):
        moeq.moeq_expert_product(z(8, 60, dt=BF), z(3, 64, 60, dt=BF), offs, z(8, 64))
    with pytest.raises(ValueError, match="x:"):
        moeq.moeq_expert_product_grad_w(z(8, 64, dt=BF), z(7, 64, dt=BF), offs, z(3, 64, 64))


@pytest.mark.parametrize("dt", [BF, F32])
def test_widest(dt):
    """Rows of the largest width, and one row less than a block has."""
    from bandwidth_bound_fp8_gb300 import moeq
    K = 1 << 20
    x = _rand(11, 2, K, dt=dt)
    codes, scales = _quant(x)
    _same_codes(x, codes, scales)
    back, xs = torch.empty_like(x), torch.full((4, K), float("nan"), dtype=dt, device="cuda")
    moeq.moeq_fp8_dequant_rows(codes, scales, back)
    assert torch.equal(back.cpu(), torch.from_numpy(kp.values(codes.cpu().numpy(), scales.cpu().numpy())).to(dt))
    offs, pair_row, _ = _pairs(3, 2, 2, 16, 0)
    moeq.moeq_fp8_gather_rows(codes, scales, offs, pair_row, xs)
    assert all(torch.equal(xs[pair_row[t, j]], back[t]) for t in range(2) for j in range(2))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,k,I,drop", [(1, 1, 1 << 20, 0), (2, 2, (1 << 20) - 1, 0.3), (700, 3, 1, 0.3), (4000, 2, 24, 0.3)])
def test_widest_and_narrow_swiglu(T, k, I, drop, dt):
    test_swiglu_and_its_gradient(T, k, I, drop, dt, True)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,k,I", [(16, 3, 1408), (40, 8, 384), (130, 2, 1409), (70, 3, 2816), (20, 2, 2176), (5000, 3, 72),
                                   (5000, 3, 267)])
def test_groups_that_do_not_fill_a_block(T, k, I, dt):
    test_swiglu_and_its_gradient(T, k, I, 0.2, dt, True)
    test_codes_and_values(T, I, dt)


def test_codes_of_tiny_groups():
    """fp32 groups whose scale lies between 2^-102 and 2^-86, where the remainder of a quotient may lie below the smallest
    fp32: two that did get another code, and quotients at the borders of the lowest codes and up to six steps beside."""
    g = np.random.default_rng(11)
    x = np.zeros((2048, 128), np.float32)
    x[0, :3] = 7.068192747815294e-28, 1.5407438636742925e-33, 4.622231131845397e-33
    mids = ((kp.E4M3[:-1] + kp.E4M3[1:]) / 2)[:9]
    for i in range(1, len(x)):
        x[i, 0] = 448 * 2.0 ** g.uniform(-102, -86)
        s = float(x[i, 0] / np.float32(448))
        b = (mids[g.integers(0, 9, 127)] * s).astype(np.float32)
        x[i, 1:] = (b.view(np.int32) + g.integers(-6, 7, 127).astype(np.int32)).view(np.float32)
    x *= np.where(g.random(x.shape) < 0.5, np.float32(-1), np.float32(1))
    x[0] = np.abs(x[0])
    t = torch.from_numpy(x).cuda()
    codes, scales = _quant(t)
    _same_codes(t, codes, scales)
    assert codes[0, :3].tolist() == [126, 1, 1]
    # the same as gate and up rows
    from bandwidth_bound_fp8_gb300 import moeq
    gu = torch.cat((t, t.flip(0)), 1)
    codes2, scales2 = _kept(len(x), 128, 2)
    moeq.moeq_swiglu_rows(gu, torch.empty_like(t), codes=codes2, scales=scales2)
    assert torch.equal(codes2, torch.cat((codes, codes.flip(0)), 1)) and torch.equal(scales2, torch.cat((scales, scales.flip(0)), 1))


@pytest.mark.parametrize("dt", [BF, F32])
def test_swiglu_where_the_sigmoid_is_subnormal(dt):
    """Gates down to -104: a sigmoid below 2^-126 counts where the other factors are large.  It is a multiple of 2^-149, two
    of them off at most, and so is its product with the gate: (2 |gate| + 1) 2^-149 of the other factors beside the steps."""
    from bandwidth_bound_fp8_gb300 import moeq
    R, I = 5, 256
    gate = torch.linspace(-104, -70, I).to(dt)
    ups = torch.tensor([1e38, -1e37, 1e30, 1.0, 0.0])
    gu = torch.cat((gate.expand(R, I), ups[:, None].expand(R, I).to(dt)), 1).contiguous().cuda()
    half, least = rp.type_half_ulp(dt), 2.0 ** -149
    h = torch.empty((R, I), dtype=dt, device="cuda")
    codes, scales = _kept(R, I, 2)
    moeq.moeq_swiglu_rows(gu, h, codes=codes, scales=scales)
    z = rp.to64(gu)
    x, u = z[:, :I], z[:, I:]
    ref = kp.swiglu(x, u, np.ones(R))
    tiny = lambda g, f: (2 * np.abs(g) + 1) * least * np.abs(f) + rp.TINY
    # (the forward pass of bf16 rows has its exponent 24 lower: 24 log 2 steps of rounding more)
    _within(h, ref, (_steps(dt, x, 12 + 17 * (dt == BF)) + half) * np.abs(ref) + tiny(x, u), "h")

    x, u = (v.astype(np.float64) for v in kp.values_gate_up(codes.cpu().numpy(), scales.cpu().numpy()))
    pairs = torch.arange(R, dtype=torch.int32, device="cuda")
    w, dh = torch.full((R, 1), 0.5, device="cuda"), torch.full((R, I), 1.5, dtype=dt, device="cuda")
    dgu, again, dw = torch.empty_like(gu), torch.empty_like(h), torch.empty_like(w)
    moeq.moeq_swiglu_rows_grad(dh, codes, scales, dgu, h=again, row_pair=pairs, topk_w=w, pair_row=pairs.view(R, 1), d_topk_w=dw)
    d, wr = rp.to64(dh), np.full(R, 0.5)
    dgate, dup, hh, dot = kp.swiglu_grad(d, x, u, wr)
    sig = 1 / (1 + np.exp(-x))
    parts = np.abs(0.5 * d * u) * sig * (1 + np.abs(x))
    _within(dgu[:, :I], dgate, _steps(dt, x, 30, 6) * parts + half * np.abs(dgate) + tiny(x, 0.5 * d * u), "d_gate")
    _within(dgu[:, I:], dup, (_steps(dt, x) + half) * np.abs(dup) + tiny(x, 0.5 * d), "d_up")
    _within(again, hh, (_steps(dt, x) + half) * np.abs(hh) + tiny(x, 0.5 * u), "h again")
    terms = np.abs(d * x * sig * u) * ((I / 8 + 40) * U + _steps(dt, x)) + tiny(x, d * u)
    _within(dw.reshape(-1), dot, terms.sum(1), "d_topk_w")
