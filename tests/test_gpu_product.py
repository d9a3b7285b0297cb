"""The experts' bf16 products in their three directions against 64 bits.

Tolerances: a sum over C indices is C/16 accumulations of the tensor core, each
off by at most a step (2^-23, it may truncate) of what the terms add up to, and
the products of an accumulation are summed with a few steps more: (C/16 + 8)
2^-22 of the sum of |terms|; then half a step of the output's type."""
import pytest
import torch

import rows_plain as rp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(BF).cuda()


def _offs(counts):
    return torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device="cuda")


def _call(way, a, b, offs, out, **kw):
    from bandwidth_bound_fp8_gb300 import moeq
    getattr(moeq, {"y": "moeq_expert_product", "dx": "moeq_expert_product_grad_x", "dw": "moeq_expert_product_grad_w"}[way])(
        a, b, offs, out, **kw)


def _ref(way, a, b, counts, out_shape):
    """The result and the sum of |terms|, in 64 bits."""
    ref, terms = (torch.zeros(out_shape, dtype=torch.float64, device="cuda") for _ in range(2))
    r = 0
    for e, n in enumerate(counts):
        at = slice(r, r + n)
        for out, f in ((ref, lambda t: t), (terms, torch.abs)):
            if way == "dw":
                out[e] = f(a[at].double()).t() @ f(b[at].double())
            else:
                w = f(b[e].double())
                out[at] = f(a[at].double()) @ (w.t() if way == "y" else w)
        r += n
    return ref, terms


def _check(got, ref, terms, C, what=""):
    bound = (C / 16 + 8) * 2.0 ** -22 * terms + rp.type_half_ulp(got.dtype) * ref.abs() + rp.TINY
    err = (got.double() - ref).abs()
    assert (err <= bound).all(), f"{what}: {int((~(err <= bound)).sum())} outside, worst {float((err - bound).max())}"


def _run(way, counts, K, N, dt, extra=0, seed=1):
    """One call on random rows, `extra` rows behind the last expert's (NaN: they are nobody's)."""
    E, kept = len(counts), sum(counts)
    R = kept + extra
    x, dy, w = _rand(seed, R, K), _rand(seed + 1, R, N), _rand(seed + 2, E, N, K, scale=0.1)
    x[kept:], dy[kept:] = float("nan"), float("nan")
    shape = {"y": (R, N), "dx": (R, K), "dw": (E, N, K)}[way]
    a, b = {"y": (x, w), "dx": (dy, w), "dw": (dy, x)}[way]
    out = torch.full(shape, float("nan"), dtype=dt, device="cuda")
    _call(way, a, b, _offs(counts), out)
    ref, terms = _ref(way, a, b, counts, shape)
    _check(out, ref, terms, {"y": K, "dx": N, "dw": max(counts)}[way], way)
    return out


WAYS = ["y", "dx", "dw"]


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("counts", [[1], [0, 1, 0, 2, 0], [3, 0, 7, 1, 0, 0, 16, 17], [15, 16, 17, 31, 32, 33]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_few_rows(way, counts, dt):
    """Tiles of one CTA, contractions of less than a stage, experts without rows."""
    _run(way, counts, 200, 136, dt, extra=3)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("counts", [[128], [63, 64, 65, 129], [257, 0, 511, 1], [130, 700, 0, 384, 40]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_many_rows(way, counts, dt):
    """Tiles of pairs of CTAs, shared out over an expert's rows."""
    _run(way, counts, 328, 520, dt, extra=5)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("K,N", [(8, 8), (8, 264), (64, 128), (72, 1000), (1000, 24), (1064, 256), (2048, 2816)])
def test_sizes(way, K, N):
    """Widths around the stages', the tiles' and the swizzle's, of one CTA and of pairs."""
    _run(way, [5, 0, 20], K, N, BF, extra=1)
    _run(way, [200, 90], K, N, BF)


@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 15, 16, 17, 47, 48, 49, 63, 64, 65, 100, 127, 128, 129, 191, 255])
def test_weight_gradient_of_every_last_stage(n):
    """The last stage's rows are copied in boxes of every size, and what follows them is another expert's."""
    _run("dw", [n, n + 1, 0, 2], 128, 64, F32, extra=2, seed=n)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("rows", [1, 40, 300, 5000])
def test_dense(way, rows):
    _run(way, [rows], 512, 384, BF)


@pytest.mark.parametrize("way", ["y", "dx"])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("counts,C,features", [([1], 4096, 200), ([16], 1024, 136), ([40], 4104, 136), ([100], 2048, 264),
                                               ([128], 4096, 72), ([200], 1032, 520), ([0, 3, 0], 4096, 128), ([1, 0, 2, 5], 2056, 264),
                                               ([0, 0], 4096, 64), ([9], 2568, 2000), ([16], 8192, 136),
                                               ([64], 8200, 72), ([128], 4096, 4000), ([130, 100], 2560, 2304)])
def test_few_units_of_long_contraction(way, counts, C, features, dt):
    """Units split over clusters of two, four and eight CTAs; the same result every time."""
    K, N = (C, features) if way == "y" else (features, C)
    out = _run(way, counts, K, N, dt, extra=2)
    assert torch.equal(out, _run(way, counts, K, N, dt, extra=2))


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("K,N", [(576, 320), (192, 1088)])
@pytest.mark.parametrize("counts", [[257, 256, 300, 0, 511, 512, 513, 1025], [64, 128, 640, 1]])
def test_whole_columns(way, K, N, counts):
    """Widths that are multiples of 64 and not of 128: one copy a stage."""
    _run(way, counts, K, N, BF, extra=7)


@pytest.mark.parametrize("N,K", [(1032, 2064), (264, 9000), (1288, 1800), (1024, 2304)])
@pytest.mark.parametrize("counts", [[257, 256, 300, 0, 511, 512, 513, 1025], [1, 16, 17, 0, 63, 64, 65, 129]])
def test_weight_gradient_in_wide_units(N, K, counts):
    """Two blocks of dW share their dy; odd numbers of blocks, an expert without rows, ragged last stages."""
    _run("dw", counts, K, N, BF, extra=7)


@pytest.mark.parametrize("way", ["y", "dx"])
def test_many_tiles_of_one_expert(way):
    """More row tiles than a band of them, the last band narrower."""
    _run(way, [2304 + 100, 0, 2048], 128, 520, BF)


def test_many_experts():
    counts = [(7 * e) % 5 for e in range(1024)]
    for way in WAYS:
        _run(way, counts, 64, 72, BF, extra=9)


@pytest.mark.parametrize("way", ["y", "dx"])
@pytest.mark.parametrize("counts", [[0, 0], [0]])
def test_no_expert_has_rows(way, counts):
    out = _run(way, counts, 64, 64, BF, extra=6)
    assert (out == 0).all()


def test_weight_gradient_without_rows_is_zero():
    assert (_run("dw", [0, 0, 0], 72, 40, F32, extra=4) == 0).all()
    assert (_run("dw", [0, 0], 72, 40, BF) == 0).all()   # R = 0


@pytest.mark.parametrize("way", ["y", "dx"])
def test_no_rows_at_all(way):
    from bandwidth_bound_fp8_gb300 import moeq
    out = torch.empty((0, 64), dtype=BF, device="cuda")
    _call(way, torch.empty((0, 64), dtype=BF, device="cuda"), _rand(1, 2, 64, 64), _offs([0, 0]), out)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("counts", [[3, 9, 0, 4], [140, 70, 0, 300]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_stays_where_it_is(way, counts, bad):
    """One row of expert 1 is NaN or infinite: its row of y and d_x, its expert's d_w, and nothing else."""
    E, R, K, N = len(counts), sum(counts), 136, 264
    x, dy, w = _rand(1, R, K), _rand(2, R, N), _rand(3, E, N, K)
    row = counts[0] + counts[1] - 1
    x[row], dy[row] = bad, bad
    shape = {"y": (R, N), "dx": (R, K), "dw": (E, N, K)}[way]
    out = torch.zeros(shape, device="cuda")
    _call(way, *{"y": (x, w), "dx": (dy, w), "dw": (dy, x)}[way], _offs(counts), out)
    ok = torch.isfinite(out).flatten(1).all(1)
    want = torch.ones_like(ok)
    want[1 if way == "dw" else row] = False
    assert torch.equal(ok, want)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("counts", [[3, 9, 0, 4], [140, 70, 0, 300]])
def test_strides(way, counts):
    """Rows apart, from an offset of 16 bytes; what lies between the output's rows stays."""
    E, R, K, N = len(counts), sum(counts), 72, 200
    def wide(seed, rows, cols, dt=BF):
        return _rand(seed, rows + 1, cols + 48).to(dt)
    xb, yb, w = wide(1, R, K), wide(2, R, N), _rand(3, E, N, K)
    x, dy = xb[1:, 8:8 + K], yb[1:, 16:16 + N]
    a, b = {"y": (x, w), "dx": (dy, w), "dw": (dy, x)}[way]
    C = {"y": K, "dx": N, "dw": max(counts)}[way]
    if way == "dw":
        out = torch.empty((E, N, K), dtype=BF, device="cuda")
        _call(way, a, b, _offs(counts), out)
        _check(out, *_ref(way, a, b, counts, out.shape), C)
        return
    F = N if way == "y" else K
    for dt, off, gap in ((BF, 8, 40), (BF, 3, 5), (F32, 4, 20), (F32, 1, 2)):
        big = torch.full((R + 2, F + off + gap), 7.0, dtype=dt, device="cuda")
        out = big[1:-1, off:off + F]
        _call(way, a, b, _offs(counts), out)
        _check(out, *_ref(way, a, b, counts, (R, F)), C)
        big[1:-1, off:off + F] = 7.0
        assert (big == 7.0).all()


@pytest.mark.parametrize("way", WAYS)
def test_offsets_out_of_range_stay_inside(way):
    """offs that fall, or pass the rows: nothing outside is written, and what they say in range is done."""
    R, K, N, E = 20, 64, 64, 4
    x, dy, w = _rand(1, R, K), _rand(2, R, N), _rand(3, E, N, K)
    offs = torch.tensor([-5, 8, 3, 10 ** 9, 15], dtype=torch.int32, device="cuda")
    counts = [8, 0, 12, 0]
    a, b = {"y": (x, w), "dx": (dy, w), "dw": (dy, x)}[way]
    shape = {"y": (R, N), "dx": (R, K), "dw": (E, N, K)}[way]
    big = torch.full((2, *shape), 7.0, device="cuda")
    _call(way, a, b, offs, big[0])
    _check(big[0], *_ref(way, a, b, counts, shape), 64)
    assert (big[1] == 7.0).all()


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("counts,K,N", [([2, 0, 5], 136, 72), ([300, 0, 150], 136, 72), ([2, 0, 5], 4096, 2048)])
def test_captured_and_replayed(way, counts, K, N):
    """A graph follows new inputs and new offsets, on another stream, and the status word stays as it was."""
    E, R = len(counts), sum(counts)
    x, dy, w, offs = _rand(1, R, K), _rand(2, R, N), _rand(3, E, N, K), _offs(counts)
    a, b = {"y": (x, w), "dx": (dy, w), "dw": (dy, x)}[way]
    shape = {"y": (R, N), "dx": (R, K), "dw": (E, N, K)}[way]
    out, status = torch.empty(shape, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _call(way, a, b, offs, out, status=status)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            _call(way, a, b, offs, out, status=status)
    torch.cuda.synchronize()
    new = counts[::-1]
    x.copy_(_rand(7, R, K))
    dy.copy_(_rand(8, R, N))
    offs.copy_(_offs(new))
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    _check(out, *_ref(way, a, b, new, shape), {"y": K, "dx": N, "dw": max(new)}[way])
    first = out.clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out) and int(status) == 0


def test_two_streams_at_once():
    """Products share nothing: calls that run together give what each gives alone."""
    counts, K, N = [100, 37, 260], 256, 512
    w, offs = _rand(3, 3, N, K), _offs(counts)
    xs = [_rand(10 + i, sum(counts), K) for i in range(4)]
    want, got = ([torch.empty((sum(counts), N), device="cuda") for _ in xs] for _ in range(2))
    for x, y in zip(xs, want):
        _call("y", x, w, offs, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for x, y, st in zip(xs, got, streams):
            _call("y", x, w, offs, y, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))


def test_offsets_past_32_bits():
    """Outputs and weights of more than 2^32 bytes, checked at their ends."""
    E, K, N = 9, 16384, 16384
    w = torch.zeros((E, N, K), dtype=BF, device="cuda")
    w[-1, -1, -1], w[-1, 0, 0] = 2.0, 3.0
    counts = [0] * (E - 1) + [2]
    x = torch.ones((2, K), dtype=BF, device="cuda")
    y = torch.empty((2, N), dtype=F32, device="cuda")
    _call("y", x, w, _offs(counts), y)
    assert float(y[1, -1]) == 2.0 and float(y[0, 0]) == 3.0 and float(y.sum()) == 10.0
    dx = torch.empty((2, K), dtype=F32, device="cuda")
    _call("dx", torch.ones((2, N), dtype=BF, device="cuda"), w, _offs(counts), dx)
    assert float(dx[1, -1]) == 2.0 and float(dx[0, 0]) == 3.0 and float(dx.sum()) == 10.0
    w.fill_(float("nan"))
    _call("dw", torch.ones((2, N), dtype=BF, device="cuda"), x, _offs(counts), w)
    assert (w[:-1] == 0).all() and (w[-1] == 2).all()
    del w
    R, F = (1 << 16) + 40, 1 << 15
    x, wn = _rand(1, R, 8), _rand(2, 2, F, 8)
    y = torch.empty((R, F), dtype=BF, device="cuda")
    _call("y", x, wn, _offs([5, R - 45]), y)
    _check(y[R - 300:R - 40], x[R - 300:R - 40].double() @ wn[1].double().t(),
           x[R - 300:R - 40].double().abs() @ wn[1].double().abs().t(), 8)
    assert (y[R - 40:] == 0).all()


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("K,N", [(1 << 20, 8), (8, 1 << 20)])
@pytest.mark.parametrize("counts", [[1], [3, 0, 18]])
def test_widest(way, K, N, counts):
    """The largest width: as the contraction, split or not, and as the features."""
    for dt in (BF, F32):
        _run(way, counts, K, N, dt, extra=2)


@pytest.mark.parametrize("way", WAYS)
def test_many_experts_of_many_rows(way):
    """The most experts beside the largest tiles: the plan leaves the fewest stages."""
    _run(way, [(37 * e) % 401 for e in range(1024)], 72, 136, F32, extra=5)
    _run(way, [(37 * e) % 401 for e in range(1024)], 128, 192, BF)


@pytest.mark.parametrize("way", WAYS)
def test_widest_of_many_rows(way):
    for K, N in ((1 << 18, 64), (64, 1 << 18)):
        _run(way, [300, 0, 212], K, N, F32)


def test_weight_gradient_of_one_long_expert():
    """2^29 rows of ones: a sum that one accumulator does not hold, of more stages than one wait lasts."""
    R = (1 << 29) + 64
    ones = torch.ones((R, 8), dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (F32, BF):
        out = torch.empty((2, 8, 8), dtype=dt, device="cuda")
        _call("dw", ones, ones, torch.tensor([0, R - 64, R], dtype=torch.int32, device="cuda"), out, status=status)
        assert int(status) == 0 and (out[0] == R - 64).all() and (out[1] == 64).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("E,N,K", [(8, 768, 768), (8, 776, 776), (2, 264, 1032), (2, 256, 1024), (1, 1000, 1064),
                                   (40, 512, 128), (40, 512, 136)])
def test_weight_gradient_in_units_of_both_widths(E, N, K, dt):
    """Few units (halves), many (whole ones), and many of one half's columns, with every kind of last stage."""
    counts = [(0, 1, 15, 16, 17, 63, 64, 65, 127, 600, 31, 47)[(5 * e + E) % 12] for e in range(E)]
    _run("dw", counts, K, N, dt, extra=3)


def test_every_way_at_once():
    """The three products and SwiGLU on a stream each, of few and of many rows: the same results as one after the other."""
    from bandwidth_bound_fp8_gb300 import moeq
    calls = []
    for i, counts in enumerate(([3, 0, 9], [300, 77, 0, 513], [2] * 40)):
        E, R, K, N = len(counts), sum(counts), 1024, 520
        x, dy, w, offs = _rand(i, R, K), _rand(i + 9, R, N), _rand(i + 18, E, N, K, scale=0.1), _offs(counts)
        for way, a, b, shape in (("y", x, w, (R, N)), ("dx", dy, w, (R, K)), ("dw", dy, x, (E, N, K))):
            calls.append((lambda out, st, way=way, a=a, b=b, offs=offs: _call(way, a, b, offs, out, stream=st), shape))
        calls.append((lambda out, st, x=x: moeq.moeq_swiglu_rows(x, out, stream=st), (R, K // 2)))
    want, got = ([torch.empty(shape, dtype=BF, device="cuda") for _, shape in calls] for _ in range(2))
    for (f, _), out in zip(calls, want):
        f(out, None)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for (f, _), out, st in zip(calls, got, streams):
            f(out, st)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("C,rows,features", [(8192, 40, 640), (65536, 16, 640), (65536, 200, 264), (1 << 20, 16, 64)])
def test_long_bf16_sums_are_rounded_once(way, C, rows, features):
    """Sums of C positive terms: within half a step of bf16 at the exact sum, and what fp32 sums in parts of 1024 indices
    are off by: 64 accumulations and 8 as above, and half a step for each part that is added."""
    g = torch.Generator(device="cuda").manual_seed(C + rows)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda").to(BF)
    if way == "dw":
        a, b = rand(C, features), rand(C, rows // 8 * 8)
        counts, shape = [C], (1, features, rows // 8 * 8)
    else:
        a, b = rand(rows, C), rand(1, *((features, C) if way == "y" else (C, features)))
        counts, shape = [rows], (rows, features)
    out = torch.empty(shape, dtype=BF, device="cuda")
    _call(way, a, b, _offs(counts), out)
    ref, _ = _ref(way, a, b, counts, shape)
    half = torch.exp2(torch.floor(torch.log2(ref)) - 8)
    off = (out.double() - ref).abs() - half
    bound = (72 * 2.0 ** -22 + C / 1024 * 2.0 ** -24) * ref
    assert (off <= bound).all(), f"{int((off > bound).sum())} of {off.numel()} outside, worst {float((off / ref).max())}"


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("C,rows,features", [(2048, 40, 640), (2048, 300, 640), (8192, 40, 264)])
def test_fp32_sums_are_taken_in_parts(way, C, rows, features):
    """Sums of C positive terms, in parts of 512 indices.  A part is 32 accumulations, each of which truncates up to a step
    (2^-23) of what is there by then, and that grows evenly: 33/2 2^-23 of the terms, and 8 2^-22 for the products as
    above; adding the parts up half a step for each.  Truncation loses half as much on average, 33/4 2^-23 at most
    (9.8e-7); an accumulator of 2048 indices would lose 129/4 2^-24 at least (1.9e-6)."""
    g = torch.Generator(device="cuda").manual_seed(C + rows)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda").to(BF)
    if way == "dw":
        a, b = rand(C, features), rand(C, rows // 8 * 8)
        counts, shape = [C], (1, features, rows // 8 * 8)
    else:
        a, b = rand(rows, C), rand(1, *((features, C) if way == "y" else (C, features)))
        counts, shape = [rows], (rows, features)
    out = torch.empty(shape, dtype=F32, device="cuda")
    _call(way, a, b, _offs(counts), out)
    ref, _ = _ref(way, a, b, counts, shape)
    off = (out.double() - ref) / ref
    assert float(off.abs().max()) <= 33 / 2 * 2.0 ** -23 + 8 * 2.0 ** -22 + C / 512 * rp.U24
    assert abs(float(off.mean())) <= 1.4e-6
