"""The expert layer at any number of tokens: Mx4MoeLayer against the same
layer in 64 bits, and the training functions against
torch's autograd in 64 bits."""
import pytest
import torch

import rows_plain as rp

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda()


def _q(x):
    """MXFP4 values of [R, K], in 64 bits."""
    return torch.from_numpy(rp.mx4_values(*rp.mx4_codes(rp.to64(x)))).cuda()


def _product64(xq, wq, offs, rows):
    """y and sum of |terms| of sorted rows, in 64 bits."""
    y, T = (torch.zeros((len(rows), wq[0].shape[0]), dtype=torch.float64, device="cuda") for _ in range(2))
    for e, w in enumerate(wq):
        i = rows[offs[e]:offs[e + 1]]
        y[offs[e]:offs[e + 1]] = xq[i] @ w.t()
        T[offs[e]:offs[e + 1]] = xq[i].abs() @ w.abs().t()
    return y, T


def _within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert (err <= bound).all(), f"{what}: {int((err > bound).sum())} outside, worst {float((err - bound).max())}"


@pytest.mark.parametrize("T", [1, 3, 16, 17, 250])
@pytest.mark.parametrize("shared", [True, False])
def test_layer_step_by_step(T, shared):
    """Each step of the layer against 64 bits, from the buffers the step before left (4-bit codes of h are those of
    the quantiser, which has its own test): products within (K/64 + 8) 2^-22 of their terms and half a bf16 ulp, the
    combine within k + 2 fp32 roundings and half a bf16 ulp."""
    from bandwidth_bound_fp8_gb300 import moeq
    from bandwidth_bound_fp8_gb300.expert_layer import Mx4MoeLayer
    E, H, I, k = 12, 512, 256, 3
    w_gu, w_d = 0.05 * _rand(1, E, 2 * I, H), 0.05 * _rand(2, E, H, I)
    s_gu, s_d = 0.05 * _rand(3, 1, 2 * I, H), 0.05 * _rand(4, 1, H, I)
    layer = Mx4MoeLayer(w_gu, w_d, k, s_gu if shared else None, s_d if shared else None)
    x, logits = _rand(5, T, H).to(BF), _rand(6, T, E)
    logits[0, 5:] = float("-inf")
    logits[T - 1] = float("-inf")          # no expert: the shared one alone, or zero
    out = layer(x, logits)
    again = layer(x, logits)
    assert torch.equal(out, again)
    assert moeq.moeq_read_device_status(layer.ws.t, layer.ws.nbytes) == 0

    ids, w = rp.route(rp.to64(logits), k)
    assert torch.equal(layer.ids.cpu(), torch.from_numpy(ids))
    offs, pair_row, row_pair = rp.sort_pairs(ids, E)
    kept = int(offs[-1])
    xq = _q(x)

    def ffn(wg, wd, off, rows, h, y):
        ref, terms = _product64(xq, [_q(v) for v in wg], off, rows)
        n = len(rows)
        _within(h[:n], ref, (H / 64 + 8) * 2.0 ** -22 * terms + 2.0 ** -8 * ref.abs() + rp.TINY, "gate and up")
        q = torch.empty((h.shape[0], I // 2), dtype=torch.uint8, device="cuda")
        s = torch.empty((h.shape[0], moeq.moeq_mx4_scale_pitch(I)), dtype=torch.uint8, device="cuda")
        hq = torch.empty((h.shape[0], I), device="cuda")
        moeq.moeq_mx4_quant_act(h, q, s, act=moeq.MOEQ_ACT_SWIGLU)
        moeq.moeq_mx4_dequant_act(q, s, hq)
        ref, terms = _product64(hq.double(), [_q(v) for v in wd], off, torch.arange(n, device="cuda"))
        _within(y[:n], ref, (I / 64 + 8) * 2.0 ** -22 * terms + 2.0 ** -8 * ref.abs() + rp.TINY, "down")

    ffn(w_gu, w_d, offs, torch.from_numpy(row_pair[:kept] // k).long().cuda(), layer.h, layer.y)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    if shared:
        ffn(s_gu, s_d, [0, T], torch.arange(T, device="cuda"), layer.sh, layer.sy)
        ref = layer.sy.double()
    mag = ref.abs()
    for j in range(k):
        t = torch.from_numpy((pair_row[:, j] >= 0).nonzero()[0]).cuda()
        term = layer.w[t, j, None].double() * layer.y[torch.from_numpy(pair_row[:, j]).cuda()[t].long()].double()
        ref[t] += term
        mag[t] += term.abs()
    _within(out, ref, (k + 2) * rp.U24 * mag + 2.0 ** -8 * ref.abs() + rp.TINY, "combine")
    if not shared:
        assert (out[T - 1] == 0).all()


def test_training_step_matches_autograd_in_64_bits():
    """fp32 chains of at most 64 products and a few sums: below 200 * 2^-24 of the terms; 1e-4 of the largest gradient
    is asked for."""
    from bandwidth_bound_fp8_gb300 import expert_layer as el
    T, H, E, k = 53, 64, 6, 2
    x0, lg0, W0, b0, do = _rand(1, T, H), _rand(2, T, E), 0.2 * _rand(3, E, H, H), _rand(4, T, H), _rand(5, T, H)
    lg0[3, 2:] = float("-inf")
    lg0[4] = float("-inf")

    leaf = lambda t, dt: t.detach().to(dt).requires_grad_()
    x, lg, W, b = (leaf(t, torch.float32) for t in (x0, lg0, W0, b0))
    ids, w = el.route(lg, k)
    d = el.Dispatch(ids, E)
    xs = el.dispatch(x, d)
    offs = d.offs.tolist()
    y = torch.cat([torch.tanh(xs[offs[e]:offs[e + 1]] @ W[e]) for e in range(E)] + [xs[offs[E]:] * 0])
    out = el.combine(y, w, d, base=b)
    (out * do).sum().backward()

    X, L, V, B = (leaf(t, torch.float64) for t in (x0, lg0, W0, b0))
    ref = B + 0
    rows = []
    for t in range(T):
        n = int(torch.isfinite(lg0[t]).sum().clamp(max=k))
        acc = ref[t]
        if n:
            idx = ids[t, :n].long()
            ww = torch.softmax(L[t][idx], 0)
            for j in range(n):
                acc = acc + ww[j] * torch.tanh(X[t] @ V[int(idx[j])])
        rows.append(acc)
    R = torch.stack(rows)
    (R * do.double()).sum().backward()
    assert (out.double() - R).abs().max() <= 1e-4 * R.abs().max()
    for got, want in ((x.grad, X.grad), (lg.grad, L.grad), (W.grad, V.grad), (b.grad, B.grad)):
        want = torch.nan_to_num(want)
        assert (got.double() - want).abs().max() <= 1e-4 * want.abs().max()


def test_gradient_penalty_matches_autograd_in_64_bits():
    """Second derivatives: at most four chained products of 64 terms and about a hundred other roundings, 360 * 2^-24 =
    2.1e-5 of the terms; 5e-4 of the largest gradient leaves terms 20 times their sum."""
    from bandwidth_bound_fp8_gb300 import expert_layer as el
    T, H, E, k = 37, 64, 5, 3
    x0, lg0, W0, b0 = _rand(1, T, H), _rand(2, T, E), 0.2 * _rand(3, E, H, H), _rand(4, T, H)
    lg0[3, 2:] = float("-inf")
    lg0[4] = float("-inf")
    leaf = lambda t, dt: t.detach().to(dt).requires_grad_()

    def penalty(out, leaves):
        g = torch.autograd.grad((out ** 2).sum(), leaves, create_graph=True)
        g = [torch.where(torch.isfinite(t), t, torch.zeros_like(t)) for t in g]
        sum((t ** 2).sum() for t in g).backward()

    x, lg, W, b = mine = [leaf(t, torch.float32) for t in (x0, lg0, W0, b0)]
    ids, w = el.route(lg, k)
    d = el.Dispatch(ids, E)
    xs = el.dispatch(x, d)
    offs = d.offs.tolist()
    y = torch.cat([torch.tanh(xs[offs[e]:offs[e + 1]] @ W[e]) for e in range(E)] + [xs[offs[E]:] * 0])
    penalty(el.combine(y, w, d, base=b), mine)

    X, L, V, B = ref = [leaf(t, torch.float64) for t in (x0, lg0, W0, b0)]
    rows = []
    for t in range(T):
        n = int(torch.isfinite(lg0[t]).sum().clamp(max=k))
        acc = B[t]
        if n:
            idx = ids[t, :n].long()
            ww = torch.softmax(L[t][idx], 0)
            for j in range(n):
                acc = acc + ww[j] * torch.tanh(X[t] @ V[int(idx[j])])
        rows.append(acc)
    penalty(torch.stack(rows), ref)
    for a, r in zip(mine, ref):
        assert (a.grad.double() - r.grad).abs().max() <= 5e-4 * r.grad.abs().max()


def _small_layer(shared=True):
    from bandwidth_bound_fp8_gb300.expert_layer import Mx4MoeLayer
    E, H, I, k = 12, 512, 256, 3
    return Mx4MoeLayer(0.05 * _rand(1, E, 2 * I, H), 0.05 * _rand(2, E, H, I), k,
                       0.05 * _rand(3, 1, 2 * I, H) if shared else None, 0.05 * _rand(4, 1, H, I) if shared else None)


def _tokens(T):
    return _rand(100 + T, T, 512).to(BF), _rand(200 + T, T, 12)


@pytest.mark.parametrize("shared", [True, False])
def test_one_layer_for_many_token_counts(shared):
    """The bits of a layer that has seen no other number of tokens."""
    layer = _small_layer(shared)
    want = {T: _small_layer(shared)(*_tokens(T)) for T in (1, 3, 16, 250, 700)}
    for T in (16, 1, 250, 3, 700, 16, 250, 1):
        assert torch.equal(layer(*_tokens(T)), want[T])
        assert layer.h.shape[0] == 3 * T


def test_graphs_of_several_token_counts():
    """Graphs captured from one layer, some after a warm-up and one without, replayed in any order between plain calls
    and with other tensors taking whatever memory is free."""
    layer = _small_layer()
    want = {T: _small_layer()(*_tokens(T)) for T in (2, 17, 300, 400)}
    graphs = {}
    for T in (2, 17, 300, 400):
        x, lg = _tokens(T)
        out = torch.zeros_like(x)
        if T != 400:
            layer(x, lg, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer(x, lg, out=out)
        graphs[T] = g, x, lg, out
    assert torch.equal(layer(*_tokens(400)), want[400])
    fill = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (1 << 9, 1 << 14, 1 << 18, 1 << 21, 1 << 24) * 8]
    layer.reserve(900)
    for T in (300, 2, 400, 17, 2, 300, 400):
        g, x, lg, out = graphs[T]
        out.zero_()
        g.replay()
        assert torch.equal(out, want[T]), T
        other = {2: 300, 17: 2, 300: 17, 400: 2}[T]
        assert torch.equal(layer(*_tokens(other)), want[other])
    torch.cuda.synchronize()
    assert all(bool((t == 0xFF).all()) for t in fill)


def test_layer_of_packed_weights():
    """Weights given as MXFP4 codes and scales: the bits of the layer that quantised them itself."""
    from bandwidth_bound_fp8_gb300.expert_layer import Mx4MoeLayer, Mx4Weights
    E, H, I, k = 12, 512, 256, 3
    packed = []
    for s, shape in ((1, (E, 2 * I, H)), (2, (E, H, I)), (3, (1, 2 * I, H)), (4, (1, H, I))):
        code, scale = rp.mx4_codes(rp.to64(0.05 * _rand(s, *shape)).reshape(-1, shape[2]))
        packed.append(Mx4Weights.from_codes(torch.from_numpy(rp.pack_codes(code)).reshape(*shape[:2], -1).cuda(),
                                            torch.from_numpy(scale).reshape(*shape[:2], -1).cuda()))
    layer = Mx4MoeLayer(packed[0], packed[1], k, packed[2], packed[3])
    for T in (1, 250):
        assert torch.equal(layer(*_tokens(T)), _small_layer()(*_tokens(T)))


def test_layer_refuses_tensors_elsewhere():
    layer = _small_layer()
    x, lg = _tokens(4)
    want = layer(x, lg)
    for bad in (dict(x=x.cpu(), logits=lg), dict(x=x, logits=lg.cpu()), dict(x=x, logits=lg, out=x.cpu())):
        with pytest.raises(ValueError, match="on the current CUDA device"):
            layer(**bad)
    assert torch.equal(layer(x, lg), want)
