"""What expert_layer makes of its training calls, on the CPU: the calls are
replaced by plain forms that write through .data, as the kernels write through
pointers."""
import pytest
import torch

import keep_plain as kp
import rows_standins

F = torch.nn.functional


def _each(offs, E):
    return [(e, slice(int(offs[e]), int(offs[e + 1]))) for e in range(E)]


def _fits(t):
    """Rows that tensor copies can read."""
    assert t.dim() == 2 and t.stride(1) == 1 and t.data_ptr() % 16 == 0 and (t.shape[0] <= 1 or t.stride(0) % 8 == 0)


def product(x, w, offs, y, status=None, stream=None):
    _fits(x)
    assert w.is_contiguous()
    y.data.zero_()
    for e, at in _each(offs, w.shape[0]):
        y.data[at] = x.data[at] @ w.data[e].t()


def product_grad_x(dy, w, offs, dx, status=None, stream=None):
    _fits(dy)
    dx.data.zero_()
    for e, at in _each(offs, w.shape[0]):
        dx.data[at] = dy.data[at] @ w.data[e]


def product_grad_w(dy, x, offs, dw, status=None, stream=None):
    _fits(dy), _fits(x)
    for e, at in _each(offs, dw.shape[0]):
        dw.data[e] = dy.data[at].t() @ x.data[at]


def quant(x, codes, scales, stream=None):
    c, s = kp.keep(x.detach().float().numpy())
    codes.copy_(torch.from_numpy(c))
    scales.copy_(torch.from_numpy(s))


def gather8(codes, scales, offs, pair_row, xs, stream=None):
    v = torch.from_numpy(kp.values(codes.numpy(), scales.numpy())).to(xs.dtype)
    rows_standins.gather_rows(v, offs, pair_row, xs)


def _w(row_pair, w):
    live = row_pair >= 0
    v = torch.ones(row_pair.shape[0], dtype=torch.float64) if w is None else w.data.reshape(-1)[row_pair.clamp(min=0).long()].double()
    return torch.where(live, v, torch.zeros((), dtype=torch.float64)).numpy(), live


def swiglu(gu, h, row_pair=None, topk_w=None, codes=None, scales=None, stream=None):
    w, live = _w(row_pair, topk_w)
    z = torch.where(live[:, None], gu.data, torch.zeros((), dtype=gu.dtype)).double().numpy()
    I = z.shape[1] // 2
    h.data.copy_(torch.from_numpy(kp.swiglu(z[:, :I], z[:, I:], w)))
    if codes is not None:
        c, s = kp.keep_gate_up(z.astype("float32"))
        codes.copy_(torch.from_numpy(c))
        scales.copy_(torch.from_numpy(s))


def swiglu_grad(d_h, codes, scales, d_gu, h=None, row_pair=None, topk_w=None, pair_row=None, d_topk_w=None, stream=None):
    w, live = _w(row_pair, topk_w)
    gate, up = (v.astype("float64") for v in kp.values_gate_up(codes.numpy(), scales.numpy()))
    dg, du, hh, dw = kp.swiglu_grad(d_h.data.double().numpy(), gate, up, w)
    d_gu.data.copy_(torch.cat((torch.from_numpy(dg), torch.from_numpy(du)), 1))
    if h is not None:
        h.data.copy_(torch.from_numpy(hh))
    if d_topk_w is not None:
        d_topk_w.data.zero_()
        d_topk_w.data.view(-1)[row_pair[live].long()] = torch.from_numpy(dw).float()[live]


@pytest.fixture()
def el(monkeypatch):
    from bandwidth_bound_fp8_gb300 import expert_layer, moeq
    rows_standins.use(monkeypatch)
    for name, f in (("expert_product", product), ("expert_product_grad_x", product_grad_x),
                    ("expert_product_grad_w", product_grad_w), ("fp8_quant_rows", quant), ("fp8_gather_rows", gather8),
                    ("swiglu_rows", swiglu), ("swiglu_rows_grad", swiglu_grad)):
        monkeypatch.setattr(moeq, "moeq_" + name, f)
    return expert_layer


def _plan(el, T=9, E=4, k=2, seed=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    ids[0, 1] = -1
    ids[2] = -1
    return el.Dispatch(ids, E), ids


def _leaf(g, *s, dt=torch.float64, scale=1.0):
    return (scale * torch.randn(s, generator=g, dtype=torch.float64)).to(dt).requires_grad_()


def test_product_gradients_to_second_order(el):
    """In 64 bits, against differences."""
    d, _ = _plan(el)
    g = torch.Generator().manual_seed(1)
    R, K, N = d.row_pair.numel(), 8, 16
    x, w = _leaf(g, R, K), _leaf(g, 4, N, K)
    f = lambda x, w: el.expert_product(x, w, d)
    assert torch.autograd.gradcheck(f, (x, w))
    assert torch.autograd.gradgradcheck(f, (x, w))


def test_product_takes_any_layout(el):
    """Rows that tensor copies cannot read are copied; an expanded gradient too."""
    d, _ = _plan(el)
    g = torch.Generator().manual_seed(2)
    R, K, N = d.row_pair.numel(), 8, 16
    x, w = _leaf(g, R, K), _leaf(g, 4, N, K)
    want = torch.autograd.grad(el.expert_product(x, w, d).sum(), (x, w))
    odd = torch.zeros((R, K + 3), dtype=torch.float64)
    odd[:, 1:K + 1] = x.detach()
    odd.requires_grad_()
    wt = w.detach().transpose(1, 2).contiguous().requires_grad_()
    gx, gw = torch.autograd.grad(el.expert_product(odd[:, 1:K + 1], wt.transpose(1, 2), d).sum(), (odd, wt))
    assert torch.equal(gx[:, 1:K + 1], want[0]) and torch.equal(gw.transpose(1, 2), want[1])


def _values(t):
    return torch.from_numpy(kp.values(*kp.keep(t.detach().float().numpy()))).to(t.dtype)


def test_swiglu_sees_eight_bits(el):
    """Its gradient is the formula's at the 8-bit values; without a gradient nothing is kept."""
    d, _ = _plan(el)
    g = torch.Generator().manual_seed(3)
    R, I = d.row_pair.numel(), 24
    gu, w = _leaf(g, R, 2 * I, dt=torch.float32), _leaf(g, 9, 2, dt=torch.float32)
    dh = torch.randn(R, I, generator=g)
    h = el.swiglu(gu, d, w)
    got = torch.autograd.grad(h, (gu, w), dh)
    at = torch.cat((_values(gu[:, :I]), _values(gu[:, I:])), 1).double().requires_grad_()
    w64 = w.detach().double().requires_grad_()
    live = d.row_pair >= 0
    wr = torch.where(live, w64.reshape(-1)[d.row_pair.clamp(min=0).long()], torch.zeros((), dtype=torch.float64))
    want = torch.autograd.grad(wr[:, None] * F.silu(at[:, :I]) * at[:, I:], (at, w64), dh.double())
    for a, b in zip(got, want):
        assert torch.allclose(a.double(), b, rtol=1e-5, atol=1e-6)
    with torch.no_grad():
        assert torch.equal(el.swiglu(gu, d, w), h)
    (once,) = torch.autograd.grad(el.swiglu(gu, d, w), gu, dh, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        once.sum().backward()


def test_expert_mlp_refuses_what_does_not_fit(el):
    d, _ = _plan(el)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    ok = dict(x=z(9, 16), w=z(9, 2, dt=torch.float32), w_gu=z(4, 48, 16), w_d=z(4, 16, 24))
    call = lambda **kw: el.expert_mlp(*{**ok, **kw}.values(), d)
    for bad in (dict(x=z(8, 16)), dict(x=z(9, 16, dt=torch.float32)), dict(w=z(9, 3, dt=torch.float32)), dict(w=z(9, 2)),
                dict(w_gu=z(5, 48, 16)), dict(w_gu=z(4, 48, 8)), dict(w_gu=z(4, 47, 16)), dict(w_d=z(4, 16, 23)),
                dict(w_d=z(4, 24, 16)), dict(w_d=z(3, 16, 24))):
        with pytest.raises(ValueError, match="expert_mlp"):
            call(**bad)
    with pytest.raises(ValueError, match="expert_product"):
        el.expert_product(z(18, 16), z(4, 48, 8), d)
    with pytest.raises(ValueError, match="swiglu"):
        el.swiglu(z(18, 15), d)
    with pytest.raises(ValueError, match="swiglu"):
        el.swiglu(z(17, 16), d)
    with pytest.raises(ValueError, match="swiglu"):
        el.swiglu(z(18, 16), d, z(9, 2))


def _penalised(f, leaf):
    """A loss that is linear in f(leaf), and the square of its gradient: the latter's gradient has to raise."""
    (plain,) = torch.autograd.grad(f(leaf).double().sum(), leaf)
    out = f(leaf).double().sum()
    (g,) = torch.autograd.grad(out, leaf, create_graph=True)
    assert torch.equal(g.detach(), plain)
    penalty = g.double().square().sum()
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(penalty + leaf.double().sum(), leaf, retain_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        (out + penalty).backward()


@pytest.mark.parametrize("weighted", [False, True])
def test_a_second_derivative_through_swiglu_raises(el, weighted):
    """d_gu depends on gu through its 8-bit codes, also where d_h and the weights need no gradient."""
    d, _ = _plan(el)
    g = torch.Generator().manual_seed(5)
    R, I = d.row_pair.numel(), 24
    w = _leaf(g, 9, 2, dt=torch.float32).detach() if weighted else None
    _penalised(lambda gu: el.swiglu(gu, d, w), _leaf(g, R, 2 * I, dt=torch.float32))
    # ahead of it a function that is differentiable to any order
    x, ew = _leaf(g, R, 8, dt=torch.float32), _leaf(g, 4, 2 * I, 8, dt=torch.float32)
    (dx,) = torch.autograd.grad(el.swiglu(el.expert_product(x, ew, d), d, w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(dx.square().sum(), ew)


@pytest.mark.parametrize("which", range(4))
def test_a_second_derivative_through_expert_mlp_raises(el, which):
    """With each of x, w, w_gu and w_d as the only one that needs a gradient."""
    d, _ = _plan(el)
    g = torch.Generator().manual_seed(6)
    bf = torch.bfloat16
    args = [_leaf(g, *s, dt=dt, scale=0.3).detach() for s, dt in (((9, 16), bf), ((9, 2), torch.float32), ((4, 48, 16), bf),
                                                                  ((4, 16, 24), bf))]
    leaf = args[which].clone().requires_grad_()
    _penalised(lambda t: el.expert_mlp(*args[:which], t, *args[which + 1:], d), leaf)


def test_product_wants_the_dispatched_rows(el):
    """Rows that are not the plan's T * k (tokens that were not dispatched, a part of the rows) are refused."""
    d, _ = _plan(el)
    w = torch.zeros((4, 8, 16))
    for rows in (9, 17, 19, 0):
        with pytest.raises(ValueError, match=r"expert_product: x \[18, K\]"):
            el.expert_product(torch.zeros((rows, 16)), w, d)
    for shape in ((18,), (18, 16, 1)):
        with pytest.raises(ValueError, match="expert_product"):
            el.expert_product(torch.zeros(shape), w, d)
    assert el.expert_product(torch.zeros((18, 16)), w, d).shape == (18, 8)


@pytest.mark.parametrize("name", ["expert_product", "expert_product_grad_x", "expert_product_grad_w"])
@pytest.mark.parametrize("turn", [0, 1])
def test_a_product_that_gives_up_is_reported(el, monkeypatch, name, turn):
    """The plan's status word reaches every product, of each pass; check() raises what one of them left there."""
    from bandwidth_bound_fp8_gb300 import moeq
    plain, calls = getattr(moeq, "moeq_" + name), []

    def gives_up(a, b, offs, out, status=None, stream=None):
        plain(a, b, offs, out)
        assert status is not None and status.dtype is torch.int32 and status.shape == (1,)
        calls.append(status)
        if len(calls) == turn + 1:
            status.data.fill_(moeq.MOEQ_ERR_TIMEOUT)
    monkeypatch.setattr(moeq, "moeq_" + name, gives_up)
    g = torch.Generator().manual_seed(7)
    bf, dx = torch.bfloat16, None
    d, _ = _plan(el)
    d.check()
    args = [_leaf(g, *s, dt=dt) for s, dt in (((9, 16), bf), ((9, 2), torch.float32), ((4, 48, 16), bf), ((4, 16, 24), bf))]
    el.expert_mlp(*args, d).sum().backward()
    assert len(calls) == 2 and all(c is d.status for c in calls)
    with pytest.raises(moeq.MoeqError) as e:
        d.check()
    assert e.value.status == moeq.MOEQ_ERR_TIMEOUT
    # a plan of its own knows nothing of it; the product's own gradients, to second order
    calls.clear()
    d, _ = _plan(el)
    x, w = _leaf(g, 18, 8), _leaf(g, 4, 16, 8)
    dx, dw = torch.autograd.grad(el.expert_product(x, w, d).square().sum(), (x, w), create_graph=True)
    (dx.square().sum() + dw.square().sum()).backward()
    assert len(calls) > 1 and all(c is d.status for c in calls)
    with pytest.raises(moeq.MoeqError):
        d.check()


def test_a_tangent_is_not_dropped(el):
    """Forward-mode differentiation through a backward pass: none of the functions has a rule for it, so all raise, in
    place of gradients without their tangent."""
    from torch.autograd import forward_ad as fwd
    d, ids = _plan(el)
    g = torch.Generator().manual_seed(8)
    f32, bf = torch.float32, torch.bfloat16
    x, w, lg = _leaf(g, 18, 8), _leaf(g, 9, 2, dt=f32), _leaf(g, 9, 4, dt=f32)
    ew, gu, t = _leaf(g, 4, 16, 8), _leaf(g, 18, 48, dt=f32), _leaf(g, 9, 8, dt=f32)
    mlp = [_leaf(g, *s, dt=bf).detach() for s in ((4, 48, 16), (4, 16, 24))]
    tok = _leaf(g, 9, 16, dt=bf)
    for out, leaves in ((el.expert_product(x, ew, d), (x, ew)), (el.swiglu(gu, d, w), (gu, w)), (el.swiglu(gu, d), (gu,)),
                        (el.expert_mlp(tok, w, *mlp, d), (tok, w)), (el.dispatch(t, d), (t,)),
                        (el.combine(gu, w, d), (gu, w)), (el.route(lg, 2)[1], (lg,))):
        first = torch.autograd.grad(out, leaves, torch.ones_like(out), retain_graph=True)
        with fwd.dual_level():
            dual = fwd.make_dual(torch.ones_like(out), torch.ones_like(out))
            with pytest.raises(RuntimeError, match="forward"):
                torch.autograd.grad(out, leaves, dual, retain_graph=True)
            again = torch.autograd.grad(out, leaves, torch.ones_like(out), retain_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    # and through a second backward pass
    gx, gw = torch.autograd.grad(el.expert_product(x, ew, d), (x, ew), torch.ones(18, 16, dtype=x.dtype), create_graph=True)
    for a, leaf in ((gx, ew), (gw, x)):
        with fwd.dual_level():
            with pytest.raises(RuntimeError, match="forward"):
                torch.autograd.grad(a, leaf, fwd.make_dual(torch.ones_like(a), torch.ones_like(a)), retain_graph=True)


def _off(t):
    """t in a buffer, contiguous, off a boundary of 16 bytes."""
    flat = torch.zeros(t.numel() + 8, dtype=t.dtype)
    n = 1 if flat.data_ptr() % 16 == 0 else 0
    out = flat[n:n + t.numel()].view(t.shape)
    out.copy_(t.detach())
    assert out.is_contiguous() and out.data_ptr() % 16
    return out.requires_grad_(t.requires_grad)


def test_weights_off_16_bytes_are_copied(el, monkeypatch):
    """Contiguous weights (and second-order gradients in their place) that are slices of a flat buffer."""
    from bandwidth_bound_fp8_gb300 import moeq
    for name in ("moeq_expert_product", "moeq_expert_product_grad_x"):
        def aligned(a, w, offs, out, status=None, stream=None, plain=getattr(moeq, name)):
            assert w.is_contiguous() and w.data_ptr() % 16 == 0
            plain(a, w, offs, out)
        monkeypatch.setattr(moeq, name, aligned)
    d, _ = _plan(el)
    g = torch.Generator().manual_seed(9)
    bf = torch.bfloat16
    x, w = _leaf(g, 18, 8), _leaf(g, 4, 16, 8)
    dy, gw = torch.randn(18, 16, generator=g, dtype=x.dtype), torch.randn(4, 16, 8, generator=g, dtype=x.dtype)
    def second(w, gw):
        y = el.expert_product(x, w, d)
        dx, dw = torch.autograd.grad(y, (x, w), dy, create_graph=True)
        return (y.detach(), dx.detach(), dw.detach(), *torch.autograd.grad((dx, dw), (x, w), (torch.ones_like(dx), gw)))
    for a, b in zip(second(w, gw), second(_off(w), _off(gw))):
        assert torch.equal(a, b)
    args = [_leaf(g, *s, dt=dt, scale=0.3) for s, dt in (((9, 16), bf), ((9, 2), torch.float32), ((4, 48, 16), bf), ((4, 16, 24), bf))]
    moved = args[:2] + [_off(t) for t in args[2:]]
    out, out2 = el.expert_mlp(*args, d), el.expert_mlp(*moved, d)
    assert torch.equal(out, out2)
    for a, b in zip(torch.autograd.grad(out.float().sum(), args), torch.autograd.grad(out2.float().sum(), moved)):
        assert torch.equal(a, b)


def test_no_gradient_of_the_output_is_zero(el):
    """What follows has no gradient to give: zeros, as ever."""
    class Nothing(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            return t.clone()

        @staticmethod
        def backward(ctx, _):
            return None
    d, _ = _plan(el)
    g = torch.Generator().manual_seed(10)
    gu, w = _leaf(g, 18, 48, dt=torch.float32), _leaf(g, 9, 2, dt=torch.float32)
    tok, *mlp = (_leaf(g, *s, dt=torch.bfloat16) for s in ((9, 16), (4, 48, 16), (4, 16, 24)))
    for out, leaves in ((el.swiglu(gu, d, w), (gu, w)), (el.expert_mlp(tok, w, *mlp, d), (tok, w, *mlp))):
        for got, leaf in zip(torch.autograd.grad(Nothing.apply(out).sum(), leaves), leaves):
            assert got.shape == leaf.shape and got.dtype is leaf.dtype and (got == 0).all()
