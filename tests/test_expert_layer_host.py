"""expert_layer's own part (autograd, buffers, checks), on the CPU: the kernel
calls are replaced by torch operations that autograd does not see, as it does
not see the kernels."""
import gc
import weakref

import pytest

torch = pytest.importorskip("torch")

import rows_standins  # noqa: E402

F64 = torch.float64


@pytest.fixture()
def el(monkeypatch):
    rows_standins.use(monkeypatch)
    from bandwidth_bound_fp8_gb300 import expert_layer
    return expert_layer


def _rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def _ids():
    return torch.tensor([[0, 2], [2, 1], [-1, 1], [3, -1], [-1, -1]], dtype=torch.int32)  # 3: an expert held elsewhere


def test_second_derivatives_of_the_movement(el):
    """First and second derivatives against differences, in 64 bits (torch's own checks and tolerances)."""
    d = el.Dispatch(_ids(), 3)
    leaf = lambda s, *shape: _rand(s, *shape).requires_grad_()
    x, y, w, b = leaf(1, 5, 3), leaf(2, 10, 3), leaf(3, 5, 2), leaf(4, 5, 3)
    for f, args in ((lambda x: el.dispatch(x, d), (x,)), (lambda y, w: el.combine(y, w, d), (y, w)),
                    (lambda y, w, b: el.combine(y, w, d, base=b), (y, w, b)),
                    (lambda x, w: el.combine(torch.tanh(el.dispatch(x, d)), w, d, base=x), (x, w))):
        assert torch.autograd.gradcheck(f, args)
        assert torch.autograd.gradgradcheck(f, args)


def test_second_derivatives_of_the_router(el):
    """The same; one row has fewer experts than slots, one has none.  The masked logits stay constants: a difference
    of -inf is no number."""
    free = _rand(5, 4, 6).requires_grad_()
    mask = torch.zeros(4, 6, dtype=torch.bool)
    mask[1, 2:] = True
    mask[2] = True

    def weights(v):
        return el.route(torch.where(mask, torch.full_like(v, -torch.inf), v), 3)[1]

    assert torch.autograd.gradcheck(weights, (free,))
    assert torch.autograd.gradgradcheck(weights, (free,))


def test_gradient_penalty_with_a_constant_incoming_gradient(el):
    """d_y = w d_out and d_logits = w (dw - ..) depend on what was saved, also where the incoming gradient is a
    constant: sum(out) leaves ones."""
    lg0, x0, y_of = _rand(6, 5, 4), _rand(7, 5, 3), _rand(8, 3, 3)
    grads = []
    for plain in (False, True):
        lg, x = lg0.clone().requires_grad_(), x0.clone().requires_grad_()
        if plain:
            v, i = torch.sort(lg, dim=1, descending=True, stable=True)
            w = torch.softmax(v[:, :2], 1)
            out = (w.unsqueeze(2) * torch.tanh(x @ y_of).unsqueeze(1)).sum(1) + w[:, :1] ** 2
        else:
            ids, w = el.route(lg, 2)
            d = el.Dispatch(ids, 4)
            out = el.combine(torch.tanh(el.dispatch(x, d) @ y_of), w, d) + w[:, :1] ** 2
        g = torch.autograd.grad(out.sum(), (lg, x), create_graph=True)
        (sum((t ** 2).sum() for t in g)).backward()
        grads.append((lg.grad, x.grad))
    for a, b in zip(*grads):
        assert b.abs().max() > 1e-3                      # there is something to lose
        assert (a - b).abs().max() <= 1e-12 * (1 + b.abs().max())


def test_any_strides_and_broadcast_inputs(el):
    """Transposes, every second row or column, one row for all: values and gradients of the plain copies, each input's
    gradient in its own shape."""
    lg, x, b, y = (_rand(s, *shape).requires_grad_() for s, shape in
                   ((1, (4, 6)), (2, (3, 6)), (3, (3,)), (4, (3, 18))))

    def loss(view):
        ids, w = el.route(view(lg.t()), 2)
        d = el.Dispatch(ids, 4)
        xs = el.dispatch(view(x.t()), d)
        a = el.combine(view(y.t()[:12]), w, d, base=view(b.expand(6, 3)))
        c = el.combine(xs, w, d, base=view(torch.stack([x.t()] * 2, 2)[:, :, 1]))
        return (a * xs[:6].detach()).sum() + (c ** 2).sum() + (w ** 3).sum()

    got = torch.autograd.grad(loss(lambda t: t), (lg, x, b, y))
    want = torch.autograd.grad(loss(lambda t: t.contiguous()), (lg, x, b, y))
    for g, r in zip(got, want):
        assert torch.equal(g, r) and r.abs().max() > 0


def test_an_overwritten_plan_is_noticed(el):
    d = el.Dispatch(_ids(), 3)
    x = _rand(1, 5, 3).requires_grad_()
    out = el.dispatch(x, d)
    d.pair_row.fill_(-1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


# ------------------------------------------------------------------- buffers
E, H, I, K = 5, 32, 16, 2


def _layer(el, shared=True):
    f = lambda s, *shape: 0.3 * _rand(s, *shape).float()
    return el.Mx4MoeLayer(f(1, E, 2 * I, H), f(2, E, H, I), K, f(3, 1, 2 * I, H) if shared else None,
                          f(4, 1, H, I) if shared else None)


def _inputs(T):
    return _rand(T, T, H).to(torch.bfloat16), _rand(T + 1, T, E).float()


def _want(el, T, shared=True):
    """The layer alone, with buffers of its own."""
    return _layer(el, shared)(*_inputs(T))


@pytest.mark.parametrize("shared", [True, False])
def test_one_layer_for_many_token_counts(el, shared):
    layer = _layer(el, shared)
    for T in (3, 1, 9, 2, 9, 7, 300, 8, 1):
        assert torch.equal(layer(*_inputs(T)), _want(el, T, shared))
        assert layer.ids.shape == (T, K) and layer.h.shape == (T * K, 2 * I)
        if shared:
            assert layer.s_offs.tolist() == [0, T]


def test_fewer_tokens_take_no_new_memory(el, monkeypatch):
    layer = _layer(el)
    layer(*_inputs(12))
    made = []
    real = el._Buffers.__init__
    monkeypatch.setattr(el._Buffers, "__init__", lambda self, *a: (made.append(a), real(self, *a))[1])
    for T in (6, 12, 3, 9):
        layer(*_inputs(T))
    assert not made
    layer.reserve(20)
    layer(*_inputs(18))
    assert len(made) == 1


def test_what_a_captured_graph_uses_stays(el, monkeypatch):
    """A graph replays the addresses it was captured with: they must stay allocated, and the values that no replay
    writes (the shared expert's row range) must stay as they were, whatever runs after."""
    layer = _layer(el)
    state = rows_standins.use(monkeypatch)
    tensors = {}
    for T in (3, 9, 1, 30, 2):
        layer(*_inputs(T))                      # a warm-up, as capture asks for
        state.capturing = True
        layer(*_inputs(T))
        state.capturing = False
        for name, v in [*vars(layer).items(), ("ws", layer.ws.t)]:
            if isinstance(v, torch.Tensor):
                owner = v if v._base is None else v._base
                tensors[T, name] = weakref.ref(owner), v.data_ptr() - owner.data_ptr()
    for T in (50, 4, 30):
        layer(*_inputs(T))
    gc.collect()
    assert len(tensors) == 5 * 11
    assert not [at for at, (owner, _) in tensors.items() if owner() is None]
    for T in (3, 9, 1, 30, 2):
        owner, at = tensors[T, "s_offs"]
        assert owner().reshape(-1)[at // 4:at // 4 + 2].tolist() == [0, T]


def test_a_capture_without_a_warm_up_keeps_nothing(el, monkeypatch):
    """Memory and zeroing inside a capture are the graph's: a later call outside must not take them for its own."""
    layer = _layer(el)
    state = rows_standins.use(monkeypatch)
    state.capturing = True
    layer(*_inputs(4))
    with pytest.raises(RuntimeError, match="captured"):
        layer.reserve(8)
    state.capturing = False
    graph_ws = layer.ws
    layer(*_inputs(4))
    assert layer.ws is not graph_ws
    kept = layer.ws
    state.capturing = True
    layer(*_inputs(40))
    assert layer.ws is not kept
    state.capturing = False
    layer(*_inputs(4))
    assert layer.ws is kept


def test_another_stream_is_recorded(el, monkeypatch):
    layer = _layer(el)
    state = rows_standins.use(monkeypatch)
    layer(*_inputs(4))
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: state.stream)
    layer(*_inputs(4))
    assert not seen
    state.stream = 7
    layer(*_inputs(3))
    layer(*_inputs(4))
    assert {s for _, s in seen} == {7} and len(seen) == len(layer._kept.t) + 1


# -------------------------------------------------------------------- checks
def test_layer_refuses_other_shapes(el):
    """Logits wider than the experts named some that the sort drops; a narrower x fits the same number of tiles."""
    layer = _layer(el)
    x, lg = _inputs(4)
    layer(x, lg)
    wide = torch.cat([lg, lg + 9], 1)
    for bad in ((x, wide), (x, lg[:, :-1]), (x, lg[:3]), (x[:, :-8], lg), (x[0], lg), (x[:0, :-8], lg[:0])):
        with pytest.raises(ValueError):
            layer(*bad)
    for out in (torch.empty(4, H + 1, dtype=x.dtype), torch.empty(5, H, dtype=x.dtype)):
        with pytest.raises(ValueError):
            layer(x, lg, out=out)
    assert layer(x[:0], lg[:0]).shape == (0, H)


def test_layer_refuses_weights_that_do_not_fit(el):
    f = lambda *shape: torch.zeros(shape)
    ok = dict(w_gu=f(E, 2 * I, H), w_d=f(E, H, I), top_k=K, shared_gu=f(1, 2 * I, H), shared_d=f(1, H, I))
    el.Mx4MoeLayer(**ok)
    for bad in (dict(w_gu=f(E, 2 * I + 2, H)), dict(w_gu=f(E + 1, 2 * I, H)), dict(w_gu=f(E, 2 * I, H - 8)),
                dict(w_d=f(E, H, I + 1)), dict(w_d=f(H, I)), dict(shared_gu=f(2, 2 * I, H)), dict(shared_gu=None),
                dict(shared_d=f(1, H - 8, I)), dict(shared_d=f(1, H, I).to("meta"))):
        with pytest.raises(ValueError):
            el.Mx4MoeLayer(**{**ok, **bad})
    el.Mx4MoeLayer(**{**ok, "shared_gu": f(1, 6 * I, H), "shared_d": f(1, H, 3 * I)})   # a shared expert of another width


def test_layer_refuses_a_backward_pass(el):
    """The forward pass is the same for inputs that require a gradient; asking for one raises."""
    layer = _layer(el)
    x, lg = _inputs(4)
    want = layer(x, lg)
    for xr, lr in ((True, False), (False, True)):
        a, b = x.clone().requires_grad_(xr), lg.clone().requires_grad_(lr)
        given = torch.empty_like(x)
        for out in (layer(a, b), layer(a, b, out=given)):
            assert torch.equal(out, want)
            with pytest.raises(RuntimeError, match="no backward pass"):
                out.sum().backward()
        assert torch.equal(given, want) and not given.requires_grad and out.data_ptr() == given.data_ptr()
        with torch.no_grad():
            assert torch.equal(layer(a, b), want) and not layer(a, b).requires_grad


def test_layer_takes_weights_that_are_mxfp4_already(el):
    import rows_plain as rp
    ws = [0.3 * _rand(s, *shape).float() for s, shape in
          ((1, (E, 64, H)), (2, (E, H, 32)), (3, (1, 64, H)), (4, (1, H, 32)))]   # I = 32: a block of scales
    packed, values = [], []
    for w in ws:
        code, scale = rp.mx4_codes(w.reshape(-1, w.shape[2]).numpy())
        packed.append(el.Mx4Weights.from_codes(torch.from_numpy(rp.pack_codes(code)).reshape(*w.shape[:2], -1),
                                               torch.from_numpy(scale).reshape(*w.shape[:2], -1)))
        values.append(torch.from_numpy(rp.mx4_values(code, scale)).float().reshape(w.shape))
        assert packed[-1].shape == tuple(w.shape)
    x, lg = _inputs(4)
    assert torch.equal(el.Mx4MoeLayer(packed[0], packed[1], K, packed[2], packed[3])(x, lg),
                       el.Mx4MoeLayer(values[0], values[1], K, values[2], values[3])(x, lg))
    with pytest.raises(ValueError):
        el.Mx4MoeLayer(packed[0], packed[0], K)


def test_layer_output_may_be_added_to_in_place(el):
    layer = _layer(el)
    x, lg = _inputs(4)
    want = layer(x, lg) + x
    out = layer(x.clone().requires_grad_(), lg)
    out += x
    assert torch.equal(out, want)
    with pytest.raises(RuntimeError, match="no backward pass"):
        out.sum().backward()
