"""expert_layer's own part (autograd, buffers, checks), on the CPU: the kernel
calls are replaced by torch operations that autograd does not see, as it does
not see the kernels."""
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


def test_an_overwritten_plan_is_noticed(el):
    d = el.Dispatch(_ids(), 3)
    x = _rand(1, 5, 3).requires_grad_()
    out = el.dispatch(x, d)
    d.pair_row.fill_(-1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
