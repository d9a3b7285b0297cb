"""The trainable experts: expert_product to second order, swiglu and
expert_mlp, a whole training step of a layer through them, and its capture."""
import numpy as np
import pytest
import torch

import keep_plain as kp
import rows_plain as rp

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _rand(seed, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).cuda()


def _setup(T=57, E=6, k=2, H=128, I=136, seed=1):
    from bandwidth_bound_fp8_gb300 import expert_layer as el
    lg = _rand(seed, T, E)
    lg[3, 1:] = float("-inf")     # one expert left
    lg[4] = float("-inf")         # none
    lg[:, E - 1] = float("-inf")  # an expert without rows
    x = _rand(seed + 1, T, H).to(BF)
    w_gu, w_d = _rand(seed + 2, E, 2 * I, H, scale=0.1).to(BF), _rand(seed + 3, E, H, I, scale=0.1).to(BF)
    dout = _rand(seed + 4, T, H).to(BF)
    return el, lg, x, w_gu, w_d, dout


def _close(got, ref, rel, what):
    """Off by at most `rel` of the largest of ref's row (matrix)."""
    ref = ref.to(got.device)
    top = ref.abs().amax(-1, keepdim=True)
    err = (got.double() - ref).abs()
    assert (err <= rel * top + 1e-30).all(), f"{what}: {float((err / (top + 1e-30)).max()):.3g} of the largest"


def _layer64(el, lg, x, w_gu, w_d, dout, ids, eight):
    """out and the gradients (logits, x, w_gu, w_d) in 64 bits.  eight: gate, up and x as their 8-bit values in the
    backward pass, through what rounds to bf16 in the kernels' chain."""
    T, k = ids.shape
    b = lambda t: t.to(BF).double()
    L = lg.double().clone().requires_grad_()
    x, w_gu, w_d, dout = (t.double() for t in (x, w_gu, w_d, dout))
    I = w_d.shape[2]
    v8 = lambda t: torch.from_numpy(kp.values(*kp.keep(t.float().cpu().numpy()))).double().cuda()
    x8 = v8(x).to(BF).double() if eight else x
    out, dx, dgu_w, dd_w = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w_gu), torch.zeros_like(w_d)
    dws = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    live = ids >= 0
    picked = torch.where(live, L.gather(1, ids.clamp(min=0).long()), torch.full((), -1e30, dtype=torch.float64, device="cuda"))
    w = torch.where(live, torch.softmax(picked, 1), torch.zeros((), dtype=torch.float64, device="cuda"))
    for e in range(w_gu.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        ww = w.detach()[t, j].float().double()[:, None]
        gu = b(x[t] @ w_gu[e].t())
        g, u = gu[:, :I], gu[:, I:]
        h = b(ww * g * torch.sigmoid(g) * u)
        out.index_add_(0, t, b(h @ w_d[e].t()))
        if eight:
            g, u = v8(g), v8(u)
        sig = torch.sigmoid(g)
        h = b(ww * g * sig * u)
        dh = b(dout[t] @ w_d[e])
        dws[t, j] = (dh * g * sig * u).sum(1)
        dgu = b(torch.cat((ww * dh * u * sig * (1 + g * (1 - sig)), ww * dh * g * sig), 1))
        dd_w[e] = dout[t].t() @ h
        dgu_w[e] = dgu.t() @ x8[t]
        dx.index_add_(0, t, b(dgu @ w_gu[e]))
    (dl,) = torch.autograd.grad(w, L, dws)
    return out, dl, dx, dgu_w, dd_w


def test_training_step_of_a_layer():
    """route, Dispatch, expert_mlp: the output and all gradients against the same chain in 64 bits.  Every value of the
    chain is off by at most a step or so of bf16 (a rounding of a slightly different number may fall the other way), and
    an 8-bit value by a step of its own where its bf16 one flipped; sums of them partly cancel.  3 % of the largest of a
    row bounds both; without the 8 bits the gradients' own error would be up to 2^-4 a term."""
    el, lg, x, w_gu, w_d, dout = _setup()
    leaves = [t.detach().clone().requires_grad_() for t in (lg, x, w_gu, w_d)]
    ids, w = el.route(leaves[0], 2)
    d = el.Dispatch(ids, lg.shape[1])
    out = el.expert_mlp(leaves[1], w, leaves[2], leaves[3], d)
    grads = torch.autograd.grad(out, leaves, dout)
    ref = _layer64(el, lg, x, w_gu, w_d, dout, ids, True)
    _close(out, ref[0], 2.0 ** -7, "out")
    for got, r, what in zip(grads, ref[1:], ("logits", "x", "w_gu", "w_d")):
        _close(got, r, 0.03, what)
    assert (out[4] == 0).all() and (grads[1][4] == 0).all()
    assert (grads[2][-1] == 0).all() and (grads[3][-1] == 0).all()      # the expert without rows
    # and near the gradients without 8 bits: relative to the whole, a term's error of at most 2^-4, uniform, is 2^-4 / sqrt(3)
    exact = _layer64(el, lg, x, w_gu, w_d, dout, ids, False)
    for got, r, what in zip(grads, exact[1:], ("logits", "x", "w_gu", "w_d")):
        assert float((got.double() - r).norm() / r.norm()) < 2 * 2.0 ** -4, what


def test_expert_mlp_is_its_parts():
    """The same output as dispatch, expert_product, swiglu, expert_product and combine with weights 1, bit for bit, and
    the same gradients but for w_gu's, whose rows are x's 8-bit values in one and x's in the other."""
    el, lg, x, w_gu, w_d, dout = _setup()
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    leaves = [t.detach().clone().requires_grad_() for t in (x, w, w_gu, w_d)]
    out = el.expert_mlp(*leaves, d)
    got = torch.autograd.grad(out, leaves, dout)
    parts = [t.detach().clone().requires_grad_() for t in (x, w, w_gu, w_d)]
    h = el.swiglu(el.expert_product(el.dispatch(parts[0], d), parts[2], d), d, parts[1])
    out2 = el.combine(el.expert_product(h, parts[3], d), torch.ones_like(w), d)
    assert torch.equal(out, out2)
    want = torch.autograd.grad(out2, parts, dout)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert float((got[2] - want[2]).float().norm() / want[2].float().norm()) < 2.0 ** -4
    assert float((got[3] - want[3]).float().norm() / want[3].float().norm()) < 2.0 ** -4


def test_only_the_gradients_asked_for():
    """Frozen inputs get none, and those left are the same."""
    el, lg, x, w_gu, w_d, dout = _setup()
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    full = [t.detach().clone().requires_grad_() for t in (x, w, w_gu, w_d)]
    want = torch.autograd.grad(el.expert_mlp(*full, d), full, dout)
    for i in range(4):
        some = [t.detach().clone().requires_grad_(i == j) for j, t in enumerate((x, w, w_gu, w_d))]
        (got,) = torch.autograd.grad(el.expert_mlp(*some, d), some[i], dout)
        assert torch.equal(got, want[i])
    with torch.no_grad():
        assert torch.equal(el.expert_mlp(*full, d), el.expert_mlp(x, w, w_gu, w_d, d))


def test_what_is_kept():
    """Between the passes: x and the gate and up rows in 8 bits, nothing else of their size.  (In the bytes that the
    tensors ask for: an allocation may be handed a whole cached block, up to 1 MB larger, that an earlier test left.)"""
    def held():
        return torch.cuda.memory_stats()["requested_bytes.all.current"]

    el, lg, x, w_gu, w_d, dout = _setup(T=4096, H=512, I=512)
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    w_gu.requires_grad_()
    x.requires_grad_()
    torch.cuda.synchronize()
    before = held()
    out = el.expert_mlp(x, w, w_gu, w_d, d)
    kept = held() - before - out.numel() * 2
    T, H, R, I = 4096, 512, 8192, 512
    assert kept <= (T * H + R * 2 * I) * (1 + 4 / 128) + (1 << 16)


def test_product_to_second_order():
    """Gradients of a gradient penalty, against torch's autograd in 64 bits on the same rows: three bf16 roundings a path
    (2^-9 each at most of what they round, of sums of 64 to 200 terms)."""
    el, lg, x, _, _, _ = _setup(H=64)
    E, N = lg.shape[1], 72
    ids, _ = el.route(lg, 2)
    d = el.Dispatch(ids, E)
    offs = d.offs.tolist()
    w0, dy0 = _rand(9, E, N, 64, scale=0.2).to(BF), _rand(10, x.shape[0] * 2, N).to(BF)
    xs0 = el.dispatch(x, d).detach()

    def penalty(x, w, dy, product):
        gx, gw = torch.autograd.grad(product(x, w), (x, w), dy, create_graph=True)
        return torch.autograd.grad((gx.double() ** 2).sum() + (gw.double() ** 3).sum(), (x, w, dy))

    leaves = [t.clone().requires_grad_() for t in (xs0, w0, dy0)]
    got = penalty(*leaves, lambda x, w: el.expert_product(x, w, d))

    def plain(x, w):
        rows = [x[offs[e]:offs[e + 1]] @ w[e].t() for e in range(E)]
        return torch.cat(rows + [torch.zeros((x.shape[0] - offs[E], N), dtype=torch.float64, device="cuda")])
    ref = penalty(*(t.double().clone().requires_grad_() for t in (xs0, w0, dy0)), plain)
    for g, r, what in zip(got, ref, ("x", "w", "dy")):
        assert float((g.double() - r).norm() / r.norm()) < 0.01, what


def test_differentiable_once():
    el, lg, x, w_gu, w_d, dout = _setup()
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    leaves = [t.detach().clone().requires_grad_() for t in (x, w, w_gu, w_d)]
    grads = torch.autograd.grad(el.expert_mlp(*leaves, d), leaves, dout, create_graph=True)
    for g in grads:
        with pytest.raises(RuntimeError, match="differentiable once"):
            torch.autograd.grad(g.float().sum(), leaves, allow_unused=True, retain_graph=True)
    gu = _rand(1, d.row_pair.numel(), 64).requires_grad_()
    (g,) = torch.autograd.grad(el.swiglu(gu, d, leaves[1]).sum(), gu, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        g.sum().backward()


def test_unusual_gradients_and_layouts():
    """An expanded gradient (of a sum), inputs with strides, a transposed weight: as with contiguous ones."""
    el, lg, x, w_gu, w_d, _ = _setup()
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    leaf = lambda t: t.detach().clone().requires_grad_()
    plain = [leaf(t) for t in (x, w, w_gu, w_d)]
    want = torch.autograd.grad(el.expert_mlp(*plain, d).sum(), plain)
    T, H = x.shape
    wide = leaf(torch.cat((x, x), 1))
    wt = leaf(w.t().contiguous())
    gt = leaf(w_gu.transpose(1, 2).contiguous())
    out = el.expert_mlp(wide[:, H:], wt.t(), gt.transpose(1, 2), plain[3], d)
    gx, gw, gg = torch.autograd.grad(out.sum(), (wide, wt, gt))
    assert torch.equal(gx[:, H:], want[0]) and (gx[:, :H] == 0).all()
    assert torch.equal(gw.t(), want[1]) and torch.equal(gg.transpose(1, 2), want[2])
    odd = torch.empty((T * 2, H + 1), dtype=BF, device="cuda")[:, 1:]
    odd.copy_(el.dispatch(x, d))
    y, y2 = el.expert_product(odd, w_gu, d), el.expert_product(el.dispatch(x, d), w_gu, d)
    assert torch.equal(y, y2)


def test_no_tokens():
    el, _, _, w_gu, w_d, _ = _setup()
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    d = el.Dispatch(ids, w_gu.shape[0])
    x, w = torch.empty((0, w_gu.shape[2]), dtype=BF, device="cuda"), torch.empty((0, 2), device="cuda")
    leaves = [t.detach().clone().requires_grad_() for t in (x, w, w_gu, w_d)]
    out = el.expert_mlp(*leaves, d)
    grads = torch.autograd.grad(out, leaves, torch.empty_like(out))
    assert out.shape == x.shape and (grads[2] == 0).all() and (grads[3] == 0).all()


def test_captured_training_step():
    """Forward and backward pass in one graph, replayed on new inputs and another routing (the eager graph is gone
    before the capture)."""
    el, lg, x, w_gu, w_d, dout = _setup(T=130, I=256)

    def step(leaves, dout):
        ids, w = el.route(leaves[0], 2)
        d = el.Dispatch(ids, leaves[0].shape[1])
        out = el.expert_mlp(leaves[1], w, leaves[2], leaves[3], d)
        return (out.detach(), *torch.autograd.grad(out, leaves, dout))
    static = [t.detach().clone().requires_grad_() for t in (lg, x, w_gu, w_d)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static, dout)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(static, dout)
    torch.cuda.synchronize()
    _, lg2, x2, gu2, d2, dout2 = _setup(T=130, I=256, seed=40)
    with torch.no_grad():
        for t, v in zip((*static, dout), (lg2, x2, gu2, d2, dout2)):
            t.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    want = step([t.requires_grad_() for t in (lg2, x2, gu2, d2)], dout2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_few_steps_of_training_run():
    """An optimiser's steps: finite gradients, changed weights."""
    el, lg, x, w_gu, w_d, dout = _setup()
    params = [torch.nn.Parameter(t) for t in (w_gu, w_d)]
    opt = torch.optim.SGD(params, lr=1e-3)
    for _ in range(3):
        ids, w = el.route(lg, 2)
        d = el.Dispatch(ids, lg.shape[1])
        loss = (el.expert_mlp(x, w, *params, d).float() - dout.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        assert all(torch.isfinite(p.grad).all() and p.grad.abs().sum() > 0 for p in params)
        opt.step()


def test_a_penalty_on_what_was_quantised_raises():
    """A loss linear in the output, with the rows or tokens as the only leaf: their gradient's square has a gradient, which
    the codes do not give.  What stands for them in the graph keeps no memory."""
    el, lg, x, w_gu, w_d, _ = _setup()
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    gu = _rand(1, d.row_pair.numel(), 64)
    for f, t in ((lambda t: el.swiglu(t, d), gu), (lambda t: el.swiglu(t, d, w), gu), (lambda t: el.expert_mlp(t, w, w_gu, w_d, d), x)):
        leaf = t.detach().clone().requires_grad_()
        (first,) = torch.autograd.grad(f(leaf).sum(), leaf)
        out = f(leaf).sum()
        (g,) = torch.autograd.grad(out, leaf, create_graph=True)
        assert torch.equal(g.detach(), first)
        with pytest.raises(RuntimeError, match="differentiable once"):
            (out + g.float().square().sum()).backward()


def test_a_plan_tells_of_its_products():
    """No product reports anything; what one leaves in the plan's word is raised, and is not the next plan's."""
    from bandwidth_bound_fp8_gb300 import moeq
    el, lg, x, w_gu, w_d, dout = _setup()
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    w_gu.requires_grad_()
    el.expert_mlp(x, w, w_gu, w_d, d).backward(dout)
    el.expert_product(el.dispatch(x, d), w_gu, d).sum().backward()
    d.check()
    d.status.fill_(moeq.MOEQ_ERR_TIMEOUT)
    with pytest.raises(moeq.MoeqError, match="status 5"):
        d.check()
    el.Dispatch(ids, lg.shape[1]).check()


def test_weights_in_a_flat_buffer():
    """Weights that start off 16 bytes: the same results, and gradients in the buffer."""
    el, lg, x, w_gu, w_d, dout = _setup()
    ids, w = el.route(lg, 2)
    d = el.Dispatch(ids, lg.shape[1])
    plain = [t.detach().clone().requires_grad_() for t in (w_gu, w_d)]
    out = el.expert_mlp(x, w, *plain, d)
    want = torch.autograd.grad(out, plain, dout)
    n = w_gu.numel()
    flat = torch.cat((torch.zeros(1, dtype=BF, device="cuda"), w_gu.reshape(-1), w_d.reshape(-1))).requires_grad_()
    gu, dn = flat[1:n + 1].view(w_gu.shape), flat[n + 1:].view(w_d.shape)
    assert gu.is_contiguous() and gu.data_ptr() % 16
    out2 = el.expert_mlp(x, w, gu, dn, d)
    (got,) = torch.autograd.grad(out2, flat, dout)
    assert torch.equal(out, out2) and torch.equal(got[1:], torch.cat([t.reshape(-1) for t in want])) and got[0] == 0
    xs = el.dispatch(x, d)
    assert torch.equal(el.expert_product(xs, gu, d), el.expert_product(xs, w_gu, d))


def test_plans_have_words_of_their_own():
    """More plans than are zeroed at once, on two streams; and one inside a graph, whose word every replay clears."""
    from bandwidth_bound_fp8_gb300 import moeq
    el, lg, *_ = _setup()
    ids, _ = el.route(lg, 2)
    E, side = lg.shape[1], torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plans = [el.Dispatch(ids, E) for _ in range(300)]
    with torch.cuda.stream(side):
        plans += [el.Dispatch(ids, E) for _ in range(300)]
    torch.cuda.synchronize()
    assert len({d.status.data_ptr() for d in plans}) == len(plans) and all(int(d.status) == 0 for d in plans)
    plans[7].status.fill_(moeq.MOEQ_ERR_TIMEOUT)
    plans[6].check(), plans[8].check()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            d = el.Dispatch(ids, E)
    graph.replay()
    d.check()
    d.status.fill_(moeq.MOEQ_ERR_TIMEOUT)
    with pytest.raises(moeq.MoeqError):
        d.check()
    graph.replay()
    d.check()
