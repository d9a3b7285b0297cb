"""Cases that time the expert layer's operators at any number of tokens:
routing, the sort of tokens by expert, moving rows to the experts and back
with their gradients, MXFP4 quantisation, and the experts' MXFP4 products.

Shapes are those of the layer this library is benchmarked on (hidden 6144,
256 experts of intermediate 2048, top-8), and generic ones around them.

MXFP4 (OCP microscaling): blocks of 32 along K share a power-of-two scale
2^s, s = max(floor(log2 amax) - 2, -127); an element is one of the sixteen
values +-{0, .5, 1, 1.5, 2, 3, 4, 6}, rounded to nearest, ties to the even
code, saturating.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------- cases
def listed():
    return [
        # the router of one decoded token: the smallest call, all latency
        dict(name="route_t1", op="route", T=1, E=256, k=8, masked=0.0, grad=False),
        # a training batch's router, forward and backward, some experts masked off
        dict(name="route_train_t8191", op="route", T=8191, E=256, k=8, masked=0.25, grad=True),
        # a decode batch of 16 tokens sorted by expert
        dict(name="sort_t16", op="sort", T=16, E=256, k=8, drop=0.0),
        # a long prompt's tokens sorted by expert; a quarter of the slots go to experts held elsewhere
        dict(name="sort_t32768", op="sort", T=32768, E=256, k=8, drop=0.25),
        # a decode batch moved to its experts and back
        dict(name="rows_t16", op="rows", T=16, H=6144, E=256, k=8, drop=0.0, dtype="bf16", base=True, grad=False),
        # a training step's movement of rows at the benchmark's width, all four directions
        dict(name="rows_train_t4095", op="rows", T=4095, H=6144, E=256, k=8, drop=0.0, dtype="bf16", base=True,
             grad=True),
        # the same in fp32 at an odd width, no shared expert, slots dropped
        dict(name="rows_train_f32_h1001", op="rows", T=2049, H=1001, E=60, k=4, drop=0.25, dtype="f32", base=False,
             grad=True),
        # a decode batch's activations to 4 bits and back to values
        dict(name="quant_t16", op="quant", rows=16, K=6144, dtype="bf16"),
        # a prompt's activations to 4 bits and back to values
        dict(name="quant_t8191", op="quant", rows=8191, K=6144, dtype="bf16"),
        # one decoded token through its eight experts' gate and up rows: a stream of 4-bit weights
        dict(name="product_t1", op="product", T=1, K=6144, N=4096, E=256, k=8, gather=True, dtype="bf16", y="f32",
             skew=0.0),
        # a batch of decoded tokens, one or two rows at most experts: every expert's weights are read
        dict(name="product_t61", op="product", T=61, K=6144, N=4096, E=256, k=8, gather=True, dtype="bf16", y="bf16",
             skew=0.5),
        # a long prompt through the experts' gate and up rows: tensor-core work on ragged groups
        dict(name="product_t8192", op="product", T=8192, K=6144, N=4096, E=256, k=8, gather=True, dtype="bf16",
             y="bf16", skew=0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "sort", "rows", "quant", "product", "product"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, 8), masked=rng.choice([0.0, 0.25, 0.9]),
                    grad=rng.random() < 0.5)
    if op == "sort":
        return dict(op=op, T=_log_int(rng, 1, 65536), E=rng.choice([8, 60, 64, 160, 256, 1000]), k=rng.randint(1, 8),
                    drop=rng.choice([0.0, 0.25, 0.9]))
    if op == "rows":
        return dict(op=op, T=_log_int(rng, 1, 4095), H=rng.choice([128, 1000, 1001, 1408, 2048, 4096, 5120, 6144]),
                    E=rng.choice([8, 60, 256]), k=rng.randint(1, 8), drop=rng.choice([0.0, 0.25]),
                    dtype=rng.choice(["bf16", "f32"]) if rng.random() < 0.5 else "bf16", base=rng.random() < 0.5,
                    grad=rng.random() < 0.5)
    if op == "quant":
        return dict(op=op, rows=_log_int(rng, 1, 8191), K=rng.choice([32, 160, 512, 1408, 2048, 4096, 6144]),
                    dtype=rng.choice(["bf16", "f32"]))
    # experts of the benchmark's layer and of smaller ones, and dense products (E = 1)
    E, k = rng.choice([(1, 1), (8, 2), (64, 6), (256, 8)])
    K, N = rng.choice([(6144, 4096), (2048, 6144), (2048, 2816), (1408, 2048), (1056, 1000)])
    return dict(op="product", T=_log_int(rng, 1, 4096), K=K, N=N, E=E, k=k, gather=rng.random() < 0.5,
                dtype=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "f32"]), skew=rng.choice([0.0, 0.5, 1.0]))


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float32, device="cuda")


def _logits(g, T, E, skew=0.0):
    """Router logits, of bf16's precision as a bf16 projection leaves them (so ties occur)."""
    x = _normal(g, T, E) + skew * _normal(g, 1, E)
    return x.to(torch.bfloat16).to(torch.float32)


def _picks(logits, k):
    """[T, k] expert ids by falling logit, ties to the lower id."""
    return torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()


def _activations(g, T, K):
    """N(0, 1) with 1% of the channels thirty times as large."""
    x = _normal(g, T, K)
    ch = torch.randperm(K, generator=g, device="cuda")[: K // 100]
    x[:, ch] *= 30.0
    return x


def _sorted(ids, E):
    """offs [E+1], pair_row [T, k], row_pair [T*k] of the stable sort by expert; ids outside [0, E) get no row."""
    T, k = ids.shape
    P = T * k
    flat = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E)).reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    counts.index_add_(0, flat, torch.ones(P, dtype=torch.int32, device=ids.device))
    offs = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offs[1:] = torch.cumsum(counts[:E], 0)
    at = torch.arange(P, dtype=torch.int32, device=ids.device)
    kept = flat[order] < E
    row_pair = torch.where(kept, order.to(torch.int32), torch.full_like(at, -1))
    pair_row = torch.empty_like(at)
    pair_row[order] = torch.where(kept, at, torch.full_like(at, -1))
    return offs, pair_row.view(T, k), row_pair


def _dropped(g, ids, drop):
    if not drop:
        return ids
    out = torch.rand(ids.shape, generator=g, device="cuda") < drop
    return torch.where(out, torch.full_like(ids, -1), ids)


def _pow2(e):
    """2^e as fp32 for whole e in [-126, 127], from its bits."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _mx4(x):
    """fp32 [.., K] -> codes' values (fp32) and exponents (int32 [.., K/32]) of MXFP4."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    e = e.clamp(min=-127)
    v = b * _pow2(-e).unsqueeze(-1)
    a = v.abs()
    m = 0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + 1.0 * (a > 2.5) + 1.0 * (a >= 3.5)
    m = m + 2.0 * (a > 5.0)
    return torch.copysign(m, v), e


def _mx4_value(q, e):
    """The fp32 values that codes' values and exponents stand for."""
    half = e >> 1
    return (q * _pow2(half).unsqueeze(-1) * _pow2(e - half).unsqueeze(-1)).flatten(-2)


def _pack(q, e):
    """Codes' values and exponents -> two E2M1 codes a byte (the lower column in the low bits), and scale bytes."""
    a = q.abs()
    code = sum((a >= v).to(torch.uint8) for v in E2M1[1:])
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _unpack(codes, scales):
    """Packed codes and scale bytes -> fp32 values."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    q = table[c.int()].unflatten(-1, (-1, 32))
    return _mx4_value(q, scales.to(torch.int32) - 127)


def _inputs(case, seed):
    g, c = _gen(seed), case
    if c["op"] == "route":
        lg = _logits(g, c["T"], c["E"])
        if c["masked"]:
            off = torch.rand(lg.shape, generator=g, device="cuda") < c["masked"]
            lg = torch.where(off, torch.full_like(lg, -math.inf), lg)
        return dict(logits=lg, dw=_normal(g, c["T"], c["k"]))
    if c["op"] == "sort":
        return dict(ids=_dropped(g, _picks(_logits(g, c["T"], c["E"], 0.5), c["k"]), c["drop"]))
    if c["op"] == "rows":
        T, H, k, dt = c["T"], c["H"], c["k"], DT[c["dtype"]]
        ids = _dropped(g, _picks(_logits(g, T, c["E"], 0.5), k), c["drop"])
        offs, pair_row, row_pair = _sorted(ids, c["E"])
        s = dict(offs=offs, pair_row=pair_row, row_pair=row_pair, x=_normal(g, T, H).to(dt),
                 y=_normal(g, T * k, H).to(dt), w=torch.softmax(_normal(g, T, k), 1),
                 base=_normal(g, T, H).to(dt) if c["base"] else None)
        if c["grad"]:
            s.update(dxs=_normal(g, T * k, H).to(dt), dout=_normal(g, T, H).to(dt))
        return s
    if c["op"] == "quant":
        return dict(x=_activations(g, c["rows"], c["K"]).to(DT[c["dtype"]]))
    T, K, N, E, k = c["T"], c["K"], c["N"], c["E"], c["k"]
    offs, pair_row, row_pair = _sorted(_picks(_logits(g, T, E, c["skew"]), k), E)
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
    for e in range(E):
        codes[e], scales[e] = _pack(*_mx4(_normal(g, N, K) * 0.02))
    x = _activations(g, T if c["gather"] else T * k, K).to(DT[c["dtype"]])
    return dict(x=x, offs=offs, row_pair=row_pair if c["gather"] else None, codes=codes, scales=scales,
                bounds=offs.tolist())


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    s["case"] = c
    if not own:
        return s
    from bandwidth_bound_fp8_gb300 import moeq

    def out(shape, dt):
        return torch.empty(shape, dtype=dt, device="cuda")

    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        s.update(id_out=out((T, k), i32), w_out=out((T, k), f32), dl_out=out((T, E), f32) if c["grad"] else None)
    elif c["op"] == "sort":
        T, k = c["T"], c["k"]
        s.update(offs_out=out((c["E"] + 1,), i32), pair_row_out=out((T, k), i32), row_pair_out=out((T * k,), i32))
    elif c["op"] == "rows":
        T, H, k, dt = c["T"], c["H"], c["k"], DT[c["dtype"]]
        s.update(xs_out=out((T * k, H), dt), out_out=out((T, H), dt))
        if c["grad"]:
            s.update(dx_out=out((T, H), dt), dy_out=out((T * k, H), dt), dw_out=out((T, k), f32))
    elif c["op"] == "quant":
        s.update(q_out=out((c["rows"], c["K"] // 2), u8), v_out=out((c["rows"], c["K"]), torch.bfloat16),
                 s_out=out((c["rows"], moeq.moeq_mx4_scale_pitch(c["K"])), u8))
    else:
        # the weights are laid out once, as a server does when it loads them
        T, K, N, E, R = c["T"], c["K"], c["N"], c["E"], c["T"] * c["k"]
        s["w"], s["ws_w"] = moeq.mx4_weight_buffers(E, N, K)
        moeq.moeq_mx4_pack_weight(s.pop("codes"), s.pop("scales"), s["w"], s["ws_w"])
        s["y_out"] = out((R, N), DT[c["y"]])
        s["ws"] = moeq.Workspace(moeq.moeq_mx4_expert_gemm_workspace_size(s["x"].shape[0], K, N, E, R))
    return s


# ----------------------------------------------------------------- one pass
def _run_own(s):
    from bandwidth_bound_fp8_gb300 import moeq

    c = s["case"]
    if c["op"] == "route":
        moeq.moeq_route_rows(s["logits"], s["id_out"], s["w_out"])
        if not c["grad"]:
            return s["id_out"], s["w_out"]
        moeq.moeq_route_rows_grad(s["dw"], s["id_out"], s["w_out"], s["dl_out"])
        return s["id_out"], s["w_out"], s["dl_out"]
    if c["op"] == "sort":
        moeq.moeq_expert_sort(s["ids"], c["E"], s["offs_out"], s["pair_row_out"], s["row_pair_out"])
        return s["offs_out"], s["pair_row_out"], s["row_pair_out"]
    if c["op"] == "rows":
        moeq.moeq_gather_rows(s["x"], s["offs"], s["pair_row"], s["xs_out"])
        moeq.moeq_combine_rows(s["y"], s["pair_row"], s["w"], s["out_out"], base=s["base"])
        if not c["grad"]:
            return s["xs_out"], s["out_out"]
        moeq.moeq_gather_rows_grad(s["dxs"], s["pair_row"], s["dx_out"])
        moeq.moeq_combine_rows_grad(s["dout"], s["y"], s["offs"], s["pair_row"], s["w"], s["dy_out"], s["dw_out"])
        return s["xs_out"], s["out_out"], s["dx_out"], s["dy_out"], s["dw_out"]
    if c["op"] == "quant":
        moeq.moeq_mx4_quant_act(s["x"], s["q_out"], s["s_out"])
        moeq.moeq_mx4_dequant_act(s["q_out"], s["s_out"], s["v_out"])
        return s["v_out"]
    moeq.moeq_mx4_expert_gemm(s["x"], s["w"], s["ws_w"], s["offs"], s["y_out"], s["ws"], row_pair=s["row_pair"],
                              top_k=c["k"])
    return s["y_out"]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        lg, k = s["logits"], c["k"]
        v, i = torch.sort(lg, dim=1, descending=True, stable=True)
        v, i = v[:, :k], i[:, :k]
        live = v > -math.inf
        top = torch.where(live[:, :1], v[:, :1], torch.zeros_like(v[:, :1]))
        p = torch.where(live, torch.exp(v - top), torch.zeros_like(v))
        w = p / p.sum(1, keepdim=True).clamp(min=1e-30)
        ids = torch.where(live, i, torch.full_like(i, -1)).to(torch.int32)
        if not c["grad"]:
            return ids, w
        d = w * (s["dw"] - (w * s["dw"]).sum(1, keepdim=True))
        dl = torch.zeros_like(lg)
        dl.scatter_(1, i, torch.where(live, d, torch.zeros_like(d)))
        return ids, w, dl
    if c["op"] == "sort":
        return _sorted(s["ids"], c["E"])
    if c["op"] == "rows":
        T, H, k, dt = c["T"], c["H"], c["k"], DT[c["dtype"]]
        rp, pr, w = s["row_pair"].long(), s["pair_row"].long(), s["w"]
        kept, live = (rp >= 0).unsqueeze(1), (pr >= 0).unsqueeze(2)
        zero = torch.zeros((), dtype=torch.float32, device="cuda")
        tok = rp.clamp(min=0) // k
        xs = torch.where(kept, s["x"][tok].float(), zero).to(dt)
        yj = torch.where(live, s["y"][pr.clamp(min=0)].float(), zero)
        out = (yj * w.unsqueeze(2)).sum(1)
        if s["base"] is not None:
            out = out + s["base"].float()
        out = out.to(dt)
        if not c["grad"]:
            return xs, out
        dx = torch.where(live, s["dxs"][pr.clamp(min=0)].float(), zero).sum(1).to(dt)
        dout = s["dout"].float()
        dw = (yj * dout.unsqueeze(1)).sum(2)
        dy = torch.where(kept, dout[tok] * w.reshape(-1)[rp.clamp(min=0)].unsqueeze(1), zero).to(dt)
        return xs, out, dx, dy, dw
    if c["op"] == "quant":
        return _mx4_value(*_mx4(s["x"].float())).to(torch.bfloat16)
    x = _mx4_value(*_mx4(s["x"].float()))
    y = torch.empty((c["T"] * c["k"], c["N"]), dtype=DT[c["y"]], device="cuda")
    b = s["bounds"]
    for e in range(c["E"]):
        if b[e + 1] > b[e]:
            rows = x[b[e]:b[e + 1]] if s["row_pair"] is None else x[(s["row_pair"][b[e]:b[e + 1]] // c["k"]).long()]
            y[b[e]:b[e + 1]] = (rows @ _unpack(s["codes"][e], s["scales"][e]).t()).to(y.dtype)
    return y


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "route":
        b = c["T"] * (c["E"] * 4 + c["k"] * 8)
        return dict(bytes=b + (c["T"] * (c["k"] * 4 + c["E"] * 4) if c["grad"] else 0),
                    flops=c["T"] * c["E"] * (2 if c["grad"] else 1))
    if c["op"] == "sort":
        return dict(bytes=c["T"] * c["k"] * 12 + 4 * (c["E"] + 1), flops=c["T"] * c["k"])
    if c["op"] == "rows":
        T, k, row = c["T"], c["k"], c["H"] * SIZE[c["dtype"]]
        kept = T * k * (1 - c["drop"])
        b = T * row + T * k * row + kept * row + T * row * (2 if c["base"] else 1) + 12 * T * k
        f = 2 * kept * c["H"]
        if c["grad"]:
            b += kept * row + T * row + T * row + kept * row + T * k * row + 8 * T * k
            f += 4 * kept * c["H"]
        return dict(bytes=int(b), flops=int(f))
    if c["op"] == "quant":
        n = c["rows"] * c["K"]
        return dict(bytes=int(n * (SIZE[c["dtype"]] + 2 * 17 / 32 + 2)), flops=4 * n)
    T, K, N, E, R = c["T"], c["K"], c["N"], c["E"], c["T"] * c["k"]
    used = E * (1 - (1 - c["k"] / E) ** T) if E > 1 else 1
    rows = T if c["gather"] else R
    b = used * N * K * 17 / 32 + rows * K * SIZE[c["dtype"]] + R * N * SIZE[c["y"]]
    return dict(bytes=int(b), flops=2 * R * N * K)


# -------------------------------------------------------------------- exact
def _unit(s):
    """2^s in float64 for whole s, from its bits."""
    return ((s.long() + 1023) << 52).view(torch.float64)


def _exact_quant(x):
    """MXFP4 values of float64 [R, K], block by block from the definition: the nearest of the eight magnitudes, a tie
    going to the even place in their list."""
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    amax = b.abs().max(-1, keepdim=True).values
    # floor(log2 amax) from the binary64 exponent: a logarithm may fall short of a whole number
    s = (amax.view(torch.int64) >> 52) - 1023 - 2
    unit = _unit(torch.where(amax > 0, s, torch.full_like(s, -127)).clamp(min=-127))
    a = b.abs() / unit
    best = torch.zeros_like(a)
    for n, (lo, hi) in enumerate(zip(E2M1[:-1], E2M1[1:])):
        mid = (lo + hi) / 2
        up = a > mid if n % 2 == 0 else a >= mid
        best = torch.where(up, torch.full_like(a, hi), best)
    return (torch.where(b < 0, -best, best) * unit).reshape(R, K)


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    f64 = torch.float64
    if c["op"] == "route":
        lg = s["logits"].double().cpu().numpy()
        T, E, k = c["T"], c["E"], c["k"]
        order = np.argsort(-lg, axis=1, kind="stable")[:, :k]
        ids = np.full((T, k), -1, np.int32)
        w, dl = np.zeros((T, k)), np.zeros((T, E))
        dw = s["dw"].double().cpu().numpy()
        for t in range(T):
            n = int(np.isfinite(lg[t, order[t]]).sum())
            if not n:
                continue
            e = order[t, :n]
            p = np.exp(lg[t, e] - lg[t, e[0]])
            p /= p.sum()
            ids[t, :n], w[t, :n] = e, p
            dl[t, e] = p * (dw[t, :n] - np.dot(p, dw[t, :n]))
        res = (torch.from_numpy(ids), torch.from_numpy(w), torch.from_numpy(dl))
        return res if c["grad"] else res[:2]
    if c["op"] == "sort":
        return None
    if c["op"] == "rows":
        T, H, k = c["T"], c["H"], c["k"]
        pr, w = s["pair_row"].long(), s["w"].double()
        xs = torch.zeros((T * k, H), dtype=f64, device="cuda")
        out = s["base"].double() if c["base"] else torch.zeros((T, H), dtype=f64, device="cuda")
        dx, dy, dw = torch.zeros_like(out), torch.zeros_like(xs), torch.zeros((T, k), dtype=f64, device="cuda")
        for j in range(k):
            t = torch.nonzero(pr[:, j] >= 0).flatten()
            r = pr[t, j]
            xs[r] = s["x"][t].double()
            out[t] += w[t, j, None] * s["y"][r].double()
            if c["grad"]:
                d = s["dout"][t].double()
                dx[t] += s["dxs"][r].double()
                dy[r] = w[t, j, None] * d
                dw[t, j] = (d * s["y"][r].double()).sum(1)
        return (xs, out, dx, dy, dw) if c["grad"] else (xs, out)
    if c["op"] == "quant":
        return _exact_quant(s["x"].double())
    T, K, N, E, k = c["T"], c["K"], c["N"], c["E"], c["k"]
    if T * k * K * N > 1e13:
        return None
    x = _exact_quant(s["x"].double())
    y = torch.zeros((T * k, N), dtype=f64, device="cuda")
    table = torch.tensor([v * sg for sg in (1, -1) for v in E2M1], dtype=f64, device="cuda")
    for e in range(E):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo == hi:
            continue
        w = torch.empty((N, K), dtype=f64, device="cuda")
        w[:, 0::2] = table[(s["codes"][e] % 16).long()]
        w[:, 1::2] = table[(s["codes"][e] // 16).long()]
        w *= _unit(s["scales"][e].long() - 127).repeat_interleave(32, dim=1)
        rows = x[lo:hi] if s["row_pair"] is None else x[torch.div(s["row_pair"][lo:hi], k, rounding_mode="floor").long()]
        y[lo:hi] = rows @ w.t()
    return y
