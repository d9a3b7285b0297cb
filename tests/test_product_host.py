"""Host-side refusals of the experts' bf16 products and of activations kept in
8 bits (no GPU): bad arguments are rejected before a device is asked for."""
import ctypes
import re

import pytest

from test_chained_loads_host import _bodies, _source

INVALID, SHAPE = 1, 2


@pytest.fixture(scope="module")
def lib():
    from bandwidth_bound_fp8_gb300 import build, moeq
    build.build()
    return moeq.load()


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(1 << 16)
    yield (ctypes.addressof(buf) + 255) // 256 * 256


@pytest.mark.parametrize("name,xw,yw", [("moeq_expert_product", "K", "N"), ("moeq_expert_product_grad_x", "N", "K")])
def test_product_refusals(lib, p, name, xw, yw):
    f = getattr(lib, name)
    ok = dict(x=p, ld=64, w=p, K=64, N=64, offs=p, E=2, R=4, y=p, yt=0, ldy=64, status=None, st=None)
    call = lambda **kw: f(*{**ok, **kw}.values())
    assert call(K=60) == SHAPE and call(N=4) == SHAPE and call(N=0) == SHAPE and call(K=(1 << 20) + 8) == SHAPE
    assert call(E=0) == INVALID and call(E=1025) == INVALID and call(R=-1) == INVALID and call(R=(1 << 30) + 1) == INVALID
    assert call(yt=2) == INVALID and call(yt=-1) == INVALID
    assert call(x=None) == INVALID and call(x=p + 8) == INVALID and call(ld=68) == INVALID and call(ld=56) == INVALID
    assert call(w=None) == INVALID and call(w=p + 2) == INVALID and call(offs=None) == INVALID and call(offs=p + 1) == INVALID
    assert call(y=None) == INVALID and call(y=p + 1) == INVALID and call(ldy=63) == INVALID
    assert call(y=p + 2, yt=1) == INVALID and call(status=p + 2) == INVALID
    assert call(R=0, x=None, y=None) == 0
    # the two widths are those of the right matrices
    assert call(**{xw: 72}) == INVALID and call(**{yw: 72}) == INVALID


def test_weight_gradient_refusals(lib, p):
    f = lib.moeq_expert_product_grad_w
    ok = dict(dy=p, ldy=64, x=p, ldx=64, K=64, N=64, offs=p, E=2, R=4, dw=p, dt=0, status=None, st=None)
    call = lambda **kw: f(*{**ok, **kw}.values())
    assert call(K=60) == SHAPE and call(N=4) == SHAPE
    assert call(E=0) == INVALID and call(E=1025) == INVALID and call(R=-1) == INVALID and call(dt=2) == INVALID
    assert call(dy=p + 8) == INVALID and call(x=None) == INVALID and call(ldy=60) == INVALID and call(ldx=68) == INVALID
    assert call(dw=p + 8) == INVALID and call(dw=None) == INVALID and call(offs=None) == INVALID
    assert call(R=0, dw=None) == INVALID           # it is zeroed even without rows
    assert call(status=p + 1) == INVALID


def test_keep_refusals(lib, p):
    q, dq, g = lib.moeq_fp8_quant_rows, lib.moeq_fp8_dequant_rows, lib.moeq_fp8_gather_rows
    assert q(p, 0, 64, 1, 0, p, p, None) == SHAPE and q(p, 0, 1 << 21, 1, 1 << 21, p, p, None) == SHAPE
    assert q(p, 2, 64, 1, 64, p, p, None) == INVALID and q(p, 0, 63, 1, 64, p, p, None) == INVALID
    assert q(None, 0, 64, 1, 64, p, p, None) == INVALID and q(p + 1, 0, 64, 1, 64, p, p, None) == INVALID
    assert q(p, 0, 64, 1, 64, p + 8, p, None) == INVALID and q(p, 0, 64, 1, 64, p, p + 2, None) == INVALID
    assert q(p, 0, 64, -1, 64, p, p, None) == INVALID and q(None, 0, 64, 0, 64, None, None, None) == 0
    assert dq(p, p, 1, 64, p, 0, 63, None) == INVALID and dq(p, None, 1, 64, p, 0, 64, None) == INVALID
    assert dq(p, p, 1, 0, p, 0, 64, None) == SHAPE and dq(None, None, 0, 64, None, 0, 64, None) == 0
    assert g(p, p, 1, 64, 2, p, 8, p, None, 0, 64, None) == INVALID and g(p, p, 1, 64, 2, None, 8, p, p, 0, 64, None) == INVALID
    assert g(p, p, 1, 64, 17, p, 8, p, p, 0, 64, None) == INVALID and g(p, p, 1, 0, 2, p, 8, p, p, 0, 64, None) == SHAPE
    assert g(p, p, 1, 64, 2, p, 8, p + 2, p, 0, 64, None) == INVALID and g(p, p, 1, 64, 2, p, 8, p, p, 3, 64, None) == INVALID


def test_swiglu_refusals(lib, p):
    ok = dict(gu=p, dt=0, ld=128, R=4, I=64, rp=p, w=p, h=p, ldh=64, codes=p, scales=p, st=None)
    call = lambda **kw: lib.moeq_swiglu_rows(*{**ok, **kw}.values())
    assert call(I=0) == SHAPE and call(I=1 << 21) == SHAPE
    assert call(dt=2) == INVALID and call(R=-1) == INVALID and call(ld=127) == INVALID and call(ldh=63) == INVALID
    assert call(codes=None) == INVALID and call(scales=None) == INVALID and call(codes=p + 8) == INVALID
    assert call(rp=None) == INVALID                # weights go by the rows' pairs
    assert call(rp=p + 2) == INVALID and call(w=p + 1) == INVALID and call(gu=None) == INVALID and call(h=p + 1) == INVALID
    assert call(R=0, gu=None, h=None) == 0
    ok = dict(dh=p, dt=0, ld=64, codes=p, scales=p, R=4, I=64, rp=p, w=p, pr=p, dgu=p, ldg=128, h=p, ldh=64, dw=p, st=None)
    grad = lambda **kw: lib.moeq_swiglu_rows_grad(*{**ok, **kw}.values())
    assert grad(I=0) == SHAPE
    assert grad(dt=5) == INVALID and grad(R=-1) == INVALID and grad(ld=63) == INVALID and grad(ldg=127) == INVALID
    assert grad(codes=None) == INVALID and grad(scales=None) == INVALID and grad(ldh=63) == INVALID
    assert grad(w=None) == INVALID and grad(pr=None) == INVALID and grad(rp=None) == INVALID
    assert grad(dw=p + 2) == INVALID and grad(pr=p + 1) == INVALID
    assert grad(R=0, dh=None, dgu=None, h=None) == 0


torch = pytest.importorskip("torch")
U8, BF, I32 = torch.uint8, torch.bfloat16, torch.int32


def _calls(dev):
    """Every call with fitting shapes on `dev`."""
    from bandwidth_bound_fp8_gb300 import moeq
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=dev)
    T, k, E, K, N, R = 4, 2, 3, 64, 16, 8
    offs, pr, rp, w3 = z(E + 1, dt=I32), z(T, k, dt=I32), z(R, dt=I32), z(E, N, K, dt=BF)
    x, dy = z(R, K, dt=BF), z(R, N, dt=BF)
    c, s, c2, s2 = z(R, K, dt=U8), z(R, 1), z(R, 2 * K, dt=U8), z(R, 2)
    return {
        "product": lambda **kw: moeq.moeq_expert_product(*{**dict(x=x, w=w3, offs=offs, y=z(R, N)), **kw}.values(), stream=0),
        "grad_x": lambda **kw: moeq.moeq_expert_product_grad_x(*{**dict(dy=dy, w=w3, offs=offs, dx=z(R, K)), **kw}.values(),
                                                               stream=0),
        "grad_w": lambda **kw: moeq.moeq_expert_product_grad_w(*{**dict(dy=dy, x=x, offs=offs, dw=z(E, N, K)), **kw}.values(),
                                                               stream=0),
        "quant": lambda **kw: moeq.moeq_fp8_quant_rows(*{**dict(x=x, codes=c, scales=s), **kw}.values(), stream=0),
        "dequant": lambda **kw: moeq.moeq_fp8_dequant_rows(*{**dict(codes=c, scales=s, out=x), **kw}.values(), stream=0),
        "gather": lambda **kw: moeq.moeq_fp8_gather_rows(
            *{**dict(codes=c[:T], scales=s[:T], offs=offs, pair_row=pr, xs=x), **kw}.values(), stream=0),
        "swiglu": lambda **kw: moeq.moeq_swiglu_rows(
            **{**dict(gu=z(R, 2 * K), h=z(R, K), row_pair=rp, topk_w=z(T, k), codes=c2, scales=s2), **kw}, stream=0),
        "swiglu_grad": lambda **kw: moeq.moeq_swiglu_rows_grad(
            **{**dict(d_h=z(R, K), codes=c2, scales=s2, d_gu=z(R, 2 * K), h=z(R, K), row_pair=rp, topk_w=z(T, k), pair_row=pr,
                      d_topk_w=z(T, k)), **kw}, stream=0),
    }


@pytest.mark.parametrize("dev", ["cpu", "meta"])
@pytest.mark.parametrize("name", ["product", "grad_x", "grad_w", "quant", "dequant", "gather", "swiglu", "swiglu_grad"])
def test_tensors_elsewhere_are_refused(name, dev):
    with pytest.raises(ValueError, match="on the current CUDA device"):
        _calls(dev)[name]()


def test_binding_refuses_other_shapes_and_types():
    from bandwidth_bound_fp8_gb300 import moeq
    calls = _calls("cpu")
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    with pytest.raises(ValueError, match="bf16 rows"):
        calls["product"](x=z(8, 64))
    with pytest.raises(ValueError, match="bf16 rows"):
        calls["product"](x=z(7, 64, dt=BF))
    with pytest.raises(ValueError, match="bf16 rows"):
        calls["grad_x"](dy=z(8, 16, dt=torch.float16))
    with pytest.raises(ValueError, match="bf16 rows"):
        calls["grad_w"](dy=z(8, 16))
    with pytest.raises(ValueError, match="codes and scales"):
        calls["swiglu"](codes=None)
    with pytest.raises(ValueError, match="gu"):
        calls["swiglu"](gu=z(8, 127))
    with pytest.raises(ValueError, match="gu"):
        calls["swiglu"](gu=z(8, 128, dt=BF))
    with pytest.raises(ValueError, match="d_gu"):
        calls["swiglu_grad"](d_gu=z(8, 64))
    with pytest.raises(ValueError, match="h:"):
        calls["swiglu_grad"](h=z(8, 64, dt=BF))
    with pytest.raises(ValueError, match="d_topk_w"):
        calls["swiglu_grad"](pair_row=None)
    with pytest.raises(ValueError, match="d_topk_w"):
        calls["swiglu_grad"](topk_w=None)
    assert [moeq.fp8_groups(K) for K in (1, 128, 129, 6144)] == [1, 1, 2, 48]


@pytest.mark.parametrize("name", ["moeq_keep.cu", "moeq_product.cu"])
def test_chained_kernels_read_with_plain_loads(name):
    """As in test_chained_loads_host: they are resident while their inputs are written."""
    kernels = 0
    for body in _bodies(_source(name)):
        kernel = re.search(r"__global__\s.*?\b(\w+_kernel)\(", body, re.S)
        assert "__ldg" not in body
        if kernel:
            kernels += 1
            assert "chain();" in body or "set_up<" in body
            assert not re.search(r"const\s+[\w]+\s*\*\s*__restrict__", body.split("{")[0]), kernel.group(1)
    assert kernels
    assert "chain();" in _source("moeq_product.cu")
