"""Host-side refusals of the operators on any number of tokens (no GPU): bad
arguments are rejected before a device is asked for, and the sizes."""
import ctypes

import pytest

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


def test_sizes(lib):
    assert lib.moeq_mx4_scale_pitch(6144) == 192 and lib.moeq_mx4_scale_pitch(32) == 8
    assert lib.moeq_mx4_scale_pitch(288) == 16
    assert lib.moeq_mx4_scale_pitch(0) == lib.moeq_mx4_scale_pitch(40) == lib.moeq_mx4_scale_pitch(65536) == 0
    assert lib.moeq_mx4_weight_bytes(256, 4096, 6144) == 256 * 4096 * 6144 // 2
    assert lib.moeq_mx4_weight_scale_bytes(256, 4096, 6144) == 256 * 4096 * 6144 // 32
    assert lib.moeq_mx4_weight_bytes(1, 1, 32) == 16384 and lib.moeq_mx4_weight_scale_bytes(1, 129, 288) == 4096
    assert lib.moeq_mx4_weight_bytes(0, 128, 256) == lib.moeq_mx4_weight_bytes(1, 0, 256) == 0
    assert lib.moeq_mx4_weight_bytes(1, 128, 100) == 0


def test_routing_refusals(lib, p):
    route = lib.moeq_route_rows
    assert route(None, 8, 1, 8, 2, p, p, None) == INVALID
    assert route(p + 2, 8, 1, 8, 2, p, p, None) == INVALID
    assert route(p, 7, 1, 8, 2, p, p, None) == INVALID        # rows overlap
    assert route(p, 8, 1, 8, 9, p, p, None) == INVALID        # more picks than experts
    assert route(p, 2000, 1, 2000, 2, p, p, None) == INVALID  # too many experts
    assert route(p, 32, 1, 32, 17, p, p, None) == INVALID     # too many picks
    assert route(p, 8, -1, 8, 2, p, p, None) == INVALID
    assert route(p, 8, 1 << 29, 8, 8, p, p, None) == INVALID  # 2^32 pairs
    assert route(None, 8, 0, 8, 2, None, None, None) == 0     # no tokens
    grad = lib.moeq_route_rows_grad
    assert grad(p, None, p, 1, 8, 2, p, 8, None) == INVALID
    assert grad(p, p, p, 1, 8, 2, p, 7, None) == INVALID
    sort = lib.moeq_expert_sort
    assert sort(p, 1, 2, 0, p, p, p, None) == INVALID
    assert sort(p, 1, 0, 8, p, p, p, None) == INVALID
    assert sort(p, 1, 2, 8, None, p, p, None) == INVALID
    assert sort(p, 1, 2, 8, p, p, None, None) == INVALID
    assert sort(p + 1, 1, 2, 8, p, p, p, None) == INVALID


def test_movement_refusals(lib, p):
    g = lib.moeq_gather_rows
    assert g(p, 0, 64, 1, 64, 2, p, 8, p, None, 64, None) == INVALID
    assert g(p, 2, 64, 1, 64, 2, p, 8, p, p, 64, None) == INVALID      # MXFP4 is no row type
    assert g(p, 0, 63, 1, 64, 2, p, 8, p, p, 64, None) == INVALID
    assert g(p, 0, 64, 1, 64, 2, p, 8, p, p, 63, None) == INVALID
    assert g(p + 1, 0, 64, 1, 64, 2, p, 8, p, p, 64, None) == INVALID
    assert g(p, 0, 64, 1, 0, 2, p, 8, p, p, 64, None) == SHAPE
    c = lib.moeq_combine_rows
    assert c(p, 0, 64, 1, 64, 2, p, None, None, 0, p, 0, 64, None) == INVALID
    assert c(p, 0, 64, 1, 64, 2, p, p, p, 32, p, 0, 64, None) == INVALID  # base's rows overlap
    assert c(p, 0, 64, 1, 64, 2, p, p, None, 0, p, 5, 64, None) == INVALID
    assert c(p, 0, 64, 1, 1 << 21, 2, p, p, None, 0, p, 0, 64, None) == SHAPE
    gg = lib.moeq_gather_rows_grad
    assert gg(p, 0, 64, 1, 64, 2, None, p, 64, None) == INVALID
    cg = lib.moeq_combine_rows_grad
    assert cg(p, 0, 64, p, 0, 64, 1, 64, 2, p, 8, p, p, p, 64, None, None) == INVALID
    assert cg(p, 0, 64, p, 0, 64, 1, 64, 2, None, 8, p, p, p, 64, p, None) == INVALID


def test_mx4_refusals(lib, p):
    q = lib.moeq_mx4_quant_act
    assert q(p, 0, 64, 1, 48, 0, p, p, None) == SHAPE
    assert q(p, 0, 64, 1, 64, 2, p, p, None) == INVALID        # no such activation
    assert q(p, 0, 64, 1, 64, 1, p, p, None) == INVALID        # a SwiGLU row has 2K elements
    assert q(p, 0, 64, 1, 64, 0, p + 8, p, None) == INVALID
    assert q(p, 0, 64, -1, 64, 0, p, p, None) == INVALID
    assert q(None, 0, 64, 0, 64, 0, None, None, None) == 0
    assert lib.moeq_mx4_dequant_act(p, None, 1, 64, p, 0, 64, None) == INVALID
    assert lib.moeq_mx4_quant_weight(p, 0, 0, 128, 64, p, p, None) == INVALID
    assert lib.moeq_mx4_quant_weight(p, 0, 1, 128, 65, p, p, None) == SHAPE
    assert lib.moeq_mx4_pack_weight(p, p, 1, 0, 64, p, p, None) == SHAPE
    gemm = lib.moeq_mx4_expert_gemm
    ok = dict(x=p, xt=0, ld=64, xs=None, rows=4, K=64, act=0, w=p, sw=p, N=16, offs=p, E=2, R=4, rp=None, k=1, y=p, yt=0,
              ldy=16, ws=p, wsb=0, st=None)
    call = lambda **kw: gemm(*{**ok, **kw}.values())
    assert call(R=5) == INVALID                       # more rows than activations, and no index
    assert call(R=5, rows=0, rp=p) == INVALID         # nothing to read
    assert call(K=48) == SHAPE and call(N=0) == SHAPE
    assert call(E=0) == INVALID and call(E=1025) == INVALID and call(k=0) == INVALID
    assert call(yt=2) == INVALID and call(xt=3) == INVALID and call(act=7) == INVALID
    assert call(xt=2) == INVALID and call(xs=p) == INVALID     # codes and their scales come together
    assert call(xt=2, xs=p, act=1) == INVALID
    assert call(ldy=15) == INVALID and call(ld=63) == INVALID and call(w=None) == INVALID and call(offs=p + 2) == INVALID
    assert call(R=0, y=None) == 0
    assert lib.moeq_mx4_expert_gemm_workspace_size(4, 48, 16, 2, 4) == 0


def test_binding_refuses_other_shapes_and_strides():
    torch = pytest.importorskip("torch")
    from bandwidth_bound_fp8_gb300 import moeq
    i32 = torch.int32
    with pytest.raises(ValueError):
        moeq.moeq_route_rows(torch.zeros(4, 8).t(), torch.zeros((8, 2), dtype=i32), torch.zeros(8, 2), stream=0)
    with pytest.raises(ValueError):
        moeq.moeq_route_rows(torch.zeros(4, 8), torch.zeros((3, 2), dtype=i32), torch.zeros(4, 2), stream=0)
    with pytest.raises(ValueError):
        moeq.moeq_gather_rows(torch.zeros(4, 8), torch.zeros(3, dtype=i32), torch.zeros((4, 2), dtype=i32),
                              torch.zeros(7, 8), stream=0)
    with pytest.raises(TypeError):
        moeq.moeq_mx4_quant_act(torch.zeros((4, 64), dtype=torch.float16), torch.zeros((4, 32), dtype=torch.uint8),
                                torch.zeros((4, 8), dtype=torch.uint8), stream=0)
