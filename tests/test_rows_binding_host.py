"""The binding's refusals for the operators on any number of tokens: what
would reach a kernel as a wrong pointer or a wrong width raises."""
import pytest

torch = pytest.importorskip("torch")

from bandwidth_bound_fp8_gb300 import moeq  # noqa: E402

I32, U8 = torch.int32, torch.uint8


def _calls(dev):
    """Every call with fitting shapes on `dev`."""
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=dev)
    T, k, E, H, K, N = 4, 2, 3, 8, 64, 16
    ids, w, offs = z(T, k, dt=I32), z(T, k), z(E + 1, dt=I32)
    tiles, stiles = z(E * 16384, dt=U8), z(E * 1024, dt=U8)
    ws = type("Ws", (), dict(ptr=0, nbytes=0))()
    return {
        "route_rows": lambda: moeq.moeq_route_rows(z(T, E), ids, w, stream=0),
        "route_rows_grad": lambda: moeq.moeq_route_rows_grad(w, ids, w, z(T, E), stream=0),
        "expert_sort": lambda: moeq.moeq_expert_sort(ids, E, offs, ids, z(T * k, dt=I32), stream=0),
        "gather_rows": lambda: moeq.moeq_gather_rows(z(T, H), offs, ids, z(T * k, H), stream=0),
        "gather_rows_grad": lambda: moeq.moeq_gather_rows_grad(z(T * k, H), ids, z(T, H), stream=0),
        "combine_rows": lambda: moeq.moeq_combine_rows(z(T * k, H), ids, w, z(T, H), stream=0),
        "combine_rows_base": lambda: moeq.moeq_combine_rows(z(T * k, H), ids, w, z(T, H), base=z(T, H), stream=0),
        "combine_rows_grad": lambda: moeq.moeq_combine_rows_grad(z(T, H), z(T * k, H), offs, ids, w, z(T * k, H),
                                                                 z(T, k), stream=0),
        "quant_act": lambda: moeq.moeq_mx4_quant_act(z(T, K), z(T, K // 2, dt=U8), z(T, 8, dt=U8), stream=0),
        "dequant_act": lambda: moeq.moeq_mx4_dequant_act(z(T, K // 2, dt=U8), z(T, 8, dt=U8), z(T, K), stream=0),
        "quant_weight": lambda: moeq.moeq_mx4_quant_weight(z(E, N, K), tiles, stiles, stream=0),
        "pack_weight": lambda: moeq.moeq_mx4_pack_weight(z(E, N, K // 2, dt=U8), z(E, N, K // 32, dt=U8), tiles, stiles,
                                                         stream=0),
        "expert_gemm": lambda: moeq.moeq_mx4_expert_gemm(z(T, K), tiles, stiles, offs, z(T, N), ws, stream=0),
        "expert_gemm_codes": lambda: moeq.moeq_mx4_expert_gemm(z(T, K // 2, dt=U8), tiles, stiles, offs, z(T, N), ws,
                                                               x_scales=z(T, 8, dt=U8), stream=0),
    }


@pytest.mark.parametrize("dev", ["cpu", "meta"])
@pytest.mark.parametrize("name", sorted(_calls("meta")))
def test_tensors_elsewhere_are_refused(name, dev):
    """A host address in a kernel is a fault of the GPU.  (Here, without one, the library's own answer would be a
    MoeqError after the pointer checks.)"""
    with pytest.raises(ValueError, match="on the current CUDA device"):
        _calls(dev)[name]()


def test_swiglu_rows_have_two_halves():
    """65 columns were read as a gate of 32 and an up of 32."""
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    with pytest.raises(ValueError, match="gate and up"):
        moeq.moeq_mx4_quant_act(z(4, 65), z(4, 16, dt=U8), z(4, 8, dt=U8), act=moeq.MOEQ_ACT_SWIGLU, stream=0)
    with pytest.raises(ValueError, match="gate and up"):
        moeq.moeq_mx4_expert_gemm(z(4, 65), z(16384, dt=U8), z(1024, dt=U8), z(2, dt=I32), z(4, 16),
                                  type("Ws", (), dict(ptr=0, nbytes=0))(), act=moeq.MOEQ_ACT_SWIGLU, stream=0)
