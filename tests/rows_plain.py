"""Plain 64-bit forms of the operators on any number of tokens, for the
tests: numpy (routing, sort, row movement) and the MXFP4 codec from its
definition, element by element against the table of E2M1 magnitudes."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
U24, U8 = 2.0 ** -24, 2.0 ** -8   # half an ulp, relative, of fp32 (24 significant bits) and of bf16 (8)
TINY = 2.0 ** -126


def to64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def type_half_ulp(dtype) -> float:
    return U8 if dtype == torch.bfloat16 else U24


# ------------------------------------------------------------------ routing
def route(logits64: np.ndarray, k: int):
    """ids and weights of every row; NaN and -inf never picked, +inf as the largest fp32."""
    T, E = logits64.shape
    big = float(np.finfo(np.float32).max)
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        row = np.minimum(logits64[t], big)
        live = [e for e in range(E) if row[e] > -np.inf]
        pick = sorted(live, key=lambda e: (-row[e], e))[:k]
        if pick:
            p = np.exp(row[pick] - row[pick[0]])
            ids[t, :len(pick)] = pick
            w[t, :len(pick)] = p / p.sum()
    return ids, w


def sort_pairs(ids: np.ndarray, E: int):
    T, k = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    kept = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            kept[e].append(p)
    offs = np.concatenate([[0], np.cumsum([len(v) for v in kept])]).astype(np.int32)
    row_pair = np.full(T * k, -1, np.int32)
    order = np.concatenate([np.array(v, np.int64) for v in kept]) if T * k else np.zeros(0, np.int64)
    row_pair[:len(order)] = order
    pair_row = np.full(T * k, -1, np.int32)
    pair_row[order] = np.arange(len(order))
    return offs, pair_row.reshape(T, k), row_pair


# -------------------------------------------------------------------- MXFP4
def mx4_codes(x: np.ndarray):
    """x [R, K] (fp32 values) -> code nibbles [R, K] and scale bytes [R, K/32], from the definition in 64 bits."""
    R, K = x.shape
    b = np.asarray(x, np.float64).reshape(R, K // 32, 32)
    with np.errstate(invalid="ignore"):
        bad = ~np.isfinite(b).all(-1)
        amax = np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)
    s = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)
    s = np.maximum(s, -127)
    a = np.abs(np.where(bad[..., None], 0.0, b)) * np.exp2(-s.astype(np.float64))[..., None]
    code = np.zeros(a.shape, np.uint8)
    for n in range(7):
        mid = (E2M1[n] + E2M1[n + 1]) / 2
        code = np.where(a > mid if n % 2 == 0 else a >= mid, n + 1, code)
    code = code | (np.signbit(b).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    return code.reshape(R, K), np.where(bad, 255, s + 127).astype(np.uint8)


def mx4_values(code: np.ndarray, scale: np.ndarray) -> np.ndarray:
    R, K = code.shape
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    v = v.reshape(R, K // 32, 32) * np.exp2(scale.astype(np.float64) - 127)[..., None]
    return np.where(scale[..., None] == 255, np.nan, v).reshape(R, K)


def pack_codes(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def pad_scales(scale: np.ndarray, pitch: int) -> np.ndarray:
    out = np.zeros((scale.shape[0], pitch), np.uint8)
    out[:, :scale.shape[1]] = scale
    return out


def tiles(codes: np.ndarray, scales: np.ndarray):
    """Row-major packed codes [E, N, K/2] and scales [E, N, K/32] -> the tile-major layout, byte by byte."""
    E, N, KB = codes.shape
    nb, kb = (N + 127) // 128, (KB * 2 + 255) // 256
    c = np.zeros((E, nb * 128, kb * 128), np.uint8)
    c[:, :N, :KB] = codes
    s = np.zeros((E, nb * 128, kb * 8), np.uint8)
    s[:, :N, :scales.shape[2]] = scales
    out = np.zeros((E, nb, kb, 128, 8, 16), np.uint8)
    c = c.reshape(E, nb, 128, kb, 8, 16)
    for r in range(128):
        for ch in range(8):
            out[:, :, :, r, ch ^ (r % 8)] = c[:, :, r, :, ch]
    so = np.zeros((E, nb, kb, 2, 32, 4, 4), np.uint8)
    s = s.reshape(E, nb, 128, kb, 2, 4)
    for r in range(128):
        so[:, :, :, :, r % 32, r // 32] = s[:, :, r]
    return out.reshape(-1), so.reshape(-1)
