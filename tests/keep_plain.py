"""The 8-bit format of kept activations from its definition, in numpy: groups
of 128 columns (the last shorter), s = fl32(amax / 448), the E4M3 code of
fl32(x / s) rounded to nearest even, a value fl32(code * s)."""
from __future__ import annotations

import numpy as np
import torch

# the magnitudes of codes 0 .. 126 (127 is NaN)
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def keep(x: np.ndarray):
    """fp32 [R, K] -> codes uint8 [R, K], scales fp32 [R, G]."""
    R, K = x.shape
    G = (K + 127) // 128
    codes, scales = np.zeros((R, K), np.uint8), np.zeros((R, G), np.float32)
    mids = (E4M3[:-1] + E4M3[1:]) / 2
    for g in range(G):
        b = x[:, g * 128:(g + 1) * 128].astype(np.float32)
        bad = ~np.isfinite(b).all(1)
        b = np.where(bad[:, None], np.float32(0), b)
        s = (np.abs(b).max(1) / np.float32(448)).astype(np.float32)
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(s[:, None] > 0, b / s[:, None], np.float32(0)).astype(np.float64)
        a = np.abs(q)
        # the code is the number of midpoints below, and one more for a tie whose lower code is odd
        lo = np.searchsorted(mids, a, side="left")
        tie = (lo < len(mids)) & (a == mids[np.minimum(lo, len(mids) - 1)]) & (lo % 2 == 1)
        c = np.minimum(lo + tie, 126).astype(np.uint8) | (np.signbit(b).astype(np.uint8) << 7)
        codes[:, g * 128:(g + 1) * 128] = np.where(bad[:, None], 0, c)
        scales[:, g] = np.where(bad, np.float32(np.nan), s)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp32 [R, K]."""
    K = codes.shape[1]
    v = (E4M3[codes & 127] * np.where(codes & 128, -1.0, 1.0)).astype(np.float32)
    with np.errstate(over="ignore"):
        return v * np.repeat(scales, 128, axis=1)[:, :K]


def keep_gate_up(gu: np.ndarray):
    I = gu.shape[1] // 2
    (a, s), (b, t) = keep(gu[:, :I]), keep(gu[:, I:])
    return np.concatenate((a, b), 1), np.concatenate((s, t), 1)


def values_gate_up(codes: np.ndarray, scales: np.ndarray):
    I, G = codes.shape[1] // 2, scales.shape[1] // 2
    return values(codes[:, :I], scales[:, :G]), values(codes[:, I:], scales[:, G:])


def swiglu(gate, up, w):
    """h [R, I] in 64 bits; w [R]."""
    with np.errstate(over="ignore"):
        return w[:, None] * gate / (1 + np.exp(-gate)) * up


def swiglu_grad(dh, gate, up, w):
    """d_gate, d_up, h and <dh, h / w> of 64-bit rows."""
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-gate))
    act = gate * sig
    wd = w[:, None] * dh
    return wd * up * sig * (1 + gate * (1 - sig)), wd * act, w[:, None] * act * up, (dh * act * up).sum(1)


def to_np(t: torch.Tensor) -> np.ndarray:
    return t.detach().float().cpu().numpy()
