"""fp64 oracle of the paged KV cache: the norms and the rotation of new rows, where they go, and attention over a
sequence's rows with a causal end, a window and a few first rows that stay visible.  Plain loops over sequences,
heads and rows; nothing is blocked or fused."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot: int, theta: float, scaling: str = "none", factor: float = 1.0, original: int = 0, low: float = 1.0,
                high: float = 32.0) -> np.ndarray:
    """The angle a position of each pair."""
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "parts":
        r = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        return f * (r + (1.0 - r) / factor)
    return f


def norm_rotate(x: np.ndarray, weight, eps: float, pos: np.ndarray, freq: np.ndarray, half: bool, gain: float = 1.0):
    """x [n, heads, hd] -> (y, reach): y in 64 bits, reach the sum of magnitudes that an entry of y was formed from."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out, reach, rot = y.copy(), np.abs(y), 2 * len(freq)
    for i, f in enumerate(freq):
        a, b = (i, i + rot // 2) if half else (2 * i, 2 * i + 1)
        c, s = gain * np.cos(pos * f)[:, None], gain * np.sin(pos * f)[:, None]
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
        reach[..., a] = reach[..., b] = gain * (np.abs(y[..., a]) + np.abs(y[..., b]))
    return out, reach


def seen(pos: int, length: int, causal: bool = True, window: int = 0, sinks: int = 0) -> np.ndarray:
    """Which of a sequence's rows the row at `pos` sees."""
    return np.array([(not causal or j <= pos) and (not window or j > pos - window or j < sinks) for j in range(length)], bool)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool = True, window: int = 0, sinks: int = 0):
    """q [n, H, hd], the last n of a sequence's rows k, v [L, Hkv, hd] -> (out [n, H, hd], mass [n, H, hd]: sum_j p_j |v_j|,
    reach [n, H]: the largest scale * sum_d |q_d k_jd| seen)."""
    n, H, hd = q.shape
    L, hkv = k.shape[0], k.shape[1]
    out, mass, reach = np.zeros((n, H, hd)), np.zeros((n, H, hd)), np.zeros((n, H))
    for t in range(n):
        m = seen(L - n + t, L, causal, window, sinks)
        if not m.any():
            continue
        for h in range(H):
            kk, vv = k[m, h // (H // hkv)], v[m, h // (H // hkv)]
            s = kk @ q[t, h] * scale
            reach[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h] = p @ vv
            mass[t, h] = p @ np.abs(vv)
    return out, mass, reach
