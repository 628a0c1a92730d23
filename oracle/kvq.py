"""fp64 oracle of the 4-bit KV cache: the storage rule, attention over the
stored rows with the weight that each row collects, and eviction by it.  Plain
loops over sequences, heads and rows; nothing is blocked or fused."""
from __future__ import annotations

import numpy as np

GROUP = 32
F16_MAX = 65504.0


def quantize(x: np.ndarray):
    """(codes 0..15, f16 scales) of groups of 32 along the last axis.  NaN counts as 0."""
    g = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf)
    g = g.reshape(g.shape[:-1] + (g.shape[-1] // GROUP, GROUP))
    hi, lo = g.max(-1), g.min(-1)
    m = np.where(hi > -lo, hi, lo)
    d = np.clip(m / -8.0, -F16_MAX, F16_MAX).astype(np.float16)
    dd = d.astype(np.float64)[..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where(dd == 0, 8.0, np.clip(np.rint(g / np.where(dd == 0, 1.0, dd)) + 8.0, 0.0, 15.0))
    return c.astype(np.uint8).reshape(np.asarray(x).shape), d


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What codes and scales stand for, d (c - 8) (exact in f32 too)."""
    c = codes.astype(np.float64).reshape(scales.shape + (GROUP,)) - 8.0
    return (c * scales.astype(np.float64)[..., None]).reshape(codes.shape)


def stored(x: np.ndarray) -> np.ndarray:
    return values(*quantize(x))


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool = False, first: int = 0):
    """q [T, H, hd] over one sequence's rows k, v [L, Hkv, hd] -> (out [T, H, hd], weights [Hkv, L],
    mass [T, H, hd]: sum_j p_j |v_j|, reach [T, H]: the largest sum_d |q_d| K_jd scale, K_jd the largest |k_j| of d's
    group -- the scales of the errors)."""
    T, H, hd = q.shape
    L, hkv = k.shape[0], k.shape[1]
    out, mass = np.zeros((T, H, hd)), np.zeros((T, H, hd))
    reach = np.zeros((T, H))
    w = np.zeros((hkv, L))
    for t in range(T):
        end = min(L, L - T + t + 1) if causal else L
        if end <= first:
            continue
        for h in range(H):
            g = h // (H // hkv)
            kk, vv = k[first:end, g], v[first:end, g]
            s = kk @ q[t, h] * scale
            top = np.abs(kk).reshape(len(kk), -1, min(GROUP, hd)).max(-1)
            reach[t, h] = abs(scale) * np.max(np.repeat(top, min(GROUP, hd), -1) @ np.abs(q[t, h]))
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h] = p @ vv
            mass[t, h] = p @ np.abs(vv)
            w[g, first:end] += p
    return out, w, mass, reach


def attend_heads(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, causal: bool = False, first: int = 0):
    """attend's results by matrix products, a KV head at a time, for cases of many rows."""
    T, H, hd = q.shape
    L, hkv = k.shape[0], k.shape[1]
    out, mass, reach = np.zeros((T, H, hd)), np.zeros((T, H, hd)), np.zeros((T, H))
    w = np.zeros((hkv, L))
    if T == 0 or L == 0:
        return out, w, mass, reach
    n = H // hkv
    size = min(GROUP, hd)
    end = np.minimum(L, L - T + 1 + np.arange(T)) if causal else np.full(T, L)
    seen = (np.arange(L) >= first) & (np.arange(L) < end[:, None])                    # [T, L]
    for g in range(hkv):
        rows = q[:, g * n:(g + 1) * n].reshape(T * n, hd)
        see = np.repeat(seen, n, 0)
        kk, vv = k[:, g], v[:, g]
        top = np.repeat(np.abs(kk).reshape(L, -1, size).max(-1), size, -1)
        s = np.where(see, rows @ kk.T * scale, -np.inf)
        far = np.where(see, np.abs(rows) @ top.T, 0.0)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        total = p.sum(-1, keepdims=True)
        p /= np.where(total > 0, total, 1.0)
        out[:, g * n:(g + 1) * n] = (p @ vv).reshape(T, n, hd)
        mass[:, g * n:(g + 1) * n] = (p @ np.abs(vv)).reshape(T, n, hd)
        reach[:, g * n:(g + 1) * n] = abs(scale) * far.max(-1).reshape(T, n)
        w[g] = p.sum(0)
    return out, w, mass, reach


def kept_rows(w: np.ndarray, keep: int, recent: int) -> np.ndarray:
    """The rows of one head that stay, in order: the last `recent`, and of the others the keep - recent with the
    largest weight, ties to the lowest row, NaN below every number."""
    n = len(w)
    if n <= keep:
        return np.arange(n)
    old = n - recent
    rank = sorted(range(old), key=lambda r: (np.isnan(w[r]), 0.0 if np.isnan(w[r]) else -w[r], r))
    return np.array(sorted(rank[:keep - recent]) + list(range(old, n)), dtype=np.int64)
