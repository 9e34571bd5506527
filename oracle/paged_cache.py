"""Plain float64 reference of the paged cache and of the attention over it (test
infrastructure; shares no code with the CUDA path).

A cache is a dict: fmt ("bf16", "e4m3_head" or "e4m3_token"), k / v numpy float64
arrays [pages, page, hkv, d] of the values as stored (codes for e4m3), k_scale /
v_scale float64 ([hkv] or [pages, hkv, page]; None for bf16), table int [R, max],
kv_lens int [R]. New tokens of request r: its last cu[r+1] - cu[r] positions.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value of float64 x (ties to even mantissa), saturating at +-448; NaN stays NaN."""
    x = np.clip(np.asarray(x, dtype=np.float64), -E4M3_MAX, E4M3_MAX)
    _, e = np.frexp(x)                       # x = f * 2^e, f in [0.5, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.round(x / step) * step         # np.round: ties to even


def slots(cache, r: int, pos) -> np.ndarray:
    """Flat slots (page id * page + offset) of request r's positions."""
    page = cache["k"].shape[1]
    pos = np.asarray(pos)
    return cache["table"][r, pos // page].astype(np.int64) * page + pos % page


def new_positions(cache, cu, r: int) -> np.ndarray:
    kv = int(cache["kv_lens"][r])
    return np.arange(kv - (int(cu[r + 1]) - int(cu[r])), kv)


def scales(cache, name: str, flat) -> np.ndarray:
    """[tokens, hkv] scales of the cached tokens in flat slots."""
    hkv, page = cache["k"].shape[2], cache["k"].shape[1]
    sc = cache[name + "_scale"]
    if sc is None:
        return np.ones((len(flat), hkv))
    if sc.ndim == 1:
        return np.broadcast_to(sc, (len(flat), hkv))
    return sc[flat // page, :, flat % page]


def tokens(cache, name: str, flat) -> np.ndarray:
    """float64 values [tokens, hkv, d] of the cached tokens in flat slots."""
    pool = cache[name].reshape(-1, *cache[name].shape[2:])
    return pool[flat] * scales(cache, name, flat)[..., None]


def tree_attention(cache, cu, q, mask, scale):
    """(O [T, hq, d], lse [hq, T], W [T, hq, d], A [T, hq]) of float64 q: the output, the
    log-sum-exp, sum_j p_j |v_j|, and the largest scale * sum_i |q_i k_i| of a key the row
    sees. mask: bool [T, max new tokens] or None (row t of a request sees its new tokens
    0 .. t). Values a row does not see are never touched, so they may be anything."""
    T, hq, d = q.shape
    hkv = cache["k"].shape[2]
    G = hq // hkv
    O, W = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, A = np.full((hq, T), -np.inf), np.zeros((T, hq))
    for r in range(len(cache["kv_lens"])):
        a, b = int(cu[r]), int(cu[r + 1])
        n, kv = b - a, int(cache["kv_lens"][r])
        if n == 0:
            continue
        flat = slots(cache, r, np.arange(kv))
        K, V = tokens(cache, "k", flat), tokens(cache, "v", flat)
        for t in range(n):
            see = np.ones(kv, dtype=bool)
            see[kv - n:] = mask[a + t, :n] if mask is not None else np.arange(n) <= t
            if not see.any():
                continue
            for h in range(hq):
                Ks, Vs = K[see, h // G], V[see, h // G]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = (Ks @ q[a + t, h]) * scale
                    m = s.max()
                    p = np.exp(s - m)
                    z = p.sum()
                    O[a + t, h] = (p @ Vs) / z
                    W[a + t, h] = (p @ np.abs(Vs)) / z
                lse[h, a + t] = m + np.log(z)
                A[a + t, h] = (np.abs(Ks) @ np.abs(q[a + t, h])).max() * scale
    return O, lse, W, A
