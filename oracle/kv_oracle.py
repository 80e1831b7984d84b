"""Plain oracle of the key/value cache in 4 bits: float64 NumPy, one token after
another (test infrastructure only; shares no code with the library).

quantise: the pair and codes of every group, every border compared exactly.
attention: softmax over what a row sees, with the magnitudes that error bounds
are made of.  evict: the slots that stay, by sorting.
"""
from __future__ import annotations

import numpy as np

__all__ = ["quantise", "values", "attention", "evict"]

CLAMP = 32768.0


def quantise(x: np.ndarray, g: int):
    """x [..., D] (any float type) -> (u int [..., D], lo, s float64 [..., D / g])."""
    x = np.asarray(x, np.float64)
    x = np.clip(np.where(np.isnan(x), 0.0, x), -CLAMP, CLAMP)
    grp = x.reshape(*x.shape[:-1], x.shape[-1] // g, g)
    mn, mx = grp.min(-1), grp.max(-1)
    lo = mn.astype(np.float32).astype(np.float16).astype(np.float64)
    step = (mx.astype(np.float32) - mn.astype(np.float32)) / np.float32(15.0)
    s = step.astype(np.float16).astype(np.float64)
    u = np.zeros(grp.shape, np.int64)
    for j in range(15):   # lo + (j + 1/2) s is exact in float64
        u += grp >= (lo + (j + 0.5) * s)[..., None]
    u[np.broadcast_to((s == 0)[..., None], u.shape)] = 0
    return u.reshape(x.shape), lo, s


def values(u, lo, s):
    g = u.shape[-1] // lo.shape[-1]
    return np.repeat(lo, g, -1) + np.repeat(s, g, -1) * u


def attention(q, k_q, v_q, scale, causal=True, window=0, absent=()):
    """One sequence and kv head.  q float64 [T, H, D] (the kv head's q heads), k_q
    and v_q = (u, lo, s) of its n tokens, absent: slots without a page.
    Returns a dict of out [T, H, D], lse [T, H], weights [n] and, for bounds,
    code (sum of P s u, like out), size (sum of P |v|, like out), reach_z
    [T, H] (the largest of scale sum |q| (|lo| + s u) over the slots seen) and
    keys_z (the same of scale sum |q| |k|)."""
    k, v = values(*k_q), values(*v_q)
    n, D = k.shape
    T, H, _ = q.shape
    g = D // k_q[1].shape[-1]
    k_abs = np.repeat(np.abs(k_q[1]), g, -1) + np.repeat(k_q[2], g, -1) * k_q[0]
    v_code = np.repeat(v_q[2], g, -1) * v_q[0]
    r = dict(out=np.zeros((T, H, D)), lse=np.full((T, H), -np.inf), weights=np.zeros(n), code=np.zeros((T, H, D)),
             size=np.zeros((T, H, D)), reach_z=np.zeros((T, H)), keys_z=np.zeros((T, H)))
    for i in range(T):
        p = n - T + i
        see = np.ones(n, bool)
        see[list(absent)] = False
        t = np.arange(n)
        if causal:
            see &= t <= p
        if window:
            see &= t > p - window
        if not see.any():
            continue
        for h in range(H):
            z = scale * (k[see] @ q[i, h])
            m = z.max()
            e = np.exp(z - m)
            P = e / e.sum()
            r["out"][i, h] = P @ v[see]
            r["lse"][i, h] = m + np.log(e.sum())
            r["weights"][see] += P
            r["code"][i, h] = P @ v_code[see]
            r["size"][i, h] = P @ np.abs(v[see])
            r["reach_z"][i, h] = abs(scale) * (k_abs[see] @ np.abs(q[i, h])).max()
            r["keys_z"][i, h] = abs(scale) * (np.abs(k[see]) @ np.abs(q[i, h])).max()
    return r


def evict(w: np.ndarray, keep: int, sinks: int, recent: int) -> np.ndarray:
    """The slots that stay of one sequence and kv head with weights w [n], ascending."""
    n = len(w)
    if n <= keep:
        return np.arange(n)
    w = np.where(np.isnan(w), np.inf, w)   # stable sort: ties to the lowest slot
    middle = np.arange(sinks, n - recent)
    order = middle[np.argsort(-w[middle], kind="stable")][: keep - sinks - recent]
    return np.sort(np.concatenate([np.arange(sinks), order, np.arange(n - recent, n)])).astype(np.int64)
