"""Rotary positions and softmax attention over a paged key/value cache in fp64 numpy: the definitions that the
library's la_rope, la_kv_store, la_attn_* and la_kv_commit are tested against (test infrastructure only)."""
import numpy as np


def rope(x, positions, inv_freq, interleaved=False, mscale=1.0):
    """x [T, heads, D] -> the same, its first 2 * len(inv_freq) columns rotated."""
    y = np.array(x, np.float64)
    R = 2 * len(inv_freq)
    # whole turns are dropped before the product loses bits to them
    angle = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)[None]
    angle = np.fmod(angle, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    cos, sin = (np.asarray(f(angle), np.float64)[:, None] * mscale for f in (np.cos, np.sin))
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * cos - v * sin, u * sin + v * cos
    return y


def rows(pages, table, n):
    """The first n positions of a request: pages [E, Hkv, P, D], table [max_pages] -> [n, Hkv, D]."""
    P = pages.shape[2]
    at = np.arange(n)
    return np.asarray(pages[table[at // P], :, at % P], np.float64)


def attend(q, k, v, seen, scale):
    """q [n, H, D], k, v [L, Hkv, D], seen [n, L] bool -> (out [n, H, D], sum_j w_ij |v_j| [n, H, D]); rows that see
    nothing are zero."""
    n, H, D = q.shape
    Hkv = k.shape[1]
    out, size = np.zeros((2, n, H, D))
    for h in range(H):
        kh, vh = k[:, h // (H // Hkv)], v[:, h // (H // Hkv)]
        s = np.where(seen, scale * (q[:, h] @ kh.T), -np.inf)
        m = s.max(-1, initial=-np.inf, keepdims=True)
        w = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        total = w.sum(-1, keepdims=True)
        w = w / np.where(total == 0, 1.0, total)
        out[:, h], size[:, h] = w @ vh, w @ np.abs(vh)
    return out, size


def causal(n, total):
    """Row i of the last n of `total` positions sees those at and before its own."""
    return np.arange(total)[None] <= np.arange(total - n, total)[:, None]


def tree(parents, total):
    """Draft t, one of the last len(parents) of `total` positions, sees the ones before them, its path and itself."""
    n = len(parents)
    seen = np.zeros((n, total), bool)
    seen[:, :total - n] = True
    for t in range(n):
        a = t
        while a >= 0:
            seen[t, total - n + a] = True
            a = parents[a]
    return seen


def path(parents, last):
    """Drafts from the context to `last`, in order."""
    found = []
    while last >= 0:
        found.insert(0, int(last))
        last = parents[last]
    return found
