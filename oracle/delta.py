"""fp64 oracle of the gated delta rule and of the packed state store, in plain numpy.

Per request and value head h, with key head h // (H / Hk):

    S <- e^{g_t} S;  u_t = beta_t (v_t - S^T k_t);  S <- S + k_t u_t^T;  o_t = D^-0.5 S^T q_t

token by token.  Test infrastructure only; it shares no code with the CUDA path.
"""
import numpy as np

EPS = 1e-6


def _heads(x, heads, D):
    return np.asarray(x, dtype=np.float64).reshape(-1, heads, D)


def _unit(x):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + EPS)


def run(q, k, v, g, beta, S, qk_l2norm=False, keep=False):
    """One request: q, k [n, Hk, D], v [n, H, D], g, beta [n, H], S [H, D, D] (not modified).
    Returns (out [n, H, D], final S, states after every token [n, H, D, D] or None)."""
    H = v.shape[1]
    S = np.array(S, dtype=np.float64)
    if qk_l2norm:
        q, k = _unit(q), _unit(k)
    rep = H // q.shape[1]
    D = q.shape[2]
    out = np.zeros_like(v, dtype=np.float64)
    states = np.zeros((v.shape[0],) + S.shape) if keep else None
    for t in range(v.shape[0]):
        kt, qt = np.repeat(k[t], rep, 0), np.repeat(q[t], rep, 0)
        S = S * np.exp(g[t])[:, None, None]
        u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, kt))
        S = S + kt[:, :, None] * u[:, None, :]
        out[t] = np.einsum("hkv,hk->hv", S, qt) * D ** -0.5
        if keep:
            states[t] = S
    return out, S, states


def extend(q, k, v, g, beta, pool, state_idx, cu_seqlens, prefix_mask, H, Hk, D, qk_l2norm=False):
    """Returns (out [T, H*D], pool with the final states); rows of no request are NaN in out."""
    q, k, v = _heads(q, Hk, D), _heads(k, Hk, D), _heads(v, H, D)
    g, beta = np.asarray(g, np.float64), np.asarray(beta, np.float64)
    pool = np.array(pool, dtype=np.float64)
    out = np.full(v.shape, np.nan)
    for b, slot in enumerate(state_idx):
        r = slice(int(cu_seqlens[b]), int(cu_seqlens[b + 1]))
        S0 = pool[slot] if prefix_mask[b] else np.zeros(pool.shape[1:])
        out[r], pool[slot], _ = run(q[r], k[r], v[r], g[r], beta[r], S0, qk_l2norm)
    return out.reshape(-1, H * D), pool


def verify_chain(q, k, v, g, beta, pool, state_idx, N, H, Hk, D, qk_l2norm=False):
    """Returns (out [B*N, H*D], states [B, N, H, D, D])."""
    q, k, v = _heads(q, Hk, D), _heads(k, Hk, D), _heads(v, H, D)
    g, beta = np.asarray(g, np.float64), np.asarray(beta, np.float64)
    out = np.zeros(v.shape)
    inter = np.zeros((len(state_idx), N, H, D, D))
    for b, slot in enumerate(state_idx):
        r = slice(b * N, (b + 1) * N)
        out[r], _, inter[b] = run(q[r], k[r], v[r], g[r], beta[r], pool[slot], qk_l2norm, keep=True)
    return out.reshape(-1, H * D), inter


def decode(q, k, v, g, beta, pool, state_idx, H, Hk, D, qk_l2norm=False):
    """Returns (out [B, H*D], pool with the updated states)."""
    out, inter = verify_chain(q, k, v, g, beta, pool, state_idx, 1, H, Hk, D, qk_l2norm)
    pool = np.array(pool, dtype=np.float64)
    pool[np.asarray(state_idx)] = inter[:, 0]
    return out, pool


def pack(x):
    """(codes int8, scales uint8) of fp32 values [..., n * 32] in blocks of 32 along the last axis; the
    largest scale is 2^121, so that every code stands for a finite fp32 value."""
    x = np.asarray(x, dtype=np.float64)
    x = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    top = np.abs(x).max(-1)
    codes = np.zeros(x.shape, np.int8)
    scales = np.full(top.shape, 255, np.uint8)
    for at in np.ndindex(top.shape):
        if not np.isfinite(top[at]):
            continue
        s = 0
        while s < 248 and np.rint(np.ldexp(top[at], 127 - s)) > 127:
            s += 1
        scales[at] = s
        codes[at] = np.clip(np.rint(np.ldexp(x[at], 127 - s)), -127, 127)
    return codes.reshape(codes.shape[:-2] + (-1,)), scales


def unpack(codes, scales):
    """The values codes * 2^(scale - 127) in fp64; NaN in blocks of scale 255."""
    c = np.asarray(codes, np.float64)
    c = c.reshape(c.shape[:-1] + (c.shape[-1] // 32, 32))
    s = np.asarray(scales, np.int64)[..., None]
    x = np.where(s == 255, np.nan, np.ldexp(c, s - 127))
    return x.reshape(x.shape[:-2] + (-1,))
