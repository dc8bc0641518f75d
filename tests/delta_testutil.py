"""Inputs and comparisons of the gated-delta-rule tests.

Tolerances (derived, with u16 = 2^-8 the rounding of a bf16 value and u32 = 2^-24):
  - an output is rounded to bf16 once: u16 of its value, plus the error of the value before, below;
  - decode and verify compute in fp32: sums of 128 terms, errors of sqrt(128) u32 and a few roundings
    per token, summed as independent over tokens: 2^-19 of a state's norm covers 64 tokens;
  - extend keeps each operand it computes as a bf16 pair, off by at most u16^2 = 2^-16: the state, the
    triangular inverse, the right-hand sides and the solution, of which each element's error is
    independent and about a fifth of that: 2^-16 of a state's norm covers the four of them.
  An output before rounding is D^-0.5 q . S with a state S of the request's run: its error is at most
  the states' relative error times D^-0.5 |q| |S column|, and column norms are within the state's.
"""
import numpy as np
import torch

from oracle import delta

D = 128
U16 = 2.0 ** -8
TOL_RECURRENT = 2.0 ** -19
TOL_EXTEND = 2.0 ** -16
SENTINEL = 54321.0


def inputs(tokens, Hk, H, seed=0, l2=True, gate="model", spread=1.0):
    """q, k (unit keys unless l2), v bf16 and g, beta fp32, on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k = rand(tokens, Hk, D), torch.nn.functional.silu(rand(tokens, Hk, D))
    if l2:
        q, k = q * spread, k * spread
    else:
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    v = rand(tokens, H * D).bfloat16()
    if gate == "model":
        a = 1 + 15 * torch.rand(H, generator=gen)
        dt = torch.exp(torch.rand(H, generator=gen) * np.log(100.0) + np.log(1e-3))
        g = -a * torch.nn.functional.softplus(torch.log(torch.expm1(dt)) + 0.5 * rand(tokens, H))
    elif gate == "none":
        g = torch.zeros(tokens, H)
    elif gate == "steep":
        g = -20 * torch.rand(tokens, H, generator=gen)
    elif gate == "reset":  # some tokens empty the state
        g = -0.05 * torch.rand(tokens, H, generator=gen)
        g[torch.rand(tokens, H, generator=gen) < 0.1] = float("-inf")
        g[torch.rand(tokens, H, generator=gen) < 0.05] = torch.finfo(torch.float32).min
    beta = torch.sigmoid(rand(tokens, H))
    return (q.reshape(tokens, Hk * D).bfloat16(), k.reshape(tokens, Hk * D).bfloat16(), v,
            g.float(), beta)


def make_pool(B, H, slots, prefix, seed=0):
    """(pool, state_idx): prefix states in the slots of prefix requests, NaN in the slots of the
    others, the sentinel in slots that no request names."""
    gen = torch.Generator().manual_seed(seed + 99)
    pool = torch.full((slots, H, D, D), SENTINEL)
    idx = torch.randperm(slots, generator=gen)[:B].int()
    for b in range(B):
        pool[int(idx[b])] = torch.randn(H, D, D, generator=gen) * 0.05 if prefix[b] else float("nan")
    return pool, idx


def f64(t):
    return t.detach().to("cpu").double().numpy()


def check_states(actual, expected, tol, what):
    """Frobenius norm of the error of each [D, D] state within tol of the state's norm."""
    a, e = np.asarray(actual, np.float64), np.asarray(expected, np.float64)
    assert a.shape == e.shape, what
    assert np.isfinite(a).all(), f"{what}: non-finite values"
    err = np.sqrt(((a - e) ** 2).sum((-1, -2)))
    size = np.sqrt((e ** 2).sum((-1, -2)))
    worst = float((err / np.maximum(size, 1e-30)).max()) if err.size else 0.0
    assert (err <= tol * size).all(), f"{what}: relative error {worst:.3g} > {tol:.3g}"
    return worst


def check_out(actual, expected, q, states_norm, tol, Hk, H, l2, what):
    """|a - e| <= u16 |e| + tol D^-0.5 |q| |S|; states_norm: [rows, H], the largest state norm of the
    row's request."""
    a = np.asarray(actual, np.float64).reshape(-1, H, D)
    e = np.asarray(expected, np.float64).reshape(-1, H, D)
    assert np.isfinite(a).all(), f"{what}: non-finite values"
    qn = np.linalg.norm(f64(q).reshape(-1, Hk, D), axis=-1) if not l2 else np.ones((a.shape[0], Hk))
    room = tol * D ** -0.5 * np.repeat(qn, H // Hk, 1) * states_norm
    bad = np.abs(a - e) > U16 * np.abs(e) + room[:, :, None]
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float(np.abs(a - e).max()):.3g}")


def run_states(q, k, v, g, beta, S0, Hk, H, l2):
    """(out, final state, largest state norm [H]) of one request in fp64."""
    n = v.shape[0]
    args = [f64(x).reshape(n, x.shape[1] // D, D) for x in (q, k, v)]
    out, S, states = delta.run(*args, f64(g), f64(beta), S0, l2, keep=True)
    norms = np.sqrt((states ** 2).sum((-1, -2))).max(0) if n else np.zeros(H)
    return out, S, np.maximum(norms, np.sqrt((S0 ** 2).sum((-1, -2))))
