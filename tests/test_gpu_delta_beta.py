"""Gated delta rule on the GPU with writing strengths up to 2 (states with negative eigenvalues), and with 32 to
64 value heads, against the fp64 oracle.

Tolerances of the extend at beta up to 2, with unit keys: of the four pair roundings of a chunk (delta_testutil)
those of R, T' and U are of values that carry beta, so up to twice as large against the state as at beta up to 1;
the state's own is not.  A fifth of 2^-16 each in the mean: (1 + 3 x 2) / 5 x 2^-16, below twice TOL_EXTEND, and
below four times where a state is M S + N of a split.  The transitions I - beta k k^T have norm 1 at most, so what
a chunk adds does not grow behind it.  Decode and verify: the roundings of u, of two a token and row, carry beta: twice
TOL_RECURRENT."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from delta_testutil import (D, SENTINEL, TOL_EXTEND, TOL_RECURRENT, check_out, check_states, f64, inputs,
                            make_pool, run_states)
from oracle import delta

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _inputs(tokens, Hk, H, seed, beta, gate="model", l2=True):
    """delta_testutil's, with beta between the two bounds, a tenth of them at each."""
    q, k, v, g, _ = inputs(tokens, Hk, H, seed, l2, gate)
    gen = torch.Generator().manual_seed(seed + 1000)
    b = beta[0] + (beta[1] - beta[0]) * torch.rand(tokens, H, generator=gen)
    at = torch.rand(tokens, H, generator=gen)
    b[at < 0.1], b[at > 0.9] = beta[0], beta[1]
    return q, k, v, g, b


def _to(*ts):
    return [t.to(DEV) for t in ts]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _extend(host, lens, Hk, H, prefix, seed, tol, l2=True, max_seqlen=None):
    B = len(lens)
    pool0, idx = make_pool(B, H, B + 2, prefix, seed)
    pool, cu = pool0.to(DEV), np.cumsum([0] + list(lens))
    out = la.delta_extend(*_to(*host), pool, idx.to(DEV), _i32(cu), torch.tensor(prefix, dtype=torch.uint8, device=DEV),
                          max_seqlen=max_seqlen or max(lens), qk_l2norm=l2)
    la.poll_error()
    for b in range(B):
        r = slice(int(cu[b]), int(cu[b + 1]))
        S0 = f64(pool0[int(idx[b])]) if prefix[b] else np.zeros((H, D, D))
        o, S, norms = run_states(*[x[r] for x in host], S0, Hk, H, l2)
        what = f"request {b} of {lens}"
        check_out(f64(out[r]), o, host[0][r], np.broadcast_to(norms, (lens[b], H)), tol, Hk, H, l2, what)
        check_states(f64(pool[int(idx[b])]), S, tol, what)
    free = [s for s in range(B + 2) if s not in idx.tolist()]
    assert (pool[free] == SENTINEL).all()


@pytest.mark.parametrize("beta", [(0.0, 2.0), (1.0, 2.0), (1.9, 2.0)])
@pytest.mark.parametrize("gate,l2", [("model", True), ("none", True), ("reset", False)])
def test_extend(beta, gate, l2):
    lens, Hk, H = [1, 64, 200, 333, 17], 2, 4
    host = _inputs(sum(lens), Hk, H, 71, beta, gate, l2)
    _extend(host, lens, Hk, H, [1, 0, 1, 0, 1], 71, 2 * TOL_EXTEND, l2)


@pytest.mark.parametrize("lens,H", [([2500], 2), ([41] * 20 + [3000] + [64, 0, 1] * 7, 2), ([70] * 90, 2)])
@pytest.mark.parametrize("gate", ["model", "none"])
def test_extend_split_planned_and_in_waves(lens, H, gate):
    host = _inputs(sum(lens), 1, H, 72, (0.0, 2.0), gate)
    _extend(host, lens, 1, H, [b % 2 for b in range(len(lens))], 72, 4 * TOL_EXTEND)


def test_keys_nearly_the_same():
    """Keys within 8 degrees of one another and beta near 2: every token nearly mirrors what the last one wrote.  The
    derivation of the same test at beta near 1, with values twice as large: 16 sqrt(2) 2^-16, below 24 x 2^-16."""
    n, H = 300, 2
    gen = torch.Generator().manual_seed(73)
    base = torch.randn(1, D, generator=gen)
    k = (base + 0.1 * torch.randn(n, D, generator=gen)).bfloat16()
    q = (base + torch.randn(n, D, generator=gen)).bfloat16()
    v = torch.randn(n, H * D, generator=gen).bfloat16()
    host = (q, k, v, torch.zeros(n, H), 1.9 + 0.1 * torch.rand(n, H, generator=gen))
    _extend(host, [n], 1, H, [0], 73, 24 * TOL_EXTEND)


@pytest.mark.parametrize("lens,Hk,H,l2", [
    ([37, 130], 16, 32, True), ([100], 8, 32, False), ([64, 1, 0, 90], 16, 64, True), ([70] * 5, 1, 48, True),
    ([1500], 4, 40, True), ([2800], 32, 64, True), ([1900, 40, 100], 32, 32, True), ([2, 6, 1, 0], 16, 64, True)])
def test_many_heads(lens, Hk, H, l2):
    """Heads of 32 and more, grouped or not: whole, split (40 heads of 1,500 tokens, 64 of 2,800), in waves, and
    token by token."""
    host = inputs(sum(lens), Hk, H, 74, l2)
    _extend(host, lens, Hk, H, [(b + 1) % 2 for b in range(len(lens))], 74, 2 * TOL_EXTEND, l2)


@pytest.mark.parametrize("B,N,Hk,H,beta", [(3, 1, 2, 4, 2.0), (40, 1, 16, 64, 1.0), (2, 5, 16, 64, 2.0), (2, 40, 1, 2, 2.0),
                                           (9, 3, 32, 32, 2.0)])
def test_decode_and_verify(B, N, Hk, H, beta):
    host = _inputs(B * N, Hk, H, 75 + B, (0.0, beta))
    pool0, idx = make_pool(B, H, B + 2, [1] * B, 75)
    pool = pool0.to(DEV)
    out, inter = la.delta_verify_chain(*_to(*host), pool, idx.to(DEV), N, qk_l2norm=True)
    if N == 1:
        one = la.delta_decode(*_to(*host), pool, idx.to(DEV), qk_l2norm=True)
        la.poll_error()
        assert torch.equal(one, out) and torch.equal(pool[idx.long().to(DEV)], inter[:, 0])
    la.poll_error()
    for b in range(0, B, max(1, B // 4)):
        r = slice(b * N, (b + 1) * N)
        S0 = f64(pool0[int(idx[b])])
        o, _, norms = run_states(*[x[r] for x in host], S0, Hk, H, True)
        args = [f64(x[r]).reshape(N, -1, D) for x in host[:3]]
        _, _, states = delta.run(*args, f64(host[3][r]), f64(host[4][r]), S0, True, keep=True)
        check_out(f64(out[r]), o, host[0][r], np.broadcast_to(norms, (N, H)), 2 * TOL_RECURRENT, Hk, H, True, str(b))
        check_states(f64(inter[b]), states, 2 * TOL_RECURRENT, str(b))
