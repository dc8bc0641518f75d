"""Gated delta rule on the GPU (la_delta_extend, la_delta_decode, la_delta_verify_chain) against the
fp64 oracle: outputs and states at the derived tolerances of delta_testutil, untouched slots and rows
bit for bit, head layouts, lengths, gates, strides, refusals and device-detected faults."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from delta_testutil import (D, SENTINEL, TOL_EXTEND, TOL_RECURRENT, check_out, check_states, f64,
                            inputs, make_pool, run_states)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _to(*ts):
    return [t.to(DEV) for t in ts]


def check_extend(lens, Hk, H, l2=True, gate="model", seed=0, prefix=None, gap=0, tail=0, spread=1.0,
                 wide=False, max_seqlen=None, tol=TOL_EXTEND):
    """One extend call; `gap` rows before and `tail` rows behind the requests hold NaN inputs."""
    B, n = len(lens), sum(lens)
    T = gap + n + tail
    prefix = [b % 2 for b in range(B)] if prefix is None else prefix
    q, k, v, g, beta = inputs(T, Hk, H, seed, l2, gate, spread)
    for x in (q, k, v, g, beta):
        x[:gap] = float("nan")
        x[gap + n:] = float("nan")
    pool0, idx = make_pool(B, H, B + 3, prefix, seed)
    cu = torch.tensor(np.cumsum([gap] + list(lens)), dtype=torch.int32)
    if wide:  # q, k and v as column ranges of one projection
        rows = torch.cat([q, k, v, torch.full((T, 24), float("nan")).bfloat16()], 1).to(DEV)
        dq, dk, dv = rows[:, :Hk * D], rows[:, Hk * D:2 * Hk * D], rows[:, 2 * Hk * D:(2 * Hk + H) * D]
    else:
        dq, dk, dv = _to(q, k, v)
    pool = pool0.to(DEV)
    out = torch.full((T, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    got = la.delta_extend(dq, dk, dv, *_to(g, beta), pool, *_to(idx, cu),
                          torch.tensor(prefix, dtype=torch.uint8, device=DEV), out=out,
                          max_seqlen=max_seqlen or (max(lens) if lens else 0), qk_l2norm=l2)
    la.poll_error()
    assert got is out
    for b in range(B):
        r = slice(int(cu[b]), int(cu[b + 1]))
        S0 = f64(pool0[int(idx[b])]) if prefix[b] else np.zeros((H, D, D))
        o, S, norms = run_states(q[r], k[r], v[r], g[r], beta[r], S0, Hk, H, l2)
        what = f"request {b} of {lens}"
        check_out(f64(out[r]), o, q[r], np.broadcast_to(norms, (lens[b], H)), tol, Hk, H, l2, what)
        check_states(f64(pool[int(idx[b])]), S, tol, what)
        if lens[b] == 0:
            assert torch.equal(pool[int(idx[b])].cpu(), torch.from_numpy(S).float())
    free = [s for s in range(B + 3) if s not in idx.tolist()]
    assert (pool[free] == SENTINEL).all()
    assert (out[:gap] == 77.0).all() and (out[gap + n:] == 77.0).all()
    return out, pool


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 128, 129, 191, 321])
@pytest.mark.parametrize("prefix", [0, 1])
def test_extend_lengths(n, prefix):
    check_extend([n], 1, 1, prefix=[prefix], seed=n)


@pytest.mark.parametrize("lens", [[1, 2, 0, 3], [6, 5], [1] * 40, [6] * 170])
@pytest.mark.parametrize("max_seqlen", [None, 64])
def test_extend_few_tokens(lens, max_seqlen):
    # token by token, and by chunks where max_seqlen allows for more
    check_extend(lens, 1, 2, max_seqlen=max_seqlen, seed=len(lens), gap=2, tail=70)
    check_extend(lens, 2, 2, l2=False, gate="reset", max_seqlen=max_seqlen, seed=len(lens))


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 3), (2, 4), (4, 4), (3, 6)])
@pytest.mark.parametrize("l2", [True, False])
def test_extend_heads(Hk, H, l2):
    check_extend([70, 1, 0, 129], Hk, H, l2=l2, seed=Hk * 10 + H)


@pytest.mark.parametrize("gate", ["none", "steep", "reset"])
def test_extend_gates(gate):
    check_extend([200, 65, 130], 2, 2, gate=gate, seed=5)


def test_extend_rows_outside_requests():
    # NaN rows before the first and behind the last sequence are neither read into it nor written
    check_extend([37, 90, 64], 2, 4, gap=5, tail=70, seed=6)


def test_extend_neighbours_with_nan():
    """A request full of NaN does not reach the requests around it."""
    lens, Hk, H = [40, 50, 30], 1, 2
    q, k, v, g, beta = inputs(120, Hk, H, 7)
    for x in (q, k, v):
        x[40:90] = float("nan")
    pool0, idx = make_pool(3, H, 5, [1, 1, 1], 7)
    pool = pool0.to(DEV)
    cu = torch.tensor([0, 40, 90, 120], dtype=torch.int32)
    out = la.delta_extend(*_to(q, k, v, g, beta), pool, *_to(idx, cu),
                          torch.ones(3, dtype=torch.uint8, device=DEV), max_seqlen=50, qk_l2norm=True)
    la.poll_error()
    for b in (0, 2):
        r = slice(int(cu[b]), int(cu[b + 1]))
        o, S, norms = run_states(q[r], k[r], v[r], g[r], beta[r], f64(pool0[int(idx[b])]), Hk, H, True)
        check_out(f64(out[r]), o, q[r], np.broadcast_to(norms, (lens[b], H)), TOL_EXTEND, Hk, H, True, "nan")
        check_states(f64(pool[int(idx[b])]), S, TOL_EXTEND, "nan")


def test_extend_strided_projection():
    check_extend([77, 130], 2, 4, wide=True, seed=8)


def test_extend_scales_of_inputs():
    # the 2-norm is divided out: large and small q and k give the same error
    check_extend([100], 1, 2, spread=1e4, seed=9)
    check_extend([100], 1, 2, spread=1e-2, seed=9)


def test_extend_long():
    check_extend([1500], 1, 2, gate="none", seed=10, prefix=[1])
    check_extend([1500], 1, 2, seed=11, prefix=[1])


def test_extend_many_requests():
    r = np.random.default_rng(12)
    check_extend([int(x) for x in r.integers(0, 140, 90)], 1, 2, seed=12)


@pytest.mark.parametrize("lens,Hk,H,l2,gate,max_seqlen", [
    ([2500], 1, 2, True, "model", None),
    ([2048], 1, 1, True, "none", None),
    ([10000], 1, 1, True, "model", None),  # many segments
    ([2085, 0, 5, 700, 2048, 64, 130], 1, 2, True, "model", None),
    ([40, 2300], 1, 3, False, "none", 1 << 30),
    ([2111], 5, 20, True, "reset", None),  # segment 0 twice as long as the others
    ([900, 700], 1, 1, True, "model", 2100),  # taken as long, and every request is shorter
    ([1300, 900, 1279], 1, 2, True, "model", 3400),
    # one cut for all requests, planned on the device: one long among short ones, two, a mixed batch,
    # none that is worth a cut, one in very many
    ([41] * 20 + [3000] + [64, 0, 1] * 7, 1, 2, True, "model", None),
    ([1700] + [5] * 38 + [2400], 2, 2, False, "none", None),
    ([1500, 3, 0, 200, 700, 1400], 4, 16, True, "model", None),
    ([64, 0, 2500, 100, 65, 40], 4, 16, True, "model", None),
    ([100] * 77, 1, 1, True, "reset", 7700),
    ([17] * 60 + [2000] + [9] * 67, 1, 1, True, "model", None),
    ([17] * 300 + [2000] + [9] * 211, 1, 1, True, "model", None),  # too many for a plan
])
def test_extend_split(lens, Hk, H, l2, gate, max_seqlen):
    """Few long requests: the chain in segments.  A state is M S + N, with M and N each within the
    extend's tolerance."""
    check_extend(lens, Hk, H, l2=l2, gate=gate, max_seqlen=max_seqlen, seed=21, gap=3, tail=600,
                 prefix=[(b + 1) % 2 for b in range(len(lens))], tol=2 * TOL_EXTEND)


@pytest.mark.parametrize("n,H", [(20000, 1), (33333, 2), (30000, 24)])
def test_extend_split_equals_shorter_calls(n, H):
    """A long request in as many segments as there are against calls of 1,216 tokens, which are not
    split: each within the extend's tolerance of the formula, the split one within twice that."""
    q, k, v, g, beta = _to(*inputs(n, 1, H, 23))
    idx = torch.tensor([1], dtype=torch.int32, device=DEV)
    outs, pools = [], []
    for step in (n, 1216):
        pool = torch.full((3, H, D, D), SENTINEL, device=DEV)
        o = []
        for a in range(0, n, step):
            b = min(n, a + step)
            o.append(la.delta_extend(q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], pool, idx,
                                     torch.tensor([0, b - a], dtype=torch.int32, device=DEV),
                                     torch.tensor([int(a > 0)], dtype=torch.uint8, device=DEV), qk_l2norm=True))
        outs.append(torch.cat(o))
        pools.append(pool)
    la.poll_error()
    check_states(f64(pools[0][1]), f64(pools[1][1]), 3 * TOL_EXTEND, "split")
    # a state holds about one value per key direction, a norm of sqrt(128) |v| = 128; each output is
    # rounded once, and before that off by 3 x 2^-16 x 128 x 128^-0.5 at most
    assert pools[1][1].norm(dim=(1, 2)).max() < 128
    assert torch.allclose(outs[0].float(), outs[1].float(), rtol=2.0 ** -7, atol=5.2e-4)
    assert (pools[0][[0, 2]] == SENTINEL).all()


def test_extend_split_nan_stays_behind():
    """NaN inputs late in a split request leave the outputs before them as they were."""
    n, H = 2600, 2
    q, k, v, g, beta = _to(*inputs(n, 1, H, 22))
    idx = torch.tensor([1], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    mask = torch.ones(1, dtype=torch.uint8, device=DEV)
    outs = []
    for bad in (False, True):
        if bad:
            k[2000] = float("nan")
        pool = torch.full((3, H, D, D), 0.01, device=DEV)
        outs.append(la.delta_extend(q, k, v, g, beta, pool, idx, cu, mask, qk_l2norm=True))
    la.poll_error()
    assert torch.equal(outs[0][:1984], outs[1][:1984])  # 1984: the chunk of token 2000
    assert outs[1][2000:].isnan().all()
    assert pool[1].isnan().all() and (pool[[0, 2]] == 0.01).all()


def test_extend_in_two_calls_equals_one():
    Hk, H, n = 2, 2, 300
    q, k, v, g, beta = _to(*inputs(n, Hk, H, 13))
    idx = torch.tensor([1], dtype=torch.int32, device=DEV)
    outs, pools = [], []
    for cuts in ([0, 300], [0, 101, 300]):
        pool = torch.full((3, H, D, D), SENTINEL, device=DEV)
        o = []
        for a, b in zip(cuts, cuts[1:]):
            o.append(la.delta_extend(q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], pool, idx,
                                     torch.tensor([0, b - a], dtype=torch.int32, device=DEV),
                                     torch.tensor([int(a > 0)], dtype=torch.uint8, device=DEV), qk_l2norm=True))
        outs.append(torch.cat(o))
        pools.append(pool)
    la.poll_error()
    check_states(f64(pools[1][1]), f64(pools[0][1]), 2 * TOL_EXTEND, "two calls")
    assert torch.allclose(outs[0].float(), outs[1].float(), rtol=2.0 ** -6, atol=1e-3)


def _decode_like(B, N, Hk, H, l2, seed, gate="model", wide=False):
    q, k, v, g, beta = inputs(B * N, Hk, H, seed, l2, gate)
    pool0, idx = make_pool(B, H, B + 2, [1] * B, seed)
    if wide:
        rows = torch.cat([k, v, q], 1).to(DEV)
        dk, dv, dq = rows[:, :Hk * D], rows[:, Hk * D:(Hk + H) * D], rows[:, (Hk + H) * D:]
    else:
        dq, dk, dv = _to(q, k, v)
    return (q, k, v, g, beta), (dq, dk, dv, *_to(g, beta)), pool0, idx


@pytest.mark.parametrize("B,Hk,H,l2,gate,wide", [
    (1, 1, 1, True, "model", False), (3, 2, 4, False, "model", True), (7, 4, 4, True, "reset", False),
    (5, 1, 3, True, "none", True), (100, 4, 8, True, "model", False), (2, 2, 2, False, "steep", False)])
def test_decode(B, Hk, H, l2, gate, wide):
    host, dev, pool0, idx = _decode_like(B, 1, Hk, H, l2, B + H, gate, wide)
    pool = pool0.to(DEV)
    out = la.delta_decode(*dev, pool, idx.to(DEV), qk_l2norm=l2)
    la.poll_error()
    for b in range(0, B, max(1, B // 8)):
        r = slice(b, b + 1)
        o, S, norms = run_states(*[x[r] for x in host], f64(pool0[int(idx[b])]), Hk, H, l2)
        check_out(f64(out[r]), o, host[0][r], norms[None], TOL_RECURRENT, Hk, H, l2, f"decode {b}")
        check_states(f64(pool[int(idx[b])]), S, TOL_RECURRENT, f"decode {b}")
    free = [s for s in range(B + 2) if s not in idx.tolist()]
    assert (pool[free] == SENTINEL).all()


@pytest.mark.parametrize("B,N,Hk,H,l2,gate,wide", [
    (1, 1, 1, 1, True, "model", False), (3, 4, 2, 4, True, "model", True), (2, 9, 1, 2, False, "reset", False),
    (40, 3, 4, 8, True, "model", False), (2, 64, 1, 1, True, "none", False)])
def test_verify_chain_and_commit(B, N, Hk, H, l2, gate, wide):
    host, dev, pool0, idx = _decode_like(B, N, Hk, H, l2, B + N, gate, wide)
    pool = pool0.to(DEV)
    out, inter = la.delta_verify_chain(*dev, pool, idx.to(DEV), N, qk_l2norm=l2)
    assert torch.equal(pool.cpu(), pool0)
    accept = torch.tensor([(b % (N + 1)) - 1 for b in range(B)], dtype=torch.int32)
    la.commit_accepted(inter, accept.to(DEV), pool, idx.to(DEV))
    la.poll_error()
    from oracle import delta
    for b in range(0, B, max(1, B // 6)):
        r = slice(b * N, (b + 1) * N)
        S0 = f64(pool0[int(idx[b])])
        o, _, norms = run_states(*[x[r] for x in host], S0, Hk, H, l2)
        args = [f64(x[r]).reshape(N, -1, D) for x in host[:3]]
        _, _, states = delta.run(*args, f64(host[3][r]), f64(host[4][r]), S0, l2, keep=True)
        check_out(f64(out[r]), o, host[0][r], np.broadcast_to(norms, (N, H)), TOL_RECURRENT, Hk, H, l2, f"verify {b}")
        check_states(f64(inter[b]), states, TOL_RECURRENT, f"verify {b}")
        a = int(accept[b])
        assert torch.equal(pool[int(idx[b])], inter[b, a] if a >= 0 else pool0[int(idx[b])].to(DEV))


def test_modes_agree_as_they_are_used():
    """Extend a prompt, decode two tokens, verify three drafts, commit: one request's run."""
    Hk, H, n = 2, 4, 90
    q, k, v, g, beta = inputs(n + 5, Hk, H, 21)
    d = _to(q, k, v, g, beta)
    idx = torch.tensor([2], dtype=torch.int32, device=DEV)
    pool = torch.full((4, H, D, D), SENTINEL, device=DEV)
    outs = [la.delta_extend(*[x[:n] for x in d], pool, idx, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                            torch.zeros(1, dtype=torch.uint8, device=DEV), qk_l2norm=True)]
    for t in (n, n + 1):
        outs.append(la.delta_decode(*[x[t:t + 1] for x in d], pool, idx, qk_l2norm=True))
    o, inter = la.delta_verify_chain(*[x[n + 2:] for x in d], pool, idx, 3, qk_l2norm=True)
    outs.append(o)
    la.commit_accepted(inter, torch.tensor([2], dtype=torch.int32, device=DEV), pool, idx)
    la.poll_error()
    ref, S, norms = run_states(q, k, v, g, beta, np.zeros((H, D, D)), Hk, H, True)
    check_out(f64(torch.cat(outs)), ref, q, np.broadcast_to(norms, (n + 5, H)), TOL_EXTEND, Hk, H, True, "run")
    check_states(f64(pool[2]), S, TOL_EXTEND, "run")
    assert (pool[[0, 1, 3]] == SENTINEL).all()


def test_device_faults_are_reported_and_skipped():
    Hk = H = 1
    q, k, v, g, beta = _to(*inputs(30, Hk, H, 22))
    pool = torch.full((4, H, D, D), SENTINEL, device=DEV)
    one = torch.ones(2, dtype=torch.uint8, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for idx, cu, ms in ((i32(0, 4), i32(0, 10, 30), 30), (i32(-1, 2), i32(0, 10, 30), 30),
                        (i32(0, 1), i32(0, 31, 30), 31), (i32(0, 1), i32(0, 10, 31), 30),
                        (i32(0, 1), i32(0, 10, 30), 19),
                        (i32(0, 4), i32(0, 3, 6), 3), (i32(0, 1), i32(0, 3, 2), 3),
                        (i32(0, 1), i32(0, 2, 6), 3), (i32(0, 1), i32(28, 30, 31), 3)):
        la.delta_extend(q, k, v, g, beta, pool, idx, cu, one, max_seqlen=ms, qk_l2norm=True)
        with pytest.raises(la.LAError) as e:
            la.poll_error()
        assert e.value.status == 5
    before = pool.clone()
    la.delta_decode(q[:2], k[:2], v[:2], g[:2], beta[:2], pool, i32(4, -3), qk_l2norm=True)
    with pytest.raises(la.LAError):
        la.poll_error()
    la.delta_verify_chain(q[:4], k[:4], v[:4], g[:4], beta[:4], pool, i32(4, 99), 2, qk_l2norm=True)
    with pytest.raises(la.LAError):
        la.poll_error()
    assert torch.equal(pool, before)
    la.poll_error()


def test_empty_batches():
    e = torch.empty(0, D, dtype=torch.bfloat16, device=DEV)
    f = torch.empty(0, 1, device=DEV)
    pool = torch.full((2, 1, D, D), SENTINEL, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    la.delta_extend(e, e, e, f, f, pool, none, torch.zeros(1, dtype=torch.int32, device=DEV),
                    torch.empty(0, dtype=torch.uint8, device=DEV))
    la.delta_decode(e, e, e, f, f, pool, none)
    la.delta_verify_chain(e, e, e, f, f, pool, none, 3)
    # requests without tokens: states are zeroed or kept
    la.delta_extend(e, e, e, f, f, pool, torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                    torch.zeros(3, dtype=torch.int32, device=DEV),
                    torch.tensor([0, 1], dtype=torch.uint8, device=DEV))
    la.poll_error()
    assert (pool[0] == 0).all() and (pool[1] == SENTINEL).all()


def test_streams_and_graph_replay():
    """Calls on a side stream, and one graph of extend + decode replayed on new inputs."""
    Hk, H, n = 1, 2, 100
    host = inputs(n + 1, Hk, H, 23)
    d = _to(*host)
    idx = torch.tensor([0], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    zero = torch.zeros(1, dtype=torch.uint8, device=DEV)
    pool = torch.zeros(1, H, D, D, device=DEV)

    def step():
        a = la.delta_extend(*[x[:n] for x in d], pool, idx, cu, zero, max_seqlen=n, qk_l2norm=True)
        return a, la.delta_decode(*[x[n:] for x in d], pool, idx, qk_l2norm=True)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a0, b0 = step()
        p0 = pool.clone()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, b = step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, a0) and torch.equal(b, b0) and torch.equal(pool, p0)
    host2 = inputs(n + 1, Hk, H, 24)
    for x, y in zip(d, host2):
        x.copy_(y)
    g.replay()
    la.poll_error()
    ref, S, norms = run_states(*host2, np.zeros((H, D, D)), Hk, H, True)
    check_out(f64(torch.cat([a, b])), ref, host2[0], np.broadcast_to(norms, (n + 1, H)), TOL_EXTEND, Hk, H, True, "graph")
    check_states(f64(pool[0]), S, TOL_EXTEND, "graph")


def test_repeated_calls_are_bit_equal():
    lens, Hk, H = [130, 64, 1, 77], 2, 4
    q, k, v, g, beta = _to(*inputs(sum(lens), Hk, H, 25))
    idx = torch.arange(4, dtype=torch.int32, device=DEV)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device=DEV)
    got = []
    for _ in range(3):
        pool = torch.zeros(4, H, D, D, device=DEV)
        out = la.delta_extend(q, k, v, g, beta, pool, idx, cu, torch.zeros(4, dtype=torch.uint8, device=DEV),
                              max_seqlen=130, qk_l2norm=True)
        got.append((out, pool))
    la.poll_error()
    for o, p in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(p, got[0][1])
