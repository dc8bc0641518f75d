"""Gated delta rule and packed state store at the edges of what a call allows: waits that run out,
two calls at once, captured calls, offsets past 32 bits, large batches, NaN that stays within its
request, and keys that are nearly the same."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from delta_testutil import (D, SENTINEL, TOL_EXTEND, check_out, check_states, f64, inputs, make_pool,
                            run_states)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _to(*ts):
    return [t.to(DEV) for t in ts]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _i32(np.cumsum([0] + list(lens)))


def _mask(n, value=0):
    return torch.full((n,), value, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("lens,H,must", [([1000, 300], 2, True), ([3000], 2, True),
                                          ([700] * 80, 2, True), ([40] * 100, 2, False),
                                          ([3000] + [64] * 40, 2, True)])
def test_waits_that_run_out(lens, H, must):
    """Calls under a 1 us wait limit are reported as LA_ERR_TIMEOUT; the next call is as ever.  A try
    of a wait may itself be suspended for a few microseconds, so that the waits of a request of one
    chunk need not run out, and of longer ones some call's do."""
    B = len(lens)
    d = _to(*inputs(sum(lens), 1, H, 31))
    args = (_i32(list(range(B))), _cu(lens), _mask(B))
    pool = torch.zeros(B, H, D, D, device=DEV)
    want = la.delta_extend(*d, pool, *args, max_seqlen=max(lens), qk_l2norm=True)
    states = pool.clone()
    la.poll_error()
    status = []
    la.set_wait_limit(1)
    try:
        for _ in range(10):
            la.delta_extend(*d, pool, *args, max_seqlen=max(lens), qk_l2norm=True)
            try:
                la.poll_error()
            except la.LAError as e:
                status.append(e.status)
    finally:
        la.set_wait_limit(0)
    assert set(status) <= {4} and (status or not must)  # LA_ERR_TIMEOUT
    la.poll_error()
    got = la.delta_extend(*d, pool, *args, max_seqlen=max(lens), qk_l2norm=True)
    la.poll_error()
    assert torch.equal(got, want) and torch.equal(pool, states)


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, pool slots and outputs, give what they
    give alone."""
    cases = []
    for seed, lens, H in ((32, [700, 900, 64], 4), (33, [2500], 2)):
        d = _to(*inputs(sum(lens), 1, H, seed))
        B = len(lens)
        cases.append((d, lens, H, (_i32(list(range(B))), _cu(lens), _mask(B))))
    alone = []
    for d, lens, H, args in cases:
        pool = torch.zeros(len(lens), H, D, D, device=DEV)
        alone.append((la.delta_extend(*d, pool, *args, max_seqlen=max(lens), qk_l2norm=True), pool))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        for s, (d, lens, H, args) in zip(streams, cases):
            with torch.cuda.stream(s):
                pool = torch.zeros(len(lens), H, D, D, device=DEV)
                got.append((la.delta_extend(*d, pool, *args, max_seqlen=max(lens), qk_l2norm=True), pool))
    torch.cuda.synchronize()
    la.poll_error()
    for i, (o, p) in enumerate(got):
        assert torch.equal(o, alone[i % 2][0]) and torch.equal(p, alone[i % 2][1])


def test_two_graphs_with_one_workspace():
    """Two captured extends (split and whole) share one workspace and replay one after the other."""
    lens = ([2200], [300, 80])
    H = 2
    sizes = [la.delta_extend_workspace_size(len(x), sum(x), H, D) for x in lens]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device=DEV)
    runs = []
    for i, x in enumerate(lens):
        d = _to(*inputs(sum(x), 1, H, 34 + i))
        args = (_i32(list(range(len(x)))), _cu(x), _mask(len(x)))
        pool = torch.zeros(len(x), H, D, D, device=DEV)
        out = torch.empty(sum(x), H * D, dtype=torch.bfloat16, device=DEV)
        call = lambda d=d, args=args, pool=pool, out=out, x=x: la.delta_extend(  # noqa: E731
            *d, pool, *args, out=out, max_seqlen=max(x), qk_l2norm=True, workspace=ws)
        call()
        torch.cuda.synchronize()
        want = out.clone(), pool.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, out, pool, want, call))  # call keeps the captured inputs alive
    for _ in range(3):
        for g, out, pool, *_ in runs:
            out.zero_()
            pool.fill_(SENTINEL)
            g.replay()
        torch.cuda.synchronize()
        for _, out, pool, want, _ in runs:
            assert torch.equal(out, want[0]) and torch.equal(pool, want[1])
    la.poll_error()


def test_verify_commit_pack_and_unpack_in_a_graph():
    B, N, H = 3, 4, 2
    d = _to(*inputs(B * N, 1, H, 36))
    pool0, idx = make_pool(B, H, B + 2, [1] * B, 36)
    idx = idx.to(DEV)
    accept = _i32([0, 3, -1])
    store = _i32([2, 0, 1])

    def buffers():
        return (pool0.nan_to_num(0.5).to(DEV), torch.zeros(3, H, D, D, dtype=torch.int8, device=DEV),
                torch.zeros(3, H, D, D // 32, dtype=torch.uint8, device=DEV))

    def step(pool, codes, scales):
        out, inter = la.delta_verify_chain(*d, pool, idx, N, qk_l2norm=True)
        la.commit_accepted(inter, accept, pool, idx)
        la.pack_states(pool, idx, codes, scales, store)
        la.unpack_states(codes, scales, store, pool, idx)
        return out

    eager = buffers()
    want = step(*eager)
    torch.cuda.synchronize()
    mine = buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(*mine)
    for _ in range(2):
        for x, y in zip(mine, buffers()):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for x, y in zip(mine, eager):
            assert torch.equal(x, y)
    la.poll_error()


def test_slots_and_entries_past_32_bits():
    """The last slot of a pool of more than 2^31 values (8.6 GB), the last entry of a store of more
    than 2^31 codes."""
    H, slots = 16, 8200
    assert (slots - 1) * H * D * D > 2 ** 31
    pool = torch.empty(slots, H, D, D, device=DEV)
    small = torch.randn(2, H, D, D, generator=torch.Generator().manual_seed(37)).to(DEV) * 0.05
    d = _to(*inputs(100, 1, H, 37))
    far, near = _i32([slots - 1, 3]), _i32([0, 1])

    def run(pool, idx, store, entries):
        pool[idx.long()] = small
        o = [la.delta_extend(*d, pool, idx, _cu([70, 30]), _mask(2, 1), max_seqlen=70, qk_l2norm=True),
             la.delta_decode(*[x[:2] for x in d], pool, idx, qk_l2norm=True)]
        o += la.delta_verify_chain(*[x[:6] for x in d], pool, idx, 3, qk_l2norm=True)
        codes = torch.empty(entries, H, D, D, dtype=torch.int8, device=DEV)
        scales = torch.empty(entries, H, D, D // 32, dtype=torch.uint8, device=DEV)
        la.pack_states(pool, idx, codes, scales, store)
        o += [pool[idx.long()].clone(), codes[store.long()], scales[store.long()]]
        la.unpack_states(codes, scales, store, pool, idx)
        o.append(pool[idx.long()].clone())
        la.poll_error()
        return o

    want = run(torch.empty(2, H, D, D, device=DEV), near, near, 2)
    got = run(pool, far, _i32([slots - 1, 5]), slots)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_tokens_past_32_bits():
    """512 requests of 520 tokens x 64 heads: token offsets past 2^31 values, a workspace past 2^32
    bytes; sampled requests equal the same requests alone, bit for bit."""
    B, n, H, Hk = 512, 520, 64, 64
    T = B * n
    assert T * H * D > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(38)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    q, k, v = rand(T, Hk * D), rand(T, Hk * D), rand(T, H * D)
    g = -0.1 * torch.rand(T, H, generator=gen, device=DEV)
    beta = torch.rand(T, H, generator=gen, device=DEV)
    pool = torch.zeros(B, H, D, D, device=DEV)
    out = la.delta_extend(q, k, v, g, beta, pool, _i32(list(range(B))), _cu([n] * B), _mask(B),
                          max_seqlen=n, qk_l2norm=True)
    la.poll_error()
    for b in (0, 255, 511):
        r = slice(b * n, (b + 1) * n)
        p = torch.zeros(1, H, D, D, device=DEV)
        o = la.delta_extend(q[r], k[r], v[r], g[r], beta[r], p, _i32([0]), _cu([n]), _mask(1),
                            max_seqlen=n, qk_l2norm=True)
        la.poll_error()
        assert torch.equal(o, out[r]) and torch.equal(p[0], pool[b]), b


@pytest.mark.parametrize("B", [700, 8200])
def test_large_batches(B):
    """Several CTAs rank the batch; above 8,192 requests it runs in index order."""
    r = np.random.default_rng(39)
    lens = [int(x) for x in r.integers(0, 5, B)]
    lens[B // 2] = 200
    H = 1
    d = inputs(sum(lens), 1, H, 39)
    pool = torch.full((B, H, D, D), float("nan"), device=DEV)
    out = la.delta_extend(*_to(*d), pool, _i32(list(range(B))), _cu(lens), _mask(B), max_seqlen=200,
                          qk_l2norm=True)
    la.poll_error()
    cu = np.cumsum([0] + lens)
    for b in [0, 1, 2, 127, 128, B // 2, B - 2, B - 1] + [int(x) for x in r.integers(0, B, 30)]:
        x = slice(int(cu[b]), int(cu[b + 1]))
        o, S, norms = run_states(*[y[x] for y in d], np.zeros((H, D, D)), 1, H, True)
        check_out(f64(out[x]), o, d[0][x], np.broadcast_to(norms, (lens[b], H)), TOL_EXTEND, 1, H, True, str(b))
        check_states(f64(pool[b]), S, TOL_EXTEND, str(b))
    assert torch.isfinite(pool).all() and torch.isfinite(out).all()


def test_faults_in_a_planned_batch():
    """A long request among many short ones; some with a slot out of range or longer than max_seqlen
    are skipped and reported, and the others are as without them."""
    lens, H = [64] * 39 + [2400] + [100] * 10, 2
    B = len(lens)
    d = _to(*inputs(sum(lens), 1, H, 42))
    slots = list(range(B))
    want = []
    for bad, most in (([], 2400), ([0, 39, 45], 2400), ([], 2399)):
        pool = torch.full((B, H, D, D), 0.01, device=DEV)
        out = torch.full((sum(lens), H * D), 7.0, dtype=torch.bfloat16, device=DEV)
        la.delta_extend(*d, pool, _i32([B if b in bad else slots[b] for b in range(B)]), _cu(lens),
                        _mask(B, 1), out=out, max_seqlen=most, qk_l2norm=True)
        skipped = bad if most == 2400 else [39]
        if skipped:
            with pytest.raises(la.LAError) as e:
                la.poll_error()
            assert e.value.status == 5
        la.poll_error()
        if not want:
            want = [out, pool]
        cu = np.cumsum([0] + lens)
        for b in range(B):
            r = slice(int(cu[b]), int(cu[b + 1]))
            if b in skipped:
                assert (out[r] == 7.0).all() and (pool[b] == 0.01).all()
            elif lens[b] < 1000 or most == 2400:
                same = torch.equal(out[r], want[0][r]) and torch.equal(pool[b], want[1][b])
                assert same, f"request {b}, bad {bad}"


def test_planned_calls_are_bit_equal():
    lens, H = [33] * 60 + [1900, 2300], 2
    B = len(lens)
    d = _to(*inputs(sum(lens), 1, H, 43))
    got = []
    for _ in range(3):
        pool = torch.zeros(B, H, D, D, device=DEV)
        got.append((la.delta_extend(*d, pool, _i32(list(range(B))), _cu(lens), _mask(B), max_seqlen=2300,
                                    qk_l2norm=True), pool))
    la.poll_error()
    for o, p in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(p, got[0][1])


def test_nan_gates_stay_within_their_request():
    lens, H = [40, 50, 70], 2
    d = inputs(160, 1, H, 40)
    d[3][60] = float("nan")     # g
    d[4][50] = float("nan")     # beta
    d[3][61] = float("inf")
    clean = inputs(160, 1, H, 40)
    outs, pools = [], []
    for x in (clean, d):
        pool = torch.full((3, H, D, D), 0.02, device=DEV)
        outs.append(la.delta_extend(*_to(*x), pool, _i32([0, 1, 2]), _cu(lens), _mask(3, 1), max_seqlen=70,
                                    qk_l2norm=True))
        pools.append(pool)
    la.poll_error()
    for b, x in ((0, slice(0, 40)), (2, slice(90, 160))):
        assert torch.equal(outs[0][x], outs[1][x]) and torch.equal(pools[0][b], pools[1][b])
    assert pools[1][1].isnan().all()
    # the same rows as three requests' decode and verify calls: row 60's request only
    rows = [x[59:62] for x in d]
    pool = torch.full((3, H, D, D), 0.02, device=DEV)
    o = la.delta_decode(*_to(*rows), pool, _i32([0, 1, 2]), qk_l2norm=True)
    la.poll_error()
    assert torch.isfinite(o[0]).all() and o[1].isnan().all() and torch.isfinite(pool[0]).all()


@pytest.mark.parametrize("lens,bad", [([70] * 120, range(0, 120, 3)), ([64] * 30 + [2600] + [90] * 30, [30, 7]),
                                      ([2600, 130], [0])])
def test_nan_requests_among_others(lens, bad):
    """Many waves, a planned batch and a split one: requests full of NaN leave the others bit for bit."""
    H, B = 2, len(lens)
    cu = np.cumsum([0] + lens)
    outs, pools = [], []
    for poison in (False, True):
        d = inputs(sum(lens), 1, H, 44)
        if poison:
            for b in bad:
                for x in d:
                    x[cu[b]:cu[b + 1]] = float("nan")
        pool = torch.full((B, H, D, D), 0.02, device=DEV)
        outs.append(la.delta_extend(*_to(*d), pool, _i32(list(range(B))), _cu(lens), _mask(B, 1),
                                    max_seqlen=max(lens), qk_l2norm=True))
        pools.append(pool)
    la.poll_error()
    for b in range(B):
        r = slice(int(cu[b]), int(cu[b + 1]))
        if b in bad:
            assert outs[1][r].isnan().all() and pools[1][b].isnan().all()
        else:
            assert torch.equal(outs[0][r], outs[1][r]) and torch.equal(pools[0][b], pools[1][b]), b


def test_keys_nearly_the_same():
    """Keys within 8 degrees of one another, beta near 1, no decay: every token rewrites what the last
    one wrote.  A chunk's errors of u = v - S^T k then add up along one direction: 64 tokens, each of
    three pair roundings (R, T', u) of at most 2^-16 / sqrt(3) in the mean, of values of about sqrt(2)
    of the state's norm: 8 sqrt(2) 2^-16, below 12 x 2^-16."""
    n, H = 300, 2
    gen = torch.Generator().manual_seed(41)
    base = torch.randn(1, D, generator=gen)
    k = (base + 0.1 * torch.randn(n, D, generator=gen)).bfloat16()
    q = (base + torch.randn(n, D, generator=gen)).bfloat16()
    v = torch.randn(n, H * D, generator=gen).bfloat16()
    g, beta = torch.zeros(n, H), 0.98 + 0.02 * torch.rand(n, H, generator=gen)
    d = (q, k, v, g, beta)
    pool = torch.full((1, H, D, D), SENTINEL, device=DEV)
    out = la.delta_extend(*_to(*d), pool, _i32([0]), _cu([n]), _mask(1), qk_l2norm=True)
    la.poll_error()
    o, S, norms = run_states(*d, np.zeros((H, D, D)), 1, H, True)
    check_states(f64(pool[0]), S, 12 * TOL_EXTEND, "same keys")
    check_out(f64(out), o, q, np.broadcast_to(norms, (n, H)), 12 * TOL_EXTEND, 1, H, True, "same keys")
