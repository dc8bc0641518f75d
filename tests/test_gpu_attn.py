"""Softmax attention over a paged cache on the GPU (la_attn_extend, la_attn_decode, la_attn_verify_tree, la_kv_commit)
against the fp64 oracle: lengths, head layouts, page sizes, strides, trees, empty requests, garbage behind a
request's positions, device-detected faults, captured and concurrent calls."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from attn_testutil import D, SCALE, TOL_BF16, TOL_PAIR, Cache, check, f64, i32, queries
from oracle import attn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _strided(q, extra=16):
    wide = torch.full((q.shape[0], q.shape[1] + extra), float("nan"), dtype=q.dtype)
    wide[:, :q.shape[1]] = q
    return wide.to(DEV)[:, :q.shape[1]]


def check_extend(new, old, H, Hkv, P=64, seed=0, gap=0, tail=0, spread=2.0, scale=None, strided=False,
                 alternate=False, max_seqlen=None, max_kvlen=None, workspace=None):
    cache = Cache([n + m for n, m in zip(new, old)], Hkv, P, seed, alternate=alternate)
    T = gap + sum(new) + tail
    q = queries(T, H, seed, spread)
    q[:gap] = float("nan")
    q[gap + sum(new):] = float("nan")
    cu = i32(np.cumsum([gap] + list(new)).tolist())
    out = torch.full((T, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    kp, vp, table, kv = cache.to(DEV)
    got = la.attn_extend(_strided(q) if strided else q.to(DEV), kp, vp, table, cu.to(DEV), kv, out=out, scale=scale,
                         max_seqlen=max(new) if max_seqlen is None else max_seqlen, max_kvlen=max_kvlen,
                         workspace=workspace)
    la.poll_error()
    assert got is out
    o = f64(out)
    for b, n in enumerate(new):
        if n == 0:
            continue
        r = slice(int(cu[b]), int(cu[b + 1]))
        k, v = cache.rows(b)
        want, size = attn.attend(f64(q[r]).reshape(n, H, D), k, v, attn.causal(n, n + old[b]),
                                 SCALE if scale is None else scale)
        check(o[r], want, size, TOL_BF16, f"request {b} of {new} + {old}")
    assert (out[:gap] == 77.0).all() and (out[gap + sum(new):] == 77.0).all()
    return out


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257, 400])
def test_extend_lengths(n):
    check_extend([n], [0], 4, 2, seed=n)


@pytest.mark.parametrize("old", [1, 63, 64, 127, 128, 129, 300, 1000])
def test_extend_prefixes(old):
    check_extend([37], [old], 4, 1, seed=old)
    check_extend([1, 130], [old, old + 5], 2, 2, P=16, seed=old)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (12, 2), (7, 7), (16, 1), (48, 2), (128, 1)])
def test_extend_heads(H, Hkv):
    check_extend([70, 1, 0, 45], [0, 200, 3, 10], H, Hkv, seed=H)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("alternate", [False, True])
def test_extend_pages(P, alternate):
    check_extend([100, 257, 5], [0, 31, 140], 8, 2, P=P, seed=P, alternate=alternate, strided=alternate)


def test_extend_rows_outside_requests():
    check_extend([37, 90, 64], [0, 5, 0], 4, 2, gap=5, tail=70, seed=6)


@pytest.mark.parametrize("spread,scale", [(2.0, None), (0.01, None), (2.0, 0.02), (1.0, 0.5)])
def test_extend_scores(spread, scale):
    check_extend([300], [100], 2, 1, seed=8, spread=spread, scale=scale)


@pytest.mark.parametrize("new,old,H,Hkv", [([1], [4000], 4, 1), ([1, 1, 1], [300, 9000, 0], 4, 2), ([700, 5], [2000, 700], 12, 2),
                                           ([33] * 40, [0, 500, 129, 1000] * 10, 8, 2), ([3000], [0], 6, 2),
                                           ([130, 0, 257, 64] * 6, [0, 5, 300, 64] * 6, 16, 4)])
def test_extend_runs(new, old, H, Hkv):
    """Batches whose items are cut at the ends of the CTAs' runs, into two pieces and into many."""
    check_extend(new, old, H, Hkv, P=16, seed=len(new), tail=3)


def test_extend_split_and_whole():
    """Few rows over many keys run split; without scratch for that the same call runs whole."""
    new, old = [3, 40], [3000, 1200]
    assert la.attn_extend_workspace_size(2, 43, 8, 2, D, 40, 3040) > 0
    a = check_extend(new, old, 8, 2, seed=9)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    b = check_extend(new, old, 8, 2, seed=9, workspace=none)
    assert (a.float() - b.float()).abs().max() <= 2 * 2.0 ** -7 * b.float().abs().max()


def check_verify(lens, N, H, Hkv, P=64, seed=0, parents=None, strided=False, alternate=False, scale=None, width=None,
                 spread=2.0):
    """N == 0: decode.  lens: positions of each request, its drafts among them (0: an empty request)."""
    cache = Cache(lens, Hkv, P, seed, alternate=alternate, width=width)
    B, n = len(lens), max(N, 1)
    q = queries(B * n, H, seed, spread)
    kp, vp, table, kv = cache.to(DEV)
    dq = _strided(q) if strided else q.to(DEV)
    out = torch.full((B * n, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    if N == 0:
        got = la.attn_decode(dq, kp, vp, table, kv, out=out, scale=scale)
        parents = [[-1]] * B
    else:
        if parents is None:
            rng = np.random.default_rng(seed)
            parents = [[int(rng.integers(max(-1, t - 4), t)) for t in range(N)] for _ in range(B)]
        got = la.attn_verify_tree(dq, kp, vp, table, kv, i32(parents).to(DEV), N, out=out, scale=scale)
    la.poll_error()
    assert got is out
    o, G = f64(out).reshape(B, n, H, D), H // Hkv
    tol = TOL_PAIR if n * G <= 64 else TOL_BF16
    for b in range(B):
        if lens[b] == 0:
            assert (o[b] == 0).all()
            continue
        k, v = cache.rows(b)
        want, size = attn.attend(f64(q[b * n:(b + 1) * n]).reshape(n, H, D), k, v, attn.tree(parents[b], lens[b]),
                                 SCALE if scale is None else scale)
        check(o[b], want, size, tol, f"request {b}, {lens[b]} positions")
    return out


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 300, 1000])
def test_decode_lengths(n):
    check_verify([n], 0, 4, 2, seed=n)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (8, 1), (16, 1), (17, 1), (12, 2), (40, 1), (64, 1), (66, 1),
                                   (128, 1), (7, 7)])
def test_decode_heads(H, Hkv):
    check_verify([200, 1, 0, 129, 700], 0, H, Hkv, seed=H)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("alternate", [False, True])
def test_decode_pages(P, alternate):
    check_verify([100, 257, 5, 1400], 0, 8, 2, P=P, seed=P, alternate=alternate, strided=alternate)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1] * 300, [5000, 3, 0, 1, 800] * 8, [20000], [200, 1, 64, 1000] * 40])
@pytest.mark.parametrize("short", [True, False])
def test_decode_batches(lens, short):
    """Page tables that hold up to 1,280 positions and more: two CTAs an SM, or one."""
    check_verify(lens, 0, 4, 2, P=16, seed=len(lens), width=max(1, -(-max(lens) // 16)) if short else 81 + max(lens) // 16)


@pytest.mark.parametrize("N", [1, 2, 5, 8, 16, 17, 33, 64, 100, 128])
def test_tree_sizes(N):
    check_verify([N, N + 1, N + 77, N + 500, 0], N, 4, 2, seed=N)


@pytest.mark.parametrize("N,H,Hkv", [(8, 16, 2), (16, 16, 1), (5, 10, 1), (3, 128, 1), (128, 6, 2), (7, 20, 1), (9, 30, 2)])
def test_tree_heads(N, H, Hkv):
    check_verify([N + 60, N, N + 300, 0, N + 1, 1500], N, H, Hkv, P=16, seed=N)


def test_tree_shapes():
    chain, star = [[t - 1 for t in range(12)]], [[-1] * 12]
    for parents in (chain, star):
        check_verify([140], 12, 4, 1, seed=3, parents=parents)


@pytest.mark.parametrize("spread,scale", [(0.01, None), (2.0, 0.02), (1.0, 0.5)])
def test_verify_scores(spread, scale):
    check_verify([1000, 300], 6, 8, 2, seed=4, spread=spread, scale=scale)
    check_verify([1000, 300], 0, 8, 2, seed=4, spread=spread, scale=scale)


def test_rising_scores():
    """Keys that grow along the context: the reference has to follow again and again."""
    P, L, H = 64, 900, 4
    cache = Cache([L], 1, P, 3)
    at = torch.arange(L)
    ramp = torch.exp(torch.linspace(-4, 2.5, L))[:, None]
    q = torch.ones(1, H * D).bfloat16()
    k = (torch.ones(L, D) * ramp).bfloat16()
    pages = cache.table[0].long()[at // P]
    cache.both[pages, 0, 0, at % P] = k
    kp, vp, table, kv = cache.to(DEV)
    kk, vv = cache.rows(0)
    want, size = attn.attend(f64(q).reshape(1, H, D), kk, vv, np.ones((1, L), bool), SCALE)
    o1 = la.attn_decode(q.to(DEV), kp, vp, table, kv)
    o2 = la.attn_extend(q.to(DEV), kp, vp, table, i32([0, 1]).to(DEV), kv)
    la.poll_error()
    # scores up to 138: fp32 sums of 128 equal products are off by 128 * 2^-23 of that, twice for the quotient
    room = 2 * 138 * 2.0 ** -16
    check(f64(o1), want, size, room + TOL_PAIR, "decode")
    check(f64(o2), want, size, room + TOL_BF16, "extend")


def test_rising_scores_of_a_prompt():
    """The same for the rows of a prompt, whose references follow at different tiles; the second head sees none rise."""
    P, L, n, H = 64, 900, 300, 2
    cache = Cache([L], 1, P, 4)
    at = torch.arange(L)
    ramp = torch.exp(torch.linspace(-4, 2.5, L))[:, None]
    pages = cache.table[0].long()[at // P]
    cache.both[pages, 0, 0, at % P] = (torch.ones(L, D) * ramp).bfloat16()
    q = torch.ones(n, H, D)
    q[:, 1] = -1.0
    q = q.reshape(n, H * D).bfloat16()
    kp, vp, table, kv = cache.to(DEV)
    out = la.attn_extend(q.to(DEV), kp, vp, table, i32([0, n]).to(DEV), kv)
    la.poll_error()
    kk, vv = cache.rows(0)
    want, size = attn.attend(f64(q).reshape(n, H, D), kk, vv, attn.causal(n, L), SCALE)
    check(f64(out), want, size, 2 * 138 * 2.0 ** -16 + TOL_BF16, "extend")


@pytest.mark.parametrize("B", [31, 33, 512, 513, 1100])
def test_many_requests(B):
    """Batches that end before, at and behind the groups in which the requests' work is summed."""
    rng = np.random.default_rng(B)
    new, old = rng.integers(0, 6, B).tolist(), rng.integers(0, 40, B).tolist()
    check_extend(new, old, 4, 2, P=16, seed=B, tail=2)
    for width in (4, 17):  # requests of up to 256 positions stay whole
        check_verify([int(x) for x in rng.integers(0, 60, B)], 0, 4, 2, P=16, seed=B, width=width)
        check_verify([int(x) if x > 5 else 0 for x in rng.integers(0, 60, B)], 5, 32, 2, P=16, seed=B, width=width)


@pytest.mark.parametrize("N,H", [(0, 16), (0, 40), (3, 32), (8, 16)])
def test_whole_requests(N, H):
    """Requests of one tile of keys and of two, more and fewer than CTAs, with empty ones among them."""
    for lens in ([256], [200, 0, 9, 256, 129, 128], [256, 20, 127, 255] * 90):
        check_verify(lens, N, H, 2, P=16, seed=len(lens), width=16)


def check_commit(lens, N, Hkv, P, accept, seed=0, in_place=False):
    rng = np.random.default_rng(seed)
    B = len(lens)
    cache = Cache(lens, Hkv, P, seed)
    parents = [[int(rng.integers(max(-1, t - 4), t)) for t in range(N)] for _ in range(B)]
    kp, vp, table, kv = cache.to(DEV)
    got = la.kv_commit(kp, vp, table, kv, i32(parents).to(DEV), i32(accept).to(DEV), new_lens=kv if in_place else None)
    la.poll_error()
    want = cache.both.clone()
    for b in range(B):
        p = attn.path(parents[b], accept[b]) if lens[b] else []
        ctx = lens[b] - N if lens[b] else 0
        assert int(got[b]) == ctx + len(p)
        src = cache.both.clone()
        for i, t in enumerate(p):
            s, d = ctx + t, ctx + i
            want[int(cache.table[b, d // P]), :, :, d % P] = src[int(cache.table[b, s // P]), :, :, s % P]
    both = torch.stack([kp, vp], 1).cpu()
    assert torch.equal(both.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("N,Hkv,P", [(1, 1, 16), (5, 2, 16), (16, 8, 64), (33, 9, 32), (128, 3, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(N, Hkv, P, in_place):
    lens = [N, N + 13, 0, N + 200, N + 1]
    check_commit(lens, N, Hkv, P, [N - 1, -1, -1, N // 2, N - 1], seed=N, in_place=in_place)
