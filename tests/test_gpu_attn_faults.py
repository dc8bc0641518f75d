"""Faults in the lists of attention calls: what is sound is right, what is not is left as it was, and it is reported."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from attn_testutil import D, SCALE, TOL_BF16, Cache, check, f64, i32, queries
from oracle import attn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def faulty():
    with pytest.raises(la.LAError) as e:
        la.poll_error()
    assert e.value.status == 5
    la.poll_error()


@pytest.mark.parametrize("width", [16, 40])  # whole items, and items that may be cut
def test_extend_with_a_bound_of_no_tokens(width):
    H, n = 2, 8
    cache = Cache([100], 1, 16, 4, width=width)
    q = queries(n, H, 4).to(DEV)
    kp, vp, table, kv = cache.to(DEV)
    out = torch.full((n, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    la.attn_extend(q, kp, vp, table, i32([0, n]).to(DEV), kv, out=out, max_seqlen=0)
    faulty()
    assert (out == 77.0).all()
    la.attn_extend(q, kp, vp, table, i32([0, 0]).to(DEV), kv, out=out, max_seqlen=0)  # rows of no request
    la.poll_error()
    assert (out == 77.0).all()


@pytest.mark.parametrize("given", [False, True])
def test_commit_leaves_no_length_unset(given):
    """Without new_lens a skipped request gets the length that it has; with it, what stands there."""
    lens, N = [60, 61, 30], 5
    cache = Cache(lens, 2, 16, 6)
    kp, vp, table, kv = cache.to(DEV)
    parents, accept = i32([[-1, 0, 1, 2, 2]] * 3).to(DEV), i32([3, N, -1]).to(DEV)
    stale = torch.full((3,), 1 << 30, dtype=torch.int32, device=DEV)
    if given:
        lens_out = la.kv_commit(kp, vp, table, kv, parents, accept, new_lens=stale)
    else:
        del stale  # memory of this size that holds something
        lens_out = la.kv_commit(kp, vp, table, kv, parents, accept)
    faulty()
    assert lens_out.tolist() == [59, 1 << 30 if given else 61, 25]
    assert kv.tolist() == lens


def expect(cache, b, q, n, H, seen, tol, got, what):
    k, v = cache.rows(b)
    want, size = attn.attend(f64(q).reshape(n, H, D), k, v, seen, SCALE)
    check(f64(got), want, size, tol, what)


@pytest.mark.parametrize("cu", [[0, 40, 30, 143], [0, 40, 200, 143], [-1, 40, 110, 143], [0, 40, 110, 144], [0, 143, 143, 0]])
@pytest.mark.parametrize("lens,width", [([300, 300, 300], 40), ([200, 256, 150], 16)])  # cut and whole
def test_extend_with_bad_cu_seqlens(cu, lens, width):
    """Requests whose rows fit are right, where no other claims their rows too; rows of no such request, and what lies
    around out, are left as they were."""
    H, Hkv, T, B = 4, 2, 143, 3
    cache = Cache(lens, Hkv, 16, 4, width=width)
    q = queries(T, H, 4)
    kp, vp, table, kv = cache.to(DEV)
    around = torch.full((T + 512, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    out = around[256:256 + T]
    la.attn_extend(q.to(DEV), kp, vp, table, i32(cu).to(DEV), kv, out=out, max_seqlen=T)
    faulty()
    claims = np.zeros(T, int)
    sound = [b for b in range(B) if 0 <= cu[b] <= cu[b + 1] <= T]
    assert 0 < len(sound) < B
    for b in sound:
        claims[cu[b]:cu[b + 1]] += 1
    got = f64(out).reshape(T, H, D)
    for b in sound:
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k, v = cache.rows(b)
        r = slice(cu[b], cu[b + 1])
        want, size = attn.attend(f64(q[r]).reshape(n, H, D), k, v, attn.causal(n, lens[b]), SCALE)
        alone = claims[r] == 1
        check(got[r][alone], want[alone], size[alone], TOL_BF16, f"request {b}")
    assert (got[claims == 0] == 77.0).all()
    assert (around[:256] == 77.0).all() and (around[256 + T:] == 77.0).all()


WIDE = [([100, 700, 40, 1000], 32), ([100, 256, 40, 131], 8)]  # items that may be cut, whole ones; pages of 32


def _wide_parents(N, B, seed):
    rng = np.random.default_rng(seed)
    return [[int(rng.integers(max(-1, t - 4), t)) for t in range(N)] for _ in range(B)]


@pytest.mark.parametrize("bad", ["page", "long", "negative", "short", "parent_high", "parent_low", "parent_self"])
@pytest.mark.parametrize("lens,width", WIDE)
def test_wide_tree_skips_faulty_requests(bad, lens, width):
    """More rows to a kv head (80) than the kernel of few rows takes."""
    H, Hkv, N, B = 8, 2, 20, len(lens)
    cache = Cache(lens, Hkv, 32, 5, width=width)
    q = queries(B * N, H, 5)
    parents = _wide_parents(N, B, 5)
    kp, vp, table, kv = cache.to(DEV)
    par = i32(parents).to(DEV)
    if bad == "page":
        table[1, 2] = 1 << 29
    elif bad.startswith("parent"):
        par[1, 13] = {"parent_high": 14, "parent_low": -2, "parent_self": 13}[bad]
    else:
        kv[1] = {"long": width * 32 + 1, "negative": -5, "short": N - 1}[bad]
    around = torch.full((B * N + 256, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    out = around[128:128 + B * N]
    la.attn_verify_tree(q.to(DEV), kp, vp, table, kv, par, N, out=out)
    faulty()
    for b in (0, 2, 3):
        r = slice(b * N, (b + 1) * N)
        expect(cache, b, q[r], N, H, attn.tree(parents[b], lens[b]), TOL_BF16, out[r], f"request {b}")
    if bad != "page":
        assert (out[N:2 * N] == 77.0).all()
    assert (around[:128] == 77.0).all() and (around[128 + B * N:] == 77.0).all()


@pytest.mark.parametrize("width", [40, 8])
@pytest.mark.parametrize("N,H", [(20, 8), (1, 136)])  # trees, and single tokens of 68 heads to a kv head
def test_wide_calls_captured_and_replayed_with_other_lengths(N, H, width):
    Hkv, P, B, pages = 2, 32, 4, 200
    top = width * P
    sets = [[top, N + 3, 0, N + 90], [N, top - 1, N + 60, N], [0, 0, 0, 0], [N, N, N, top]]
    kp = torch.zeros(pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    vp, q = torch.zeros_like(kp), torch.zeros(B * N, H * D, dtype=torch.bfloat16, device=DEV)
    table, kv = torch.zeros(B, width, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    par, out = torch.zeros(B, N, dtype=torch.int32, device=DEV), torch.zeros_like(q)

    def call():
        if N == 1:
            la.attn_decode(q, kp, vp, table, kv, out=out)
        else:
            la.attn_verify_tree(q, kp, vp, table, kv, par, N, out=out)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for s, lens in enumerate(sets):
        cache = Cache(lens, Hkv, P, s, width=width)
        E = cache.both.shape[0]
        kp[:E], vp[:E] = cache.both[:, 0].to(DEV), cache.both[:, 1].to(DEV)
        table.copy_(cache.table.to(DEV))
        kv.copy_(cache.kv)
        parents, hq = _wide_parents(N, B, s), queries(B * N, H, s)
        par.copy_(i32(parents))
        q.copy_(hq)
        out.fill_(77.0)
        graph.replay()
        first = out.clone()
        la.poll_error()
        for b in range(B):
            r = slice(b * N, (b + 1) * N)
            if lens[b] == 0:
                assert (first[r] == 0).all()
            else:
                expect(cache, b, hq[r], N, H, attn.tree(parents[b], lens[b]), TOL_BF16, first[r], f"{s}, request {b}")
        graph.replay()
        assert torch.equal(out, first)


@pytest.mark.parametrize("bad", ["page", "long", "negative", "short", "accept_high", "accept_low", "parent"])
def test_commit_keeps_the_length_of_a_skipped_request(bad):
    lens, N = [60, 61, 0], 5
    cache = Cache(lens, 2, 16, 6)
    kp, vp, table, kv = cache.to(DEV)
    parents, accept = i32([[-1, -1, 1, 2, 2]] * 3).to(DEV), i32([4, 4, 4]).to(DEV)
    if bad == "page":
        table[1, 3] = -1
    elif bad == "parent":
        parents[1, 2] = 2
    elif bad.startswith("accept"):
        accept[1] = N if bad == "accept_high" else -2
    else:
        kv[1] = {"long": table.shape[1] * 16 + 1, "negative": -1, "short": N - 1}[bad]
    before = kv.tolist()
    assert la.kv_commit(kp, vp, table, kv, parents, accept).tolist() == [58, before[1], 0]
    faulty()
