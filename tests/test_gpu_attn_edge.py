"""Calls of the rotary, cache and attention operators that users make in odd ways: faults found on the device, values
that are not finite, graphs captured and replayed with other lengths, other streams, shared pages, places past 32
bits, waits that run out, and a run of all of them as a hybrid model makes it."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from attn_testutil import D, SCALE, TOL_BF16, TOL_PAIR, Cache, check, f64, i32, queries
from oracle import attn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _faulty():
    with pytest.raises(la.LAError) as e:
        la.poll_error()
    assert e.value.status == 5
    la.poll_error()


def _expect(cache, b, q, n, H, seen, tol, got, what):
    k, v = cache.rows(b)
    want, size = attn.attend(f64(q).reshape(n, H, D), k, v, seen, SCALE)
    check(f64(got), want, size, tol, what)


@pytest.mark.parametrize("bad", ["page_high", "page_low", "long", "negative", "short"])
def test_extend_skips_faulty_requests(bad):
    H, Hkv, new, old = 4, 2, [40, 70, 33], [10, 200, 300]
    cache = Cache([a + b for a, b in zip(new, old)], Hkv, 16, 3)
    q = queries(sum(new), H, 3)
    cu = i32(np.cumsum([0] + new).tolist())
    kp, vp, table, kv = cache.to(DEV)
    if bad.startswith("page"):
        table[1, 2] = kp.shape[0] if bad == "page_high" else -1
    else:
        kv[1] = {"long": table.shape[1] * 16 + 1, "negative": -1, "short": new[1] - 1}[bad]
    out = torch.full((sum(new), H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    la.attn_extend(q.to(DEV), kp, vp, table, cu.to(DEV), kv, out=out, max_seqlen=max(new))
    _faulty()
    for b in (0, 2):
        r = slice(int(cu[b]), int(cu[b + 1]))
        _expect(cache, b, q[r], new[b], H, attn.causal(new[b], new[b] + old[b]), TOL_BF16, out[r], f"request {b}")
    if not bad.startswith("page"):
        assert (out[int(cu[1]):int(cu[2])] == 77.0).all()


@pytest.mark.parametrize("cu", [[0, 40, 30, 143], [0, 40, 200, 143], [-1, 40, 110, 143], [0, 40, 110, 144]])
def test_extend_bad_cu_seqlens(cu):
    """Requests whose rows do not fit are skipped; nothing is read or written outside."""
    H, Hkv = 4, 2
    cache = Cache([300, 300, 300], Hkv, 16, 4)
    q = queries(143, H, 4).to(DEV)
    kp, vp, table, kv = cache.to(DEV)
    out = torch.full((143, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    la.attn_extend(q, kp, vp, table, i32(cu).to(DEV), kv, out=out, max_seqlen=143)
    _faulty()


def test_extend_longer_than_max_seqlen():
    cache = Cache([40, 41], 1, 16, 4)
    q = queries(81, 2, 4)
    kp, vp, table, kv = cache.to(DEV)
    out = torch.full((81, 2 * D), 77.0, dtype=torch.bfloat16, device=DEV)
    la.attn_extend(q.to(DEV), kp, vp, table, i32([0, 40, 81]).to(DEV), kv, out=out, max_seqlen=40)
    _faulty()
    assert (out[40:] == 77.0).all()
    _expect(cache, 0, q[:40], 40, 2, attn.causal(40, 40), TOL_BF16, out[:40], "request 0")


@pytest.mark.parametrize("bad", ["page", "long", "negative", "short", "parent_high", "parent_low", "parent_self"])
def test_tree_skips_faulty_requests(bad):
    H, Hkv, N, lens = 8, 2, 6, [100, 700, 40, 1000]
    cache = Cache(lens, Hkv, 32, 5)
    q = queries(len(lens) * N, H, 5)
    parents = [[-1, 0, 0, 1, 3, -1]] * len(lens)
    kp, vp, table, kv = cache.to(DEV)
    par = i32(parents).to(DEV)
    if bad == "page":
        table[1, 2] = 1 << 29
    elif bad.startswith("parent"):
        par[1, 3] = {"parent_high": 4, "parent_low": -2, "parent_self": 3}[bad]
    else:
        kv[1] = {"long": table.shape[1] * 32 + 1, "negative": -5, "short": N - 1}[bad]
    out = torch.full((len(lens) * N, H * D), 77.0, dtype=torch.bfloat16, device=DEV)
    la.attn_verify_tree(q.to(DEV), kp, vp, table, kv, par, N, out=out)
    _faulty()
    for b in (0, 2, 3):
        r = slice(b * N, (b + 1) * N)
        _expect(cache, b, q[r], N, H, attn.tree(parents[b], lens[b]), TOL_PAIR, out[r], f"request {b}")
    if bad != "page":
        assert (out[N:2 * N] == 77.0).all()


@pytest.mark.parametrize("bad", ["page", "long", "negative", "accept_high", "accept_low", "parent"])
def test_commit_skips_faulty_requests(bad):
    Hkv, N, lens = 2, 5, [60, 61, 5]
    cache = Cache(lens, Hkv, 16, 6)
    kp, vp, table, kv = cache.to(DEV)
    parents, accept = i32([[-1, -1, 1, 2, 2]] * 3).to(DEV), i32([4, 4, 4]).to(DEV)
    if bad == "page":
        table[1, 3] = -1
    elif bad == "parent":
        parents[1, 2] = 2
    elif bad.startswith("accept"):
        accept[1] = N if bad == "accept_high" else -2
    else:
        kv[1] = table.shape[1] * 16 + 1 if bad == "long" else -1
    lens_out = torch.full((3,), 99, dtype=torch.int32, device=DEV)
    la.kv_commit(kp, vp, table, kv, parents, accept, new_lens=lens_out)
    _faulty()
    assert lens_out.tolist() == [58, 99, 3]
    both = torch.stack([kp, vp], 1).cpu()
    for b in range(3):
        ctx = lens[b] - N
        for i, t in enumerate([1, 2, 4] if b != 1 else []):
            at = lambda x: (int(cache.table[b, x // 16]), slice(None), slice(None), x % 16)  # noqa: E731
            assert torch.equal(both[at(ctx + i)], cache.both[at(ctx + t)])
    for j in range(table.shape[1]):  # the faulty request's pages are as they were
        e = int(cache.table[1, j])
        if e < kp.shape[0]:
            assert torch.equal(both[e].view(torch.int16), cache.both[e].view(torch.int16))


def test_non_finite_values_stay_in_their_request():
    H, Hkv, lens, new = 4, 2, [150, 300, 90], [20, 300, 90]
    cache = Cache(lens, Hkv, 16, 7)
    clean = cache.both.clone()
    for i, x in enumerate((float("nan"), float("inf"), -float("inf"))):
        cache.both[int(cache.table[1, 3 + i]), i % 2, :, 5] = x
    q = queries(sum(new), H, 7)
    q[new[0] + 17] = float("nan")
    cu = i32(np.cumsum([0] + new).tolist())
    kp, vp, table, kv = cache.to(DEV)
    out = la.attn_extend(q.to(DEV), kp, vp, table, cu.to(DEV), kv, max_seqlen=300)
    one = torch.stack([q[new[0] - 1], q[new[0] + 17], q[-1]])
    dec = la.attn_decode(one.to(DEV), kp, vp, table, kv)
    la.poll_error()
    assert not torch.equal(cache.both.view(torch.int16), clean.view(torch.int16))
    for b in (0, 2):
        r = slice(int(cu[b]), int(cu[b + 1]))
        _expect(cache, b, q[r], new[b], H, attn.causal(new[b], lens[b]), TOL_BF16, out[r], f"extend {b}")
        _expect(cache, b, one[b:b + 1], 1, H, np.ones((1, lens[b]), bool), TOL_PAIR, dec[b:b + 1], f"decode {b}")


def test_query_of_nan_reaches_its_own_row_and_head():
    H, Hkv, n = 6, 2, 200
    cache = Cache([n], Hkv, 64, 8)
    q = queries(n, H, 8)
    q[50, 2 * D:3 * D] = float("nan")
    kp, vp, table, kv = cache.to(DEV)
    out = la.attn_extend(q.to(DEV), kp, vp, table, i32([0, n]).to(DEV), kv)
    la.poll_error()
    bad = torch.isnan(out.float().cpu()).reshape(n, H, D)
    assert bad[50, 2].all() and int(bad.sum()) == D


@pytest.mark.parametrize("op", ["extend", "decode", "tree"])
def test_captured_and_replayed_with_other_lengths(op):
    """A graph's lengths, tables, rows and pages are read when it runs."""
    H, Hkv, P, B, N, width = 8, 2, 16, 4, 5, 80
    sets = [[700, 3 + N, 0, 90], [40, 1200, N + 60, N], [0, 0, 0, 0], [N, N, N, 1279]]
    n = {"extend": 64, "decode": B, "tree": B * N}[op]
    news = [[20, 3, 0, 41], [1, 1, 60, 2], [0, 0, 0, 0], [5, 5, 5, 49]]
    pages = 400
    kp = torch.zeros(pages, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    vp, q = torch.zeros_like(kp), torch.zeros(n, H * D, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    kv, cu = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    parents = [[-1, 0, 1, 0, -1]] * B
    par = i32(parents).to(DEV)
    out = torch.zeros(n, H * D, dtype=torch.bfloat16, device=DEV)

    def call():
        if op == "extend":
            la.attn_extend(q, kp, vp, table, cu, kv, out=out, max_seqlen=64)
        elif op == "decode":
            la.attn_decode(q, kp, vp, table, kv, out=out)
        else:
            la.attn_verify_tree(q, kp, vp, table, kv, par, N, out=out)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for s, (lens, new) in enumerate(zip(sets, news)):
        cache = Cache(lens, Hkv, P, s, width=width)
        E = cache.both.shape[0]
        kp[:E], vp[:E] = cache.both[:, 0].to(DEV), cache.both[:, 1].to(DEV)
        table.copy_(cache.table.to(DEV))
        kv.copy_(cache.kv)
        hq = queries(n, H, s)
        q.copy_(hq)
        cu.copy_(i32(np.cumsum([0] + new).tolist()))
        out.fill_(77.0)
        graph.replay()
        first = out.clone()
        la.poll_error()
        for b in range(B):
            if op == "extend":
                r = slice(int(cu[b]), int(cu[b + 1]))
                if new[b]:
                    _expect(cache, b, hq[r], new[b], H, attn.causal(new[b], lens[b]), TOL_BF16, out[r], f"{s}, request {b}")
                continue
            m = 1 if op == "decode" else N
            r = slice(b * m, (b + 1) * m)
            if lens[b] == 0:
                assert (out[r] == 0).all()
            else:
                seen = attn.tree(parents[b], lens[b]) if op == "tree" else np.ones((1, lens[b]), bool)
                _expect(cache, b, hq[r], m, H, seen, TOL_PAIR, out[r], f"{s}, request {b}")
        if op == "extend":
            assert (out[sum(new):] == 77.0).all()
        graph.replay()
        assert torch.equal(out, first)  # the same sums in the same order


def test_calls_on_two_streams_at_once():
    """Each call has scratch of its own where it is given none."""
    H, Hkv, lens = 8, 2, [3000, 9000]
    caches = [Cache([n], Hkv, 64, i) for i, n in enumerate(lens)]
    qs = [queries(40, H, i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    dev = [(qs[i].to(DEV),) + caches[i].to(DEV) for i in range(2)]
    cu = i32([0, 40]).to(DEV)
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                q, kp, vp, table, kv = dev[i]
                outs[i].append(la.attn_extend(q, kp, vp, table, cu, kv))
                outs[i].append(la.attn_decode(q[:1], kp, vp, table, kv))
    la.poll_error()
    for i in range(2):
        _expect(caches[i], 0, qs[i], 40, H, attn.causal(40, lens[i]), TOL_BF16, outs[i][0], f"extend {i}")
        for a, b in zip(outs[i][:2] * 4, outs[i][2:]):
            assert torch.equal(a, b)


def test_requests_that_share_pages():
    """Two requests with a common prefix in the same pages."""
    H, Hkv, P = 4, 2, 16
    cache = Cache([500, 330], Hkv, P, 9)
    cache.table[1, :20] = cache.table[0, :20]
    q = queries(2, H, 9)
    kp, vp, table, kv = cache.to(DEV)
    out = la.attn_decode(q.to(DEV), kp, vp, table, kv)
    la.poll_error()
    for b in range(2):
        _expect(cache, b, q[b:b + 1], 1, H, np.ones((1, cache.lens[b]), bool), TOL_PAIR, out[b:b + 1], f"request {b}")


def test_pages_past_32_bits():
    """Pages, rows of q and places of new keys more than 2^32 bytes (and 2^31 elements) from the start."""
    Hkv, P, H = 8, 128, 8
    stride = (1 << 24) + 8 * 128 * 128
    E = 160
    pool = torch.zeros(E * stride, dtype=torch.bfloat16, device=DEV)
    both = pool.as_strided((E, Hkv, P, D), (stride, P * D, D, 1))
    other = pool[Hkv * P * D:].as_strided((E, Hkv, P, D), (stride, P * D, D, 1))
    cache = Cache([300, 200], Hkv, P, 11, spare=0)
    far = torch.tensor([E - 1, E - 2, E - 3, E - 4, 0])
    for e in range(cache.both.shape[0]):
        both[int(far[e])] = cache.both[e, 0].to(DEV)
        other[int(far[e])] = cache.both[e, 1].to(DEV)
    used = cache.table < 1 << 20
    table = torch.where(used, far[cache.table.clamp(max=4).long()].int(), 0).int().to(DEV)
    q = queries(300, H, 11)
    out = la.attn_extend(q.to(DEV), both, other, table, i32([0, 200, 300]).to(DEV), cache.kv.to(DEV))
    dec = la.attn_decode(q[:2].to(DEV), both, other, table, cache.kv.to(DEV))
    la.poll_error()
    for b, r in ((0, slice(0, 200)), (1, slice(200, 300))):
        n = r.stop - r.start
        _expect(cache, b, q[r], n, H, attn.causal(n, cache.lens[b]), TOL_BF16, out[r], f"extend {b}")
        _expect(cache, b, q[b:b + 1], 1, H, np.ones((1, cache.lens[b]), bool), TOL_PAIR, dec[b:b + 1], f"decode {b}")
    k, v = queries(2, Hkv, 12), queries(2, Hkv, 13)
    none = torch.empty(0, dtype=torch.float64, device=DEV)
    la.kv_store(q[:2].to(DEV), k.to(DEV), v.to(DEV), i32([0, 1]).to(DEV), none, both, other,
                i32([(E - 1) * P + 127, (E - 5) * P + 3]).to(DEV))
    la.poll_error()
    assert torch.equal(both[E - 1, :, 127].flatten().cpu(), k[0]) and torch.equal(other[E - 5, :, 3].flatten().cpu(), v[1])


@pytest.mark.parametrize("op", ["extend", "decode", "tree"])
@pytest.mark.parametrize("lens,must", [([24] * 6000, True), ([20000, 300], False)])
def test_waits_that_run_out(op, lens, must):
    """With a limit of a microsecond a wait gives up (for the first item of thousands of requests it always does); the
    call ends, says so, and the next one is right."""
    H, Hkv, N, P = 8, 2, 4, 64
    B = len(lens)
    gen = torch.Generator().manual_seed(12)
    need = [-(-n // P) for n in lens]
    table = torch.zeros(B, max(need), dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(n) + (sum(need[:b]) if B < 10 else b)
    kp, vp = (torch.randn(sum(need), Hkv, P, D, generator=gen).bfloat16().to(DEV) for _ in range(2))
    table, kv = table.to(DEV), i32(lens).to(DEV)
    new = [4] * B if B > 10 else [300, 100]
    q = queries(sum(new), H, 12).to(DEV)
    par, cu = i32([[-1, 0, 1, 1]] * B).to(DEV), i32(np.cumsum([0] + new).tolist()).to(DEV)

    def call():
        if op == "extend":
            return la.attn_extend(q, kp, vp, table, cu, kv, max_seqlen=max(new))
        if op == "decode":
            return la.attn_decode(q[:B], kp, vp, table, kv)
        return la.attn_verify_tree(q[:B * N], kp, vp, table, kv, par, N)

    want = call()
    la.poll_error()
    status = []
    la.set_wait_limit(1)
    try:
        for _ in range(5):
            call()
            try:
                la.poll_error()
            except la.LAError as e:
                status.append(e.status)
    finally:
        la.set_wait_limit(0)
    assert set(status) <= {4} and (status or not must)
    for _ in range(3):
        assert torch.equal(call(), want)
    la.poll_error()


def test_a_hybrid_layer_as_it_is_served():
    """Prompt, next chunk, single tokens, a tree of drafts, its commit and one more token, next to a linear layer that gets
    the same rotary positions: every output against the whole sequence at once."""
    H, Hkv, P, gen = 8, 2, 16, torch.Generator().manual_seed(1)
    freq, mscale = la.rope_freqs(64, 10000.0, "yarn", 4.0, 64)
    df = freq.to(DEV)
    lens = [90, 33]
    B, width = 2, 20
    kp = torch.full((B * width, Hkv, P, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    vp = torch.full_like(kp, float("nan"))
    table = torch.randperm(B * width, generator=gen).int().reshape(B, width)
    seq = [[], []]  # (q, k, v) rows in order, positions
    rand = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731

    def place(b, at):
        return int(table[b, at // P]) * P + at % P

    def store(rows, where, pos):
        q, k, v = (torch.cat(x) for x in zip(*rows))
        return la.kv_store(q.to(DEV), k.to(DEV), v.to(DEV), i32(pos).to(DEV), df, kp, vp, i32(where).to(DEV), mscale=mscale)

    def want(b, upto, rows):
        """The last `rows` of the first `upto` tokens of request b, from the definition."""
        q, k, v = (torch.cat([t[i] for t in seq[b][:upto]]) for i in range(3))
        pos = np.arange(upto)
        rot = lambda x: torch.from_numpy(attn.rope(f64(x).reshape(upto, -1, D), pos, freq.numpy(), False,  # noqa: E731
                                                   np.float64(np.float32(mscale)))).bfloat16().double().numpy()
        return attn.attend(rot(q)[-rows:], rot(k), f64(v).reshape(upto, Hkv, D), attn.causal(rows, upto), SCALE)

    def close(got, ref, what):
        # rotated q and k may round the other way in the last bit: scores off by 2^-8 of theirs, a few percent of a weight
        o, size = ref
        assert (np.abs(f64(got).reshape(o.shape) - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -5 * size).all(), what

    new = lambda n: (rand(n, H * D), rand(n, Hkv * D), rand(n, Hkv * D))  # noqa: E731
    done = [0, 0]
    for chunk in ([60, 33], [30, 0]):  # the prompts, the first in two chunks
        rows = [new(n) for n in chunk]
        for b, n in enumerate(chunk):
            seq[b] += [tuple(x[i:i + 1] for x in rows[b]) for i in range(n)]
        pos = [done[b] + i for b in range(B) for i in range(chunk[b])]
        q = store(rows, [place(b, done[b] + i) for b in range(B) for i in range(chunk[b])], pos)
        done = [d + n for d, n in zip(done, chunk)]
        out = la.attn_extend(q, kp, vp, table.to(DEV), i32([0, chunk[0], sum(chunk)]).to(DEV), i32(done).to(DEV),
                             max_seqlen=max(chunk))
        for b, r in ((0, slice(0, chunk[0])), (1, slice(chunk[0], sum(chunk)))):
            if chunk[b]:
                close(out[r], want(b, done[b], chunk[b]), f"prompt {b}")
    assert done == lens
    # a linear-attention layer of the same model: the same positions, then its own update
    lq, lk, lv = new(2)
    rq, rk = la.rope(lq.to(DEV), torch.cat([lk] * 4, 1).to(DEV), i32(done).to(DEV), df, mscale=mscale)
    pool = torch.zeros(3, H, D, D, device=DEV)
    lo = la.decode(rq, rk, torch.cat([lv] * 4, 1).to(DEV), la.slopes(H, 0, 1).to(DEV), pool, i32([2, 0]).to(DEV))
    score = (rq.float() * rk.float()).reshape(2, H, D).sum(-1, keepdim=True) * D ** -0.5
    ref = score * torch.cat([lv] * 4, 1).to(DEV).float().reshape(2, H, D)
    assert (lo.float().reshape(2, H, D) - ref).abs().max() <= 2.0 ** -7 * ref.abs().max()

    def step():
        rows = [new(1) for _ in range(B)]
        for b in range(B):
            seq[b].append(rows[b])
        q = store(rows, [place(b, done[b]) for b in range(B)], done)
        for b in range(B):
            done[b] += 1
        out = la.attn_decode(q, kp, vp, table.to(DEV), i32(done).to(DEV))
        for b in range(B):
            close(out[b:b + 1], want(b, done[b], 1), f"token {done[b]} of {b}")

    step()
    step()
    # a tree of drafts: rows in draft order, positions by depth
    N, parents = 6, [[-1, 0, 0, 2, 2, -1], [-1, -1, 1, 2, 3, 0]]
    depth = [[len(attn.path(parents[b], t)) - 1 for t in range(N)] for b in range(B)]
    drafts = [new(N) for _ in range(B)]
    q = store(drafts, [place(b, done[b] + t) for b in range(B) for t in range(N)],
              [done[b] + depth[b][t] for b in range(B) for t in range(N)])
    kv = i32([d + N for d in done]).to(DEV)
    par = i32(parents).to(DEV)
    out = la.attn_verify_tree(q, kp, vp, table.to(DEV), kv, par, N)
    for b in range(B):
        for t in range(N):
            keep = seq[b]
            seq[b] = keep + [tuple(x[a:a + 1] for x in drafts[b]) for a in attn.path(parents[b], t)]
            close(out[b * N + t:b * N + t + 1], want(b, len(seq[b]), 1), f"draft {t} of {b}")
            seq[b] = keep
    accept = [4, 4]
    lens_out = la.kv_commit(kp, vp, table.to(DEV), kv, par, i32(accept).to(DEV))
    for b in range(B):
        p = attn.path(parents[b], accept[b])
        seq[b] += [tuple(x[a:a + 1] for x in drafts[b]) for a in p]
        done[b] += len(p)
    assert lens_out.tolist() == done
    step()
    la.poll_error()
