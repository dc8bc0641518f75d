"""Captured gated-delta-rule extends of every schedule, replayed on other inputs and other lengths (which are device
data: the launches go by B, T, H and max_seqlen alone) against eager calls, bit for bit, and one of each against the
oracle."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from delta_testutil import (D, SENTINEL, TOL_EXTEND, TOL_RECURRENT, check_out, check_states, f64, inputs,
                            run_states)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _set(t, values):
    t.copy_(torch.tensor(values, dtype=t.dtype))


@pytest.mark.parametrize("many,H,max_seqlen,tol", [
    ([[64] * 39 + [2400] + [100] * 10, [2400] + [60] * 49, [50] * 30 + [800] * 3 + [93] * 17], 2, 2400, 2 * TOL_EXTEND),
    ([[70] * 100, [1] * 50 + [139] * 50, [0, 140] * 50], 2, 140, TOL_EXTEND),   # waves, ranked
    ([[2200, 300], [100, 2400], [1250, 1250]], 3, 2400, 2 * TOL_EXTEND),        # segments
    ([[100, 300, 5], [300, 5, 100], [0, 200, 205]], 2, 300, TOL_EXTEND),        # a CTA per chain
    ([[6, 1, 0, 5], [0, 6, 6, 0], [3, 3, 3, 3]], 2, 6, TOL_RECURRENT),          # token by token
])
def test_replays_with_other_lengths(many, H, max_seqlen, tol):
    B, T = len(many[0]), max(sum(x) for x in many)
    d = [t.to(DEV) for t in inputs(T, 1, H, 81)]
    idx = torch.arange(B, dtype=torch.int32, device=DEV)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    mask = torch.zeros(B, dtype=torch.uint8, device=DEV)
    pool = torch.zeros(B, H, D, D, device=DEV)
    start = torch.randn(B, H, D, D, generator=torch.Generator().manual_seed(81)).to(DEV) * 0.05
    out = torch.zeros(T, H * D, dtype=torch.bfloat16, device=DEV)

    def call(out):
        return la.delta_extend(*d, pool, idx, cu, mask, out=out, max_seqlen=max_seqlen, qk_l2norm=True)

    def load(i):
        _set(cu, np.cumsum([0] + many[i]).tolist())
        _set(mask, [(b + i) % 2 for b in range(B)])
        for x, y in zip(d, inputs(T, 1, H, 82 + i)):
            x.copy_(y)
        pool.copy_(start)
        out.fill_(SENTINEL)

    load(0)
    call(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for i in (0, 1, 2, 1):
        load(i)
        call(out)
        want = out.clone(), pool.clone()
        load(i)
        g.replay()
        la.poll_error()
        assert torch.equal(out, want[0]) and torch.equal(pool, want[1]), i
    lens, at = many[1], np.cumsum([0] + many[1])
    host = [x.cpu() for x in d]
    for b in sorted({0, 1, B // 2, B - 1, int(np.argmax(lens))}):
        r = slice(int(at[b]), int(at[b + 1]))
        S0 = f64(start[b]) if (b + 1) % 2 else np.zeros((H, D, D))
        o, S, norms = run_states(*[x[r] for x in host], S0, 1, H, True)
        check_out(f64(out[r]), o, host[0][r], np.broadcast_to(norms, (lens[b], H)), tol, 1, H, True, str(b))
        check_states(f64(pool[b]), S, tol, str(b))
    assert (out[sum(lens):] == torch.tensor(SENTINEL).bfloat16().to(DEV)).all()


def test_norms_of_1e18_and_keys_of_zero():
    """qk_l2norm at the largest norms that the header promises and at vanishing ones: extend, decode and verify."""
    n, H = 130, 2
    for seed, spread in ((83, 1e17), (84, 1e-12)):
        q, k, v, g, beta = inputs(n, 1, H, seed, True, "model", spread)
        k[5::7], q[3::5] = 0.0, 0.0
        host = (q, k, v, g, beta)
        o, S, norms = run_states(*host, np.zeros((H, D, D)), 1, H, True)
        norms = np.broadcast_to(norms, (n, H))
        d = [t.to(DEV) for t in host]
        idx = torch.zeros(1, dtype=torch.int32, device=DEV)
        pool = torch.full((1, H, D, D), SENTINEL, device=DEV)
        out = la.delta_extend(*d, pool, idx, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                              torch.zeros(1, dtype=torch.uint8, device=DEV), max_seqlen=n, qk_l2norm=True)
        la.poll_error()
        check_out(f64(out), o, q, norms, TOL_EXTEND, 1, H, True, "extend")
        check_states(f64(pool[0]), S, TOL_EXTEND, "extend")
        pool.zero_()
        outs = [la.delta_decode(*[x[t:t + 1] for x in d], pool, idx, qk_l2norm=True) for t in range(5)]
        o5, inter = la.delta_verify_chain(*[x[5:40] for x in d], pool, idx, 35, qk_l2norm=True)
        la.poll_error()
        o, S, norms = run_states(*[x[:40] for x in host], np.zeros((H, D, D)), 1, H, True)
        check_out(f64(torch.cat(outs + [o5])), o, q[:40], np.broadcast_to(norms, (40, H)), TOL_RECURRENT, 1, H, True,
                  "token by token")
        check_states(f64(inter[0, -1]), S, TOL_RECURRENT, "token by token")
