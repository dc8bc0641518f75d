"""Gated delta rule extend with cu_seqlens that decreases somewhere: by chunks nothing of the batch is
written, token by token the other requests are as ever, and both are reported."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from delta_testutil import D, TOL_RECURRENT, check_states, f64, inputs, run_states

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _call(d, H, cu, max_seqlen, pool, out):
    B = len(cu) - 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    la.delta_extend(*d, pool, i32(list(range(B))), i32(cu), torch.ones(B, dtype=torch.uint8, device=DEV), out=out,
                    max_seqlen=max_seqlen, qk_l2norm=True)


def _bent(lens, at, by):
    """Ends of the requests, those from `at` on taken back by `by`."""
    cu = np.cumsum([0] + list(lens))
    cu[at:] -= by
    return [int(x) for x in cu]


@pytest.mark.parametrize("cu,H,max_seqlen", [
    ([0, 100, 60, 200], 2, 140),                                        # a CTA per chain
    ([0, 100, 200, 199], 2, 100),                                       # the last entry
    (_bent([70] * 100, 50, 75), 2, 200),                                # many waves, ranked
    (_bent([9] * 300, 7, 10), 2, 9),                                    # more requests than a CTA has threads
    ([0, 2400, 2300, 2600], 2, 2400),                                   # segments
    (_bent([64] * 39 + [2400] + [100] * 10, 45, 130), 2, 2400),         # a plan
])
def test_by_chunks_nothing_is_written(cu, H, max_seqlen):
    B, T = len(cu) - 1, max(cu)
    d = [t.to(DEV) for t in inputs(T, 1, H, 51)]
    pool = torch.full((B, H, D, D), 0.01, device=DEV)
    out = torch.full((T, H * D), 7.0, dtype=torch.bfloat16, device=DEV)
    _call(d, H, cu, max_seqlen, pool, out)
    with pytest.raises(la.LAError) as e:
        la.poll_error()
    assert e.value.status == 5
    assert (pool == 0.01).all() and (out == 7.0).all()
    # the same batch in order runs as ever: nothing is kept from the call before
    straight = sorted(cu)
    for i in range(2):
        p, o = pool.clone(), out.clone()
        _call(d, H, straight, T, p, o)
        la.poll_error()
        if i == 0:
            first = p, o
    assert torch.equal(p, first[0]) and torch.equal(o, first[1])
    assert not (p == 0.01).all()


def test_token_by_token_the_others_run():
    H, cu = 2, [0, 5, 3, 8]
    d = inputs(8, 1, H, 52)
    pool0 = torch.randn(3, H, D, D, generator=torch.Generator().manual_seed(52)) * 0.05
    pool, out = pool0.to(DEV), torch.zeros(8, H * D, dtype=torch.bfloat16, device=DEV)
    _call([t.to(DEV) for t in d], H, cu, 6, pool, out)
    with pytest.raises(la.LAError) as e:
        la.poll_error()
    assert e.value.status == 5
    assert torch.equal(pool[1].cpu(), pool0[1])
    for b in (0, 2):
        r = slice(cu[b], cu[b + 1])
        _, S, _ = run_states(*[x[r] for x in d], f64(pool0[b]), 1, H, True)
        check_states(f64(pool[b]), S, TOL_RECURRENT, str(b))
