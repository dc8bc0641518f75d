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
