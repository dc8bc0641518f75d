"""Attention calls whose waits run out at other places from limit to limit, in some warps of a CTA before others: every
call ends and says so, and the next one is right."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from attn_testutil import Cache, i32, queries

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("op", ["decode", "tree", "wide tree", "extend"])
@pytest.mark.parametrize("lens", [[3000, 129, 700], [150, 33, 256]])
def test_limits(op, lens):
    H, Hkv, P, B = 8, 2, 16, len(lens)
    N = {"decode": 1, "tree": 5, "wide tree": 20, "extend": 30}[op]
    cache = Cache(lens, Hkv, P, N)
    q = queries(B * N, H, N).to(DEV)
    kp, vp, table, kv = cache.to(DEV)
    cu, par = i32([N * b for b in range(B + 1)]).to(DEV), i32([[t // 2 - 1 for t in range(N)]] * B).to(DEV)

    def call():
        if op == "extend":
            return la.attn_extend(q, kp, vp, table, cu, kv, max_seqlen=N)
        if op == "decode":
            return la.attn_decode(q, kp, vp, table, kv)
        return la.attn_verify_tree(q, kp, vp, table, kv, par, N)

    want = call()
    la.poll_error()
    assert np.isfinite(want.float().cpu().numpy()).all()
    try:
        for limit in list(range(1, 40)) + [50, 70, 100]:
            la.set_wait_limit(limit)
            for _ in range(4):
                call()
            try:
                la.poll_error()
            except la.LAError as e:
                assert e.status == 4
    finally:
        la.set_wait_limit(0)
    for _ in range(2):
        assert torch.equal(call(), want)
    la.poll_error()
