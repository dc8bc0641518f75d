"""Scratch of the gated delta rule's extend: none where the tokens are taken one by one (at most 6 a request),
refused where it is missing otherwise."""
import ctypes

import pytest
import torch

import lightning_attention_gb300 as la
from delta_testutil import D, TOL_RECURRENT, check_states, f64, inputs, run_states
from lightning_attention_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("n,max_seqlen,ok", [(6, 6, True), (6, 1000, True), (40, 6, True), (7, 7, False),
                                             (40, 7, False)])
def test_no_workspace(n, max_seqlen, ok):
    """Requests of 6 tokens and the rest of n, under C: NULL will do where max_seqlen or T is at most 6."""
    H = 2
    lens = [6] * (n // 6) + ([n % 6] if n % 6 else [])
    B = len(lens)
    host = inputs(n, 1, H, 61)
    d = [t.to(DEV) for t in host]
    cu = torch.tensor([sum(lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    idx = torch.arange(B, dtype=torch.int32, device=DEV)
    mask = torch.zeros(B, dtype=torch.uint8, device=DEV)
    pool = torch.full((B, H, D, D), 0.5, device=DEV)
    out = torch.zeros(n, H * D, dtype=torch.bfloat16, device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = binding.load().la_delta_extend(p(d[0]), p(d[1]), p(d[2]), 0, 0, 0, p(d[3]), p(d[4]), p(pool), B, p(idx),
                                        p(cu), p(mask), p(out), B, n, H, 1, D, max_seqlen, 1, None, 0, None)
    la.poll_error()
    if not ok:
        assert st == 1 and (pool == 0.5).all() and (out == 0).all()
        return
    assert st == 0
    for b in (0, B - 1):
        r = slice(sum(lens[:b]), sum(lens[:b + 1]))
        _, S, _ = run_states(*[x[r] for x in host], torch.zeros(H, D, D).double().numpy(), 1, H, True)
        check_states(f64(pool[b]), S, TOL_RECURRENT, str(b))


def test_few_tokens_allocate_nothing():
    B, n, H = 256, 4, 8
    d = [t.to(DEV) for t in inputs(B * n, 1, H, 62)]
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    idx = torch.arange(B, dtype=torch.int32, device=DEV)
    mask = torch.zeros(B, dtype=torch.uint8, device=DEV)
    pool = torch.zeros(B, H, D, D, device=DEV)
    out = torch.zeros(B * n, H * D, dtype=torch.bfloat16, device=DEV)
    taken = lambda: torch.cuda.memory_stats()["allocated_bytes.all.allocated"]  # noqa: E731
    before = taken()
    la.delta_extend(*d, pool, idx, cu, mask, out=out, max_seqlen=n, qk_l2norm=True)
    assert taken() == before
    la.delta_extend(*d, pool, idx, cu, mask, out=out, max_seqlen=7, qk_l2norm=True)
    assert taken() - before >= la.delta_extend_workspace_size(B, B * n, H, D)
    la.poll_error()
