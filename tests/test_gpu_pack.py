"""Packed state store on the GPU (la_pack_states, la_unpack_states) against the oracle, bit for bit:
the scales are powers of two, so codes and restored values are exact on both sides."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from delta_testutil import D, SENTINEL
from oracle import delta

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _store(E, H):
    return (torch.full((E, H, D, D), 99, dtype=torch.int8, device=DEV),
            torch.full((E, H, D, D // 32), 88, dtype=torch.uint8, device=DEV))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _pool(slots, H, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(slots, H, D, D, generator=gen) * torch.exp(2 * torch.randn(slots, H, D, 1, generator=gen))


@pytest.mark.parametrize("B,H", [(1, 1), (3, 2), (6, 5)])
def test_round_trip(B, H):
    pool0 = _pool(B + 2, H, B)
    slots = list(range(B + 1, 1, -1))
    entries = [(3 * b + 1) % (B + 3) if B != 3 else b + 1 for b in range(B)]
    if len(set(entries)) < B:
        entries = list(range(B))
    codes, scales = _store(B + 3, H)
    la.pack_states(pool0.to(DEV), _i32(slots), codes, scales, _i32(entries))
    back = torch.full((B + 2, H, D, D), SENTINEL, device=DEV)
    la.unpack_states(codes, scales, _i32(entries), back, _i32(slots))
    la.poll_error()
    rc, rs = delta.pack(pool0[slots].numpy())
    assert np.array_equal(codes[entries].cpu().numpy(), rc)
    assert np.array_equal(scales[entries].cpu().numpy(), rs)
    assert np.array_equal(back[slots].cpu().double().numpy(), delta.unpack(rc, rs))
    rest = [e for e in range(B + 3) if e not in entries]
    assert (codes[rest] == 99).all() and (scales[rest] == 88).all()
    assert (back[[0, 1]] == SENTINEL).all()
    again = _store(B + 3, H)
    la.pack_states(back, _i32(slots), *again, _i32(entries))
    la.poll_error()
    assert torch.equal(again[0], codes) and torch.equal(again[1], scales)


def test_borders_of_scales_and_odd_values():
    """Values at the rounding borders of codes and scales, subnormals, zeros, the largest values."""
    x = torch.zeros(1, 1, D, D)
    f = x.view(D, 4, 32)
    tops = [127.5, 127.49999, 127.50001, 64.0, 63.999996, 1.0, 2.0 ** -126, 2.0 ** -127, 2.0 ** -149, torch.finfo(torch.float32).max,
            2.0 ** -121, 2.0 ** -120, 1.5 * 2.0 ** -120, 127.5 * 2.0 ** 60, -127.5, 1e-40]
    gen = torch.Generator().manual_seed(3)
    for i in range(D):
        for j in range(4):
            top = tops[(4 * i + j) % len(tops)]
            f[i, j] = (torch.rand(32, generator=gen) * 2 - 1) * abs(top) * 0.999
            f[i, j, (i + j) % 32] = top
    f[0, 0] = 0.0
    f[1, 1, 5] = float("inf")
    f[2, 2, 7] = float("nan")
    f[3, 3, 0] = float("-inf")
    f[4, 0] = -0.0
    half = torch.arange(32).float() + 0.5  # ties go to the even code
    f[5, 0] = torch.cat([half[:31], torch.tensor([127.0])])
    codes, scales = _store(1, 1)
    la.pack_states(x.to(DEV), _i32([0]), codes, scales, _i32([0]))
    back = torch.zeros(1, 1, D, D, device=DEV)
    la.unpack_states(codes, scales, _i32([0]), back, _i32([0]))
    la.poll_error()
    rc, rs = delta.pack(x.numpy())
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(back.cpu().double().numpy(), delta.unpack(rc, rs))


def test_one_entry_for_several_slots_and_any_bytes():
    """A packed prefix restored into several requests' slots, from arbitrary codes and scales."""
    gen = torch.Generator().manual_seed(4)
    codes = torch.randint(-128, 128, (2, 3, D, D), generator=gen).to(torch.int8)
    scales = torch.randint(0, 256, (2, 3, D, 4), generator=gen).to(torch.uint8)
    pool = torch.full((5, 3, D, D), SENTINEL, device=DEV)
    la.unpack_states(codes.to(DEV), scales.to(DEV), _i32([1, 1, 0]), pool, _i32([4, 0, 2]))
    la.poll_error()
    with np.errstate(over="ignore"):
        ref = delta.unpack(codes.numpy(), scales.numpy()).astype(np.float32)
    for entry, slot in ((1, 4), (1, 0), (0, 2)):
        np.testing.assert_array_equal(pool[slot].cpu().numpy(), ref[entry])
    assert (pool[[1, 3]] == SENTINEL).all()


def test_faults_and_empty_batch():
    codes, scales = _store(2, 1)
    pool = torch.ones(2, 1, D, D, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    la.pack_states(pool, none, codes, scales, none)
    la.unpack_states(codes, scales, none, pool, none)
    la.poll_error()
    for slot, entry in ((2, 0), (-1, 0), (0, 2), (0, -1)):
        la.pack_states(pool, _i32([slot]), codes, scales, _i32([entry]))
        with pytest.raises(la.LAError) as e:
            la.poll_error()
        assert e.value.status == 5
        la.unpack_states(codes, scales, _i32([entry]), pool, _i32([slot]))
        with pytest.raises(la.LAError):
            la.poll_error()
    assert (codes == 99).all() and (scales == 88).all() and (pool == 1).all()


def test_prefix_cache_run():
    """Extend a prefix, pack its state, drop the slot, restore it into two slots, extend both."""
    from delta_testutil import inputs

    Hk, H, n = 1, 2, 70
    d = [t.to(DEV) for t in inputs(n + 40, Hk, H, 31)]
    pool = torch.full((3, H, D, D), SENTINEL, device=DEV)
    zero = torch.zeros(1, dtype=torch.uint8, device=DEV)
    la.delta_extend(*[x[:n] for x in d], pool, _i32([1]), _i32([0, n]), zero, qk_l2norm=True)
    codes, scales = _store(1, H)
    la.pack_states(pool, _i32([1]), codes, scales, _i32([0]))
    kept = pool[1].clone()
    pool.fill_(SENTINEL)
    la.unpack_states(codes, scales, _i32([0, 0]), pool, _i32([0, 2]))
    assert torch.equal(pool[0], pool[2])
    top = kept.view(H, D, 4, 32).abs().amax(-1, keepdim=True)
    assert ((pool[0] - kept).view(H, D, 4, 32).abs() <= top / 127).all()
    out = la.delta_extend(*[x[n:] for x in d], pool, _i32([0, 2]), _i32([0, 20, 40]),
                          torch.ones(2, dtype=torch.uint8, device=DEV), qk_l2norm=True)
    la.poll_error()
    assert torch.isfinite(out.float()).all() and (pool[1] == SENTINEL).all()
