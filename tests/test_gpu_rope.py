"""Rotary positions on the GPU (la_rope, la_kv_store) against the fp64 oracle: layouts, parts of the head, far and
negative positions, strides, in place, stores into pages."""
import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from attn_testutil import D, U16, f64, i32, queries
from oracle import attn

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def check_rows(actual, x, pos, freq, interleaved, mscale, what):
    T = x.shape[0]
    y = f64(x).reshape(T, -1, D)
    want = attn.rope(y, pos.numpy(), freq.numpy(), interleaved, mscale)
    a = f64(actual).reshape(want.shape)
    R = 2 * len(freq)
    assert np.array_equal(a[..., R:], y[..., R:]), what
    # a pair's size bounds both of its values
    size = np.zeros_like(want)
    p, q = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    size[..., p] = size[..., q] = np.hypot(y[..., p], y[..., q]) * mscale
    bad = np.abs(a - want) > U16 * np.abs(want) + 2.0 ** -20 * size
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float(np.abs(a - want).max()):.3g}"


def positions(T, far, seed=0):
    gen = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, far, (T,), generator=gen).int()
    pos[0] = far - 1
    return pos


@pytest.mark.parametrize("T,H,Hkv", [(1, 1, 1), (1, 16, 16), (3, 5, 2), (33, 32, 4), (7, 64, 8), (2, 130, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_shapes(T, H, Hkv, interleaved):
    freq, _ = la.rope_freqs(D)
    q, k, pos = queries(T, H, T), queries(T, Hkv, T + 1), positions(T, 5000, T)
    qo, ko = la.rope(q.to(DEV), k.to(DEV), pos.to(DEV), freq.to(DEV), interleaved=interleaved)
    la.poll_error()
    check_rows(qo, q, pos, freq, interleaved, 1.0, "q")
    check_rows(ko, k, pos, freq, interleaved, 1.0, "k")


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 96, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_parts_and_far_positions(rot, interleaved):
    freq, mscale = la.rope_freqs(rot, 10000.0, "yarn", 8.0, 4096)
    q, k = queries(9, 3, rot), queries(9, 1, rot + 1)
    pos = positions(9, 2 ** 31 - 1, rot)
    pos[1:5] = i32([0, -1, -(2 ** 31), 1 << 20])
    qo, ko = la.rope(q.to(DEV), k.to(DEV), pos.to(DEV), freq.to(DEV), interleaved=interleaved, mscale=mscale)
    la.poll_error()
    check_rows(qo, q, pos, freq, interleaved, np.float64(np.float32(mscale)), "q")
    check_rows(ko, k, pos, freq, interleaved, np.float64(np.float32(mscale)), "k")


def test_rope_nothing_rotated():
    q, k = queries(5, 2), queries(5, 1, 3)
    none = torch.empty(0, dtype=torch.float64, device=DEV)
    qo, ko = la.rope(q.to(DEV), k.to(DEV), torch.zeros(5, dtype=torch.int32, device=DEV), none)
    assert torch.equal(qo.cpu(), q) and torch.equal(ko.cpu(), k)


def test_rope_columns_of_a_projection_in_place():
    T, H, Hkv = 50, 6, 2
    freq, _ = la.rope_freqs(64)
    x = queries(T, H + 2 * Hkv, 4)
    dx = x.to(DEV)
    q, k = dx[:, :H * D], dx[:, H * D:(H + Hkv) * D]
    pos = positions(T, 300)
    a, b = la.rope(q, k, pos.to(DEV), freq.to(DEV), q_out=q, k_out=k)
    la.poll_error()
    assert a is q and b is k
    check_rows(dx[:, :H * D], x[:, :H * D], pos, freq, False, 1.0, "q")
    check_rows(dx[:, H * D:(H + Hkv) * D], x[:, H * D:(H + Hkv) * D], pos, freq, False, 1.0, "k")
    assert torch.equal(dx[:, (H + Hkv) * D:].cpu(), x[:, (H + Hkv) * D:])


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("H,Hkv,alternate", [(8, 2, False), (3, 3, True), (40, 8, False)])
def test_store(P, H, Hkv, alternate):
    T, E = 70, 9
    freq, mscale = la.rope_freqs(D, 10000.0, "yarn", 4.0, 4096)
    q, k, v, pos = queries(T, H, 1), queries(T, Hkv, 2), queries(T, Hkv, 3), positions(T, 100000)
    loc = torch.randperm(E * P, generator=torch.Generator().manual_seed(P))[:T].int()
    loc[::7] = -1
    both = torch.full((E, 2, Hkv, P, D), 5.0, dtype=torch.bfloat16, device=DEV)
    kp, vp = both[:, 0], both[:, 1]
    if not alternate:
        kp, vp = kp.contiguous(), vp.contiguous()
    qo = la.kv_store(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), freq.to(DEV), kp, vp, loc.to(DEV), mscale=mscale)
    la.poll_error()
    check_rows(qo, q, pos, freq, False, np.float64(np.float32(mscale)), "q")
    on = (loc >= 0).nonzero()[:, 0]
    at = loc[on].long()
    check_rows(kp.cpu()[at // P, :, at % P].reshape(len(on), -1), k[on], pos[on], freq, False,
               np.float64(np.float32(mscale)), "k")
    assert torch.equal(vp.cpu()[at // P, :, at % P].reshape(len(on), -1), v[on])
    free = torch.ones(E * P, dtype=torch.bool)
    free[at] = False
    rest = free.nonzero()[:, 0]
    for pages in (kp.cpu(), vp.cpu()):
        assert (pages[rest // P, :, rest % P] == 5.0).all()


@pytest.mark.parametrize("bad", [-2, 9 * 16, 2 ** 31 - 1, -(2 ** 31)])
def test_store_bad_rows(bad):
    T, Hkv, P, E = 4, 2, 16, 9
    freq, _ = la.rope_freqs(D)
    q, k, v, pos = queries(T, 2, 1), queries(T, Hkv, 2), queries(T, Hkv, 3), positions(T, 100)
    kp = torch.zeros(E, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    la.kv_store(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), freq.to(DEV), kp, vp, i32([0, bad, 20, -1]).to(DEV))
    with pytest.raises(la.LAError) as e:
        la.poll_error()
    assert e.value.status == 5
    la.poll_error()
    rows = vp.transpose(1, 2).reshape(E * P, -1).cpu()
    assert torch.equal(rows[0], v[0]) and torch.equal(rows[20], v[2])
    rows[0] = rows[20] = 0
    assert not rows.any()
