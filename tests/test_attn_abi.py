"""CPU-side checks of the rotary, cache and attention entry points: every refusal happens on the host before anything
is launched, so it runs the same with or without a GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import lightning_attention_gb300 as la
from lightning_attention_gb300 import _build, binding
from oracle import attn

OK, BAD16, BAD4 = ctypes.c_void_p(4096), ctypes.c_void_p(4096 + 8), ctypes.c_void_p(4096 + 2)
N = None


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def rope(lib, q=OK, k=OK, rs=(0, 0), pos=OK, freq=OK, rot=64, m=1.0, qo=OK, ko=OK, ors=(0, 0), T=2, H=2, Hkv=1,
         D=128):
    return lib.la_rope(q, k, *rs, pos, freq, rot, 0, m, qo, ko, *ors, T, H, Hkv, D, N)


def store(lib, q=OK, k=OK, v=OK, rs=(0, 0, 0), pos=OK, freq=OK, rot=64, m=1.0, qo=OK, ors=0, kp=OK, vp=OK, ps=0, E=4,
          P=16, loc=OK, T=2, H=2, Hkv=1, D=128):
    return lib.la_kv_store(q, k, v, *rs, pos, freq, rot, 0, m, qo, ors, kp, vp, ps, E, P, loc, T, H, Hkv, D, N)


def extend(lib, q=OK, rs=0, kp=OK, vp=OK, ps=0, E=4, P=16, table=OK, width=2, cu=OK, kv=OK, out=OK, B=1, T=8, H=2,
           Hkv=1, D=128, ms=8, mk=32, scale=0.1, ws=OK, nbytes=1 << 30):
    return lib.la_attn_extend(q, rs, kp, vp, ps, E, P, table, width, cu, kv, out, B, T, H, Hkv, D, ms, mk, scale, ws,
                              nbytes, N)


def decode(lib, q=OK, rs=0, kp=OK, vp=OK, ps=0, E=4, P=16, table=OK, width=2, kv=OK, out=OK, B=2, H=2, Hkv=1, D=128,
           scale=0.1, ws=OK, nbytes=1 << 30):
    return lib.la_attn_decode(q, rs, kp, vp, ps, E, P, table, width, kv, out, B, H, Hkv, D, scale, ws, nbytes, N)


def tree(lib, q=OK, rs=0, kp=OK, vp=OK, ps=0, E=4, P=16, table=OK, width=2, kv=OK, parents=OK, out=OK, B=2, n=3, H=2,
         Hkv=1, D=128, scale=0.1, ws=OK, nbytes=1 << 30):
    return lib.la_attn_verify_tree(q, rs, kp, vp, ps, E, P, table, width, kv, parents, out, B, n, H, Hkv, D, scale, ws,
                                   nbytes, N)


def commit(lib, kp=OK, vp=OK, ps=0, E=4, P=16, table=OK, width=2, kv=OK, parents=OK, acc=OK, lens=OK, B=2, n=3, Hkv=1,
           D=128):
    return lib.la_kv_commit(kp, vp, ps, E, P, table, width, kv, parents, acc, lens, B, n, Hkv, D, N)


ATTN = (extend, decode, tree)
LISTS = ATTN + (commit,)
PAGED = LISTS + (store,)


def test_sizes_and_heads(lib):
    for call in (rope, store):
        for kw in ({"T": -1}, {"H": 0}, {"Hkv": 0}, {"D": 0}, {"rot": -16}, {"rot": 144}, {"m": math.nan}, {"m": math.inf}):
            assert call(lib, **kw) == 1, (call, kw)
        assert call(lib, D=64) == 2 and call(lib, rot=24) == 2 and call(lib, H=1 << 24) == 2
    for call in ATTN:
        for kw in ({"B": -1}, {"H": 0}, {"Hkv": 0}, {"H": 3, "Hkv": 2}, {"H": 1, "Hkv": 2}, {"D": 0}, {"scale": 0.0},
                   {"scale": -1.0}, {"scale": math.nan}, {"scale": math.inf}, {"scale": 3e38}):
            assert call(lib, **kw) == 1, (call, kw)
        assert call(lib, D=64) == 2 and call(lib, H=129) == 2
    assert extend(lib, T=-1) == 1 and extend(lib, ms=-1) == 1 and extend(lib, mk=-1) == 1
    for call in (tree, commit):
        assert call(lib, n=0) == 1 and call(lib, n=129) == 2
    assert tree(lib, B=1 << 25, n=128) == 1
    assert commit(lib, B=-1) == 1 and commit(lib, Hkv=0) == 1 and commit(lib, D=64) == 2


def test_cache_layout(lib):
    for call in PAGED:
        for kw in ({"E": 0}, {"P": 0}, {"P": -16}, {"ps": 16 * 128 - 8}, {"ps": 16 * 128 + 4}, {"ps": -2048}):
            assert call(lib, **kw) == 1, (call, kw)
        for kw in ({"P": 48}, {"P": 8}, {"P": 256}, {"ps": 1 << 40}, {"ps": 1 << 30, "E": 1 << 20}):
            assert call(lib, **kw) == 2, (call, kw)
    for call in LISTS:
        assert call(lib, width=0) == 1 and call(lib, width=-1) == 1
        assert call(lib, P=128, width=(1 << 23) + 1) == 2


def test_row_strides(lib):
    for rs in ((120, 0), (0, 132), (0, 120), (-256, 0), (260, 0)):
        assert rope(lib, rs=rs) == 1 and rope(lib, ors=rs) == 1
        assert store(lib, rs=rs + (0,)) == 1 and store(lib, rs=(0, 0, rs[1] or rs[0] - 128)) == 1
    for call in ATTN:
        for rs in (120, 132, -256, 260):
            assert call(lib, rs=rs) == 1, (call, rs)
        assert call(lib, rs=1 << 40) == 2


def test_empty_calls_are_no_ops(lib):
    cache = dict(kp=N, vp=N)
    assert rope(lib, q=N, k=N, pos=N, freq=N, qo=N, ko=N, T=0) == 0
    assert store(lib, q=N, k=N, v=N, pos=N, freq=N, qo=N, loc=N, T=0, **cache) == 0
    none = dict(q=N, table=N, kv=N, out=N, ws=N, nbytes=0, **cache)
    assert extend(lib, cu=N, T=0, B=0, **none) == 0 and extend(lib, cu=N, T=0, B=3, **none) == 0
    assert decode(lib, B=0, **none) == 0 and tree(lib, B=0, parents=N, **none) == 0
    assert commit(lib, table=N, kv=N, parents=N, acc=N, lens=N, B=0, **cache) == 0


def test_null_and_misaligned_pointers(lib):
    wants16 = {rope: ("q", "k", "qo", "ko"), store: ("q", "k", "v", "qo", "kp", "vp"), extend: ("q", "kp", "vp", "out"),
               decode: ("q", "kp", "vp", "out", "ws"), tree: ("q", "kp", "vp", "out", "ws"), commit: ("kp", "vp")}
    wants4 = {rope: ("pos",), store: ("pos", "loc"), extend: ("table", "cu", "kv"), decode: ("table", "kv"),
              tree: ("table", "kv", "parents"), commit: ("table", "kv", "parents", "acc", "lens")}
    for wants, bad in ((wants16, BAD16), (wants4, BAD4)):
        for call, names in wants.items():
            more = {"width": 17} if call in (decode, tree) else {}  # contexts that take scratch
            for name in names:
                assert call(lib, **more, **{name: bad}) == 1, (call, name)
                assert call(lib, **more, **{name: N}) == 1, (call, name)
    for call in (rope, store):
        assert call(lib, freq=N) == 1 and call(lib, freq=ctypes.c_void_p(4096 + 4)) == 1
    assert extend(lib, ws=BAD16) == 1


def test_workspaces(lib):
    nb = ctypes.c_size_t(7)
    size = lib.la_attn_verify_workspace_size
    for args, st in (((1, 0, 1, 1, 128, 9), 1), ((1, 1, 0, 1, 128, 9), 1), ((1, 1, 3, 2, 128, 9), 1), ((1, 1, 1, 0, 128, 9), 1),
                     ((-1, 1, 1, 1, 128, 9), 1), ((1, 1, 1, 1, 128, -1), 1), ((1, 1, 1, 1, 64, 9), 2),
                     ((1, 129, 1, 1, 128, 9), 2), ((1, 1, 129, 1, 128, 9), 2)):
        assert size(*args, ctypes.byref(nb)) == st, args
    assert size(1, 1, 1, 1, 128, 9, None) == 1
    for n, H, Hkv, rows in ((1, 16, 1, 16), (1, 17, 1, 32), (8, 8, 1, 64), (8, 64, 8, 64), (21, 3, 1, 64)):
        assert la.attn_verify_workspace_size(3, n, H, Hkv, 128, 99999) == 304 * 56 + 152 * 2 * rows * 130 * 4
    # twice as many runs where few rows meet short contexts
    assert la.attn_verify_workspace_size(3, 1, 16, 1, 128, 1280) == 304 * 56 + 304 * 2 * 16 * 130 * 4
    assert la.attn_verify_workspace_size(3, 1, 16, 1, 128, 1281) == 304 * 56 + 152 * 2 * 16 * 130 * 4
    assert la.attn_verify_workspace_size(3, 1, 17, 1, 128, 512) == 304 * 56 + 152 * 2 * 32 * 130 * 4
    assert la.attn_verify_workspace_size(0, 1, 16, 1, 128, 999) == 0
    # more rows than 64 go the way of prompts
    for n, H, Hkv in ((13, 5, 1), (128, 1, 1), (100, 4, 2), (1, 128, 1)):
        for B, kv in ((1, 200), (3, 5000), (300, 5000)):
            assert la.attn_verify_workspace_size(B, n, H, Hkv, 128, kv) == la.attn_extend_workspace_size(
                B, B * n, H, Hkv, 128, n, kv)
    need = la.attn_verify_workspace_size(2, 3, 2, 1, 128, 272)
    assert tree(lib, width=17, nbytes=need - 1) == 1 and tree(lib, width=17, ws=N) == 1
    assert decode(lib, width=17, nbytes=la.attn_verify_workspace_size(2, 1, 2, 1, 128, 272) - 1) == 1
    # short contexts stay whole
    for n, H, Hkv in ((1, 16, 1), (8, 8, 1), (3, 40, 2)):
        assert la.attn_verify_workspace_size(3, n, H, Hkv, 128, 256) == 0
        assert la.attn_verify_workspace_size(3, n, H, Hkv, 128, 257) > 0
    assert tree(lib, ws=BAD16) == 1 and decode(lib, ws=BAD16) == 1
    assert tree(lib, H=128, P=128, nbytes=1000, width=9) == 1
    size = lib.la_attn_extend_workspace_size
    for args, st in (((-1, 1, 1, 1, 128, 1, 1), 1), ((1, -1, 1, 1, 128, 1, 1), 1), ((1, 1, 3, 2, 128, 1, 1), 1),
                     ((1, 1, 1, 1, 128, -1, 1), 1), ((1, 1, 1, 1, 128, 1, -1), 1), ((1, 1, 1, 1, 64, 1, 1), 2),
                     ((1, 1, 129, 1, 128, 1, 1), 2)):
        assert size(*args, ctypes.byref(nb)) == st, args
    assert size(1, 1, 1, 1, 128, 1, 1, None) == 1
    assert la.attn_extend_workspace_size(0, 0, 1, 1, 128, 0, 0) == 0
    # pieces of items that see more than 256 keys, two per CTA at most
    piece, tails = 2 * 256 * 130 * 4, 152 * 56
    assert la.attn_extend_workspace_size(1, 16384, 32, 8, 128, 16384, 16384) == tails + 152 * piece
    assert la.attn_extend_workspace_size(1, 1, 8, 1, 128, 1, 1000) == tails + 4 * piece
    assert la.attn_extend_workspace_size(100, 25600, 8, 1, 128, 256, 256) == 0


def test_frequencies():
    R, base = 64, 10000.0
    i = np.arange(R // 2)
    f, m = la.rope_freqs(R, base)
    assert np.allclose(f.numpy(), base ** (-2 * i / R), rtol=1e-14, atol=0) and m == 1.0
    g, m = la.rope_freqs(R, base, "linear", 4.0)
    assert np.allclose(g.numpy(), f.numpy() / 4, rtol=1e-14, atol=0) and m == 1.0
    g, m = la.rope_freqs(R, base, "ntk", 4.0)
    assert np.allclose(g.numpy(), (base * 4 ** (R / (R - 2))) ** (-2 * i / R), rtol=1e-13, atol=0) and m == 1.0
    assert math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)  # the slowest pair is interpolated, the first is not
    g, m = la.rope_freqs(R, base, "yarn", 4.0, 4096)
    turns = 4096 * f.numpy() / (2 * np.pi)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1, rel_tol=1e-6)
    assert np.allclose(g.numpy()[turns > 33 * 1.4], f.numpy()[turns > 33 * 1.4], rtol=1e-14, atol=0)
    assert np.allclose(g.numpy()[turns < 0.7], f.numpy()[turns < 0.7] / 4, rtol=1e-14, atol=0)
    assert (np.diff(g.numpy()) < 0).all() and (g.numpy() <= f.numpy() * (1 + 1e-15)).all()
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=math.inf),
               dict(rot_dim=64, scaling="ntk", factor=0.5), dict(rot_dim=64, scaling="linear", factor=math.nan),
               dict(rot_dim=64, scaling="yarn", factor=2.0), dict(rot_dim=64, scaling="yarn", factor=2.0, orig_len=8,
                                                                  beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(la.LAError):
            la.rope_freqs(**kw)
    with pytest.raises(ValueError):
        la.rope_freqs(64, scaling="cubic")


def test_binding_refuses_before_the_library():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    freq = torch.ones(64, dtype=torch.float64)
    pages = bf(2, 1, 16, 128)
    with pytest.raises(ValueError):  # host tensors
        la.rope(bf(2, 256), bf(2, 128), i32(2), freq)
    with pytest.raises(TypeError):
        la.rope(None, bf(2, 128), i32(2), freq)
    with pytest.raises(ValueError):
        la.kv_store(bf(2, 256), bf(2, 128), bf(2, 128), i32(2), freq, pages, pages, i32(2))
    with pytest.raises(ValueError):
        la.attn_extend(bf(2, 256), pages, pages, i32(1, 2), i32(2), i32(1))
    with pytest.raises(ValueError):
        la.attn_decode(bf(1, 256), pages, pages, i32(1, 2), i32(1))
    with pytest.raises(ValueError):
        la.attn_verify_tree(bf(2, 256), pages, pages, i32(1, 2), i32(1), i32(1, 2), 0)
    with pytest.raises(ValueError):
        la.kv_commit(pages, pages, i32(1, 2), i32(1), i32(1, 2), i32(1))
    cpu = torch.device("cpu")
    both = bf(3, 2, 2, 16, 128)
    assert binding._need_pages(both[:, 0], both[:, 1], cpu) == (3, 2, 16, 2 * 2 * 16 * 128)
    assert binding._need_pages(pages, pages, cpu) == (2, 1, 16, 16 * 128)
    for k, v in ((both[:, 0], both[:, 1].contiguous()), (pages, bf(3, 1, 16, 128)), (bf(2, 1, 16, 64), bf(2, 1, 16, 64)),
                 (bf(2, 2, 16, 128).transpose(1, 2),) * 2, (pages[:1].expand(2, 1, 16, 128),) * 2):
        with pytest.raises(ValueError):
            binding._need_pages(k, v, cpu)
    with pytest.raises(TypeError):
        binding._need_pages(pages, pages.float(), cpu)
    with pytest.raises(TypeError):
        binding._need_pages(pages[0], pages, cpu)


def test_oracle_attention_pins():
    """The oracle against small results by hand, and its trees and paths."""
    seen = attn.tree([-1, 0, 0, 2], 6)
    assert seen.astype(int).tolist() == [[1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0], [1, 1, 1, 0, 1, 0], [1, 1, 1, 0, 1, 1]]
    assert attn.path([-1, 0, 0, 2], 3) == [0, 2, 3] and attn.path([-1, 0], -1) == []
    assert attn.causal(2, 3).tolist() == [[True, True, False], [True, True, True]]
    q = np.ones((1, 1, 2))
    k = np.array([[[0.0, 0.0]], [[math.log(3.0), 0.0]], [[9.0, 9.0]]])
    v = np.array([[[1.0, 0.0]], [[5.0, -4.0]], [[100.0, 100.0]]])
    out, size = attn.attend(q, k, v, np.array([[True, True, False]]), 1.0)
    assert np.allclose(out, [[[4.0, -3.0]]]) and np.allclose(size, [[[4.0, 3.0]]])
    assert (attn.attend(q, k, v, np.zeros((1, 3), bool), 1.0)[0] == 0).all()
    x = np.arange(4.0).reshape(1, 1, 4)
    turned = attn.rope(x, [1], [math.pi / 2], True, 2.0)
    assert np.allclose(turned, [[[-2.0, 0.0, 2.0, 3.0]]])
    turned = attn.rope(x, [2 ** 31 - 1], [math.pi / 2, 0.0])  # odd, 3 modulo 4
    assert np.allclose(turned, [[[2.0, 1.0, 0.0, 3.0]]], atol=1e-6)
