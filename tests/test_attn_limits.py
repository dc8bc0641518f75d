"""Bounds of the attention entry points, on the host: what a call refuses before anything is launched."""
import ctypes

import numpy as np
import pytest

import lightning_attention_gb300 as la
from lightning_attention_gb300 import _build, binding

OK = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def extend(lib, H, Hkv, out=OK):
    return lib.la_attn_extend(OK, 0, OK, OK, 0, 4, 16, OK, 2, OK, OK, out, 1, 8, H, Hkv, 128, 8, 32, 0.1, OK, 1 << 40, None)


def decode(lib, H, Hkv, out=OK):
    return lib.la_attn_decode(OK, 0, OK, OK, 0, 4, 16, OK, 2, OK, out, 2, H, Hkv, 128, 0.1, OK, 1 << 40, None)


def tree(lib, H, Hkv, out=OK):
    return lib.la_attn_verify_tree(OK, 0, OK, OK, 0, 4, 16, OK, 2, OK, OK, out, 2, 3, H, Hkv, 128, 0.1, OK, 1 << 40, None)


@pytest.mark.parametrize("call", [extend, decode, tree])
def test_number_of_heads(lib, call):
    """The kernels hold a place among a request's rows, up to 128 * H * 128 / 8 pieces and 64 * H * 128 values, in 32 bits."""
    for H, Hkv in ((65537, 65537), (1 << 17, 1 << 10), (1 << 24, 1 << 24), ((1 << 31) - 1, (1 << 31) - 1)):
        assert call(lib, H, Hkv) == 2, (H, Hkv)
    # the largest number gets as far as its pointers
    assert call(lib, 65536, 512, out=None) == 1


def test_a_bound_of_no_tokens_leaves_a_cta(lib):
    """It reports the requests that have tokens all the same (and would have a partial result of two items)."""
    n = ctypes.c_size_t(0)
    assert lib.la_attn_extend_workspace_size(1, 8, 2, 1, 128, 0, 256, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.la_attn_extend_workspace_size(1, 8, 2, 1, 128, 0, 300, ctypes.byref(n)) == 0
    assert n.value == 152 * 56 + 2 * (2 * 256 * 130 * 4)


def test_number_of_heads_of_a_workspace(lib):
    n = ctypes.c_size_t(0)
    for H, st in ((65536, 0), (65537, 2), (1 << 24, 2)):
        assert lib.la_attn_verify_workspace_size(2, 1, H, H, 128, 1000, ctypes.byref(n)) == st
        assert lib.la_attn_extend_workspace_size(2, 9, H, H, 128, 9, 1000, ctypes.byref(n)) == st


@pytest.mark.parametrize("keep", [0, 1])
def test_commit_with_options(lib, keep):
    def commit(kp=OK, lens=OK, B=2, n=3, Hkv=1, D=128, P=16):
        return lib.la_kv_commit_ex(kp, OK, 0, 4, P, OK, 2, OK, OK, OK, lens, keep, B, n, Hkv, D, None)

    for kw, st in (({"B": -1}, 1), ({"n": 0}, 1), ({"n": 129}, 2), ({"Hkv": 0}, 1), ({"D": 64}, 2), ({"P": 48}, 2),
                   ({"kp": None}, 1), ({"lens": None}, 1), ({"lens": ctypes.c_void_p(4098)}, 1), ({"B": 0, "lens": None}, 0)):
        assert commit(**kw) == st, kw


@pytest.mark.parametrize("orig_len", [1, 5, 6, 7, 40, 4096])
@pytest.mark.parametrize("beta_slow", [1.0, 20.0])
def test_yarn_keeps_to_its_bounds(orig_len, beta_slow):
    """Pairs that turn less than beta_slow times over the original length are interpolated in full, and those that turn
    more than beta_fast times not at all, however short that length (the ramp's ends are whole pair numbers, so that
    a pair beside an end may be on it)."""
    R, base, factor, fast = 64, 10000.0, 4.0, 32.0
    f = base ** (-2 * np.arange(R // 2) / R)
    g, _ = la.rope_freqs(R, base, "yarn", factor, orig_len, fast, beta_slow)
    turns, step = orig_len * f / (2 * np.pi), base ** (2 / R)  # from one pair to the next
    few, many = turns * step < beta_slow, turns > fast * step
    few[0] = turns[0] < beta_slow  # no pair before it
    assert np.allclose(g.numpy()[few], f[few] / factor, rtol=1e-14, atol=0)
    assert np.allclose(g.numpy()[many], f[many], rtol=1e-14, atol=0)
    assert (g.numpy() <= f * (1 + 1e-15)).all() and (g.numpy() >= f / factor * (1 - 1e-15)).all()
