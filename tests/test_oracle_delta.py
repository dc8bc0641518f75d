"""CPU pins of the gated delta rule's fp64 oracle and of the packed store's, independent of their code."""
import numpy as np
import pytest

from oracle import delta


def _inputs(n, Hk, H, D, seed=0):
    r = np.random.default_rng(seed)
    k = r.standard_normal((n, Hk, D))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return (r.standard_normal((n, Hk, D)), k, r.standard_normal((n, H, D)),
            -r.exponential(0.2, (n, H)), r.uniform(0, 1, (n, H)), r.standard_normal((H, D, D)))


def test_matrix_form():
    """S_t = e^g (I - beta k k^T) S_{t-1} + beta k v^T: the transition as one matrix."""
    q, k, v, g, beta, S0 = _inputs(20, 1, 2, 16)
    out, S, _ = delta.run(q, k, v, g, beta, S0)
    for h in range(2):
        M = S0[h].copy()
        for t in range(20):
            kt = k[t, 0]
            M = np.exp(g[t, h]) * (np.eye(16) - beta[t, h] * np.outer(kt, kt)) @ M
            M += beta[t, h] * np.outer(kt, v[t, h])
            np.testing.assert_allclose(out[t, h], q[t, 0] @ M / 4, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(S[h], M, rtol=1e-12, atol=1e-12)


def test_triangular_solve_form():
    """The closed form over a whole request: (I + A) U = beta V - beta e^G K S0."""
    q, k, v, g, beta, S0 = _inputs(37, 2, 4, 8, seed=1)
    out, S, _ = delta.run(q, k, v, g, beta, S0)
    for h in range(4):
        K, Q, G = k[:, h // 2], q[:, h // 2], np.cumsum(g[:, h])
        dec = np.tril(np.exp(np.minimum(G[:, None] - G[None, :], 0)))
        A = np.tril(beta[:, h, None] * (K @ K.T) * dec, -1)
        U = np.linalg.solve(np.eye(37) + A, beta[:, h, None] * (v[:, h] - np.exp(G)[:, None] * (K @ S0[h])))
        o = np.exp(G)[:, None] * (Q @ S0[h]) + ((Q @ K.T) * dec) @ U
        np.testing.assert_allclose(out[:, h], o * 8 ** -0.5, rtol=1e-10, atol=1e-11)
        end = np.exp(G[-1]) * S0[h] + (K * np.exp(G[-1] - G)[:, None]).T @ U
        np.testing.assert_allclose(S[h], end, rtol=1e-10, atol=1e-11)


def test_write_then_read():
    """beta = 1 and a unit key: the state answers the key with the value just written."""
    q, k, v, g, _, S0 = _inputs(9, 1, 1, 32, seed=2)
    out, _, states = delta.run(k, k, v, g, np.ones((9, 1)), S0, keep=True)
    np.testing.assert_allclose(out * 32 ** 0.5, v, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(np.einsum("thkv,tk->thv", states, k[:, 0]), v, rtol=1e-12, atol=1e-12)


def test_no_writing_and_full_forgetting():
    q, k, v, g, beta, S0 = _inputs(3, 1, 2, 8, seed=3)
    _, S, _ = delta.run(q, k, v, g, np.zeros_like(beta), S0)
    np.testing.assert_allclose(S, np.exp(g.sum(0))[:, None, None] * S0, rtol=1e-12)
    g[1] = -np.inf
    _, a, _ = delta.run(q, k, v, g, beta, S0)
    _, b, _ = delta.run(q[1:], k[1:], v[1:], np.concatenate([np.zeros((1, 2)), g[2:]]), beta[1:],
                        np.zeros_like(S0))
    np.testing.assert_allclose(a, b, rtol=1e-12)


def test_split_and_modes_agree():
    q, k, v, g, beta, S0 = _inputs(12, 2, 2, 8, seed=4)
    pool = np.stack([S0, 2 * S0, np.full_like(S0, np.nan)])
    f = lambda x: x.reshape(12, -1)  # noqa: E731
    a, pa = delta.extend(f(q), f(k), f(v), g, beta, pool, [1], [0, 12], [1], 2, 2, 8, True)
    cut = [0, 5]
    o1, p1 = delta.extend(f(q)[:5], f(k)[:5], f(v)[:5], g[:5], beta[:5], pool, [1], cut, [1], 2, 2, 8, True)
    o2, p2 = delta.extend(f(q)[5:], f(k)[5:], f(v)[5:], g[5:], beta[5:], p1, [1], [0, 7], [1], 2, 2, 8, True)
    np.testing.assert_allclose(np.concatenate([o1, o2]), a, rtol=1e-12)
    np.testing.assert_allclose(p2[1], pa[1], rtol=1e-12)
    o3, inter = delta.verify_chain(f(q), f(k), f(v), g, beta, pool, [1], 12, 2, 2, 8, True)
    np.testing.assert_allclose(o3, a, rtol=1e-12)
    np.testing.assert_allclose(inter[0, -1], pa[1], rtol=1e-12)
    o4, p4 = delta.decode(f(q)[:1], f(k)[:1], f(v)[:1], g[:1], beta[:1], pool, [1], 2, 2, 8, True)
    np.testing.assert_allclose(o4, a[:1], rtol=1e-12)
    np.testing.assert_allclose(p4[1], inter[0, 0], rtol=1e-12)
    assert np.isnan(p4[2]).all()
    # without a prefix the slot is never read
    _, p = delta.extend(f(q), f(k), f(v), g, beta, pool, [2], [0, 12], [0], 2, 2, 8)
    assert np.isfinite(p[2]).all()


def test_unit_norm():
    q, k, v, g, beta, S0 = _inputs(5, 1, 1, 8, seed=5)
    a = delta.run(q * 3, k * 7, v, g, beta, S0, qk_l2norm=True)
    b = delta.run(q / np.linalg.norm(q, axis=-1, keepdims=True), k, v, g, beta, S0)
    for x, y in zip(a[:2], b[:2]):
        np.testing.assert_allclose(x, y, rtol=2e-6, atol=2e-6)  # the 1e-6 under the root


@pytest.mark.parametrize("scale", [1.0, 1e-30, 3e38, 2.0 ** -140])
def test_pack_error_and_idempotence(scale):
    r = np.random.default_rng(6)
    with np.errstate(over="ignore"):
        x = np.clip(r.standard_normal((7, 128)) * 0.3, -1, 1).astype(np.float32) * np.float32(scale)
    codes, scales = delta.pack(x)
    y = delta.unpack(codes, scales)
    top = np.abs(x.reshape(7, 4, 32).astype(np.float64)).max(-1)
    err = np.abs(y - x).reshape(7, 4, 32).max(-1)
    assert (err <= np.maximum(top / 127, 2.0 ** -128)).all()
    again = delta.pack(y)
    assert np.array_equal(again[0], codes) and np.array_equal(again[1], scales)


def test_pack_borders():
    x = np.zeros((1, 128))
    x[0, 0], x[0, 32], x[0, 64], x[0, 96] = 127.5, 127.4, np.inf, 0.0
    codes, scales = delta.pack(x)
    assert scales.tolist() == [[128, 127, 255, 0]]  # 127.5 rounds to 128 (even): the next scale
    assert codes[0, 0] == 64 and codes[0, 32] == 127 and codes[0, 64] == 0
    y = delta.unpack(codes, scales)
    assert np.isnan(y[0, 64:96]).all() and (y[0, 96:] == 0).all() and y[0, 0] == 128


def test_pack_of_the_largest_values_stays_finite():
    x = np.full((1, 128), np.finfo(np.float32).max, np.float64)
    x[0, 32:64] = 127.5 * 2.0 ** 120
    codes, scales = delta.pack(x)
    assert scales.tolist() == [[248, 248, 248, 248]]
    assert codes[0, 0] == 127 and codes[0, 32] == 64
    assert np.isfinite(delta.unpack(codes, scales).astype(np.float32)).all()
