"""The oracle of the embedding, the RMS norm and the Muon step against facts outside itself."""
from __future__ import annotations

import numpy as np
import pytest

import oracle


def test_embedding_step_is_the_linear_step_of_a_one_hot_input():
    rng = np.random.default_rng(0)
    B, T, V, d = 3, 9, 6, 5
    ids = rng.integers(0, V, (B, T))
    dY = rng.standard_normal((B, T, d))
    scale = 1.7
    one_hot = scale * np.eye(V)[ids]
    want = oracle.linear_step(one_hot, dY, 0.8, 0.6, 3, 4, 5)
    got = oracle.embedding_step(ids, dY, V, 0.8, 0.6, 3, 4, 5, scale=scale)
    for key in ("norms", "c", "S", "out"):
        assert np.allclose(got[key], want[key], rtol=1e-13, atol=1e-13), key


def test_embedding_tokens_without_a_row():
    ids = np.array([[2, -1, 7, 2, 0]])
    dY = np.ones((1, 5, 4))
    G = oracle.embedding_gradient(ids[0], dY[0], 7, padding_idx=0)
    want = np.zeros((7, 4))
    want[2] = 2.0                       # the padding row 0, the id -1 and the id 7 name nothing
    assert np.array_equal(G, want)


def test_rmsnorm_gradients_against_differences():
    rng = np.random.default_rng(1)
    B, T, d, eps = 2, 3, 6, 1e-3
    h, dY = rng.standard_normal((B, T, d)), rng.standard_normal((B, T, d))
    gain = 1.0 + 0.3 * rng.standard_normal(d)
    dh, per = oracle.rmsnorm_gradients(h, gain, dY, eps)
    f = lambda hh, g, i=slice(None): float(np.sum(dY[i] * oracle.rmsnorm(hh[i], g, eps)))  # noqa: E731
    e = 1e-6
    for idx in [(0, 0, 0), (1, 2, 5), (0, 1, 3)]:
        up, dn = h.copy(), h.copy()
        up[idx] += e
        dn[idx] -= e
        assert abs((f(up, gain) - f(dn, gain)) / (2 * e) - dh[idx]) <= 1e-8
    for i in range(B):
        for j in range(d):
            up, dn = gain.copy(), gain.copy()
            up[j] += e
            dn[j] -= e
            assert abs((f(h, up, i) - f(h, dn, i)) / (2 * e) - per[i, j]) <= 1e-8


def test_rmsnorm_step_is_the_clipped_sum_of_its_gradients():
    rng = np.random.default_rng(2)
    h, dY, res = (rng.standard_normal((4, 5, 8)) for _ in range(3))
    gain = np.ones(8)
    out = oracle.rmsnorm_step(h, gain, dY, 0.9, 0.5, 1, 2, 3, 1e-6, residual_grad=res)
    c = oracle.clip_factors(out["norms"], 0.9)
    assert np.allclose(out["S"], c @ out["per_sample"], rtol=1e-13, atol=1e-13)
    assert np.all(c * out["norms"] <= 0.9 * (1 + 1e-12))
    assert np.allclose(out["out"] - out["S"], oracle.noise(1, 8, 0.45, 1, 2, 3)[0], rtol=0, atol=1e-15)
    dh, _ = oracle.rmsnorm_gradients(h, gain, dY, 1e-6)
    assert np.allclose(out["dX"], dh + res, rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("m,n", [(6, 9), (9, 6), (7, 7)])
def test_newton_schulz_maps_singular_values_alone(m, n):
    """On G = U diag(s) V^T the iteration acts on each s by its polynomial and keeps U and V."""
    rng = np.random.default_rng(m * n)
    G = rng.standard_normal((m, n))
    U, s, Vt = np.linalg.svd(G, full_matrices=False)
    x = s / (np.linalg.norm(s) + 1e-7)
    a, b, c = oracle.NEWTON_SCHULZ
    for _ in range(5):
        x = a * x + b * x ** 3 + c * x ** 5
    assert np.allclose(oracle.newton_schulz(G), (U * x) @ Vt, rtol=0, atol=1e-9)
    assert np.array_equal(oracle.newton_schulz(np.zeros((m, n))), np.zeros((m, n)))


def test_muon_step():
    rng = np.random.default_rng(5)
    W, R, M = (rng.standard_normal((4, 6)) for _ in range(3))
    for nesterov in (False, True):
        W1, M1 = oracle.muon_step(W, R, M, 0.1, 0.9, nesterov, 0.2, 0.5, 1.5)
        assert np.allclose(M1, 0.9 * M + 0.5 * R)
        U = oracle.newton_schulz(0.5 * R + 0.9 * M1 if nesterov else M1)
        assert np.allclose(W1, 0.98 * W - 0.15 * U)
    # With no momentum and no decay the weights move along the orthogonalised gradient alone.
    W2, M2 = oracle.muon_step(W, R, np.zeros_like(M), 0.1, 0.0, False, 0.0, 1.0, 1.0)
    assert np.allclose((W - W2) / 0.1, oracle.newton_schulz(R)) and np.allclose(M2, R)
