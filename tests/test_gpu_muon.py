"""dp_orthogonalize and dp_muon_step against the fp64 oracle.

Bounds.  The products read operands rounded to fp16 and add in fp32.  What those roundings cost is
computed for each test's own input: `_rounded_iteration` carries the iteration out in fp64 with the
library's roundings alone (the planes of X, A and B in fp16).  Another order of the fp32 additions
moves some of these roundings to the other side, which makes an independent error of the same size
or less, so the library may be twice as far off; the fp32 additions themselves are k u, u = 2^-24,
far below.  A bf16 result adds its own rounding, at most 2^-8 of each value."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from sample_gradient_clipping_b200 import _lib
from tests.gpu_helpers import host

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()


def _f16(x):
    return x.astype(np.float16).astype(np.float64)


def _rounded_iteration(G, steps=5):
    a, b, c = oracle.NEWTON_SCHULZ
    X = np.asarray(G, dtype=np.float64)
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (np.linalg.norm(X) + 1e-7)
    for _ in range(steps):
        hi = _f16(X)
        X = hi + _f16((X - hi) * 2048) / 2048
        A = hi @ hi.T
        t = np.trace(A) / len(A)
        delta = b * t + c * t * t
        A = _f16(A)
        B = _f16(b * A + c * (A @ A) - delta * np.eye(len(A)))
        X = (a + delta) * X + B @ hi
    return X.T if tall else X


def _matrix(m, n, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "gauss":
        return rng.standard_normal((m, n))
    if kind == "spikes":          # a few strong directions over noise
        k = min(4, m, n)
        return rng.standard_normal((m, k)) @ rng.standard_normal((k, n)) * 3 + rng.standard_normal((m, n)) * 0.3
    if kind == "rows":            # rows of very different size
        return rng.standard_normal((m, n)) * np.exp(2 * rng.standard_normal((m, 1)))
    return rng.standard_normal((m, 3)) @ rng.standard_normal((3, n))   # rank 3


SHAPES = [(8, 8), (8, 200), (200, 8), (64, 32), (128, 128), (136, 120), (264, 264), (128, 1024), (1024, 128),
          (16, 256), (40, 264), (128, 512), (72, 520), (2048, 120), (104, 2056), (4096, 128), (24, 4104), (128, 1416), (88, 1992),
          (520, 1400), (1400, 520), (1096, 1096),
          (136, 2000), (1544, 264), (1032, 1096), (1160, 1544)]   # symmetric products split over 4 and 2 SMs a tile


def _check(G_h, G_d, steps=5):
    U = _lib.dp_orthogonalize(G_d, steps=steps)
    want = oracle.newton_schulz(G_h, steps)
    lost = np.linalg.norm(_rounded_iteration(G_h, steps) - want)
    off = np.linalg.norm(host(U) - want)
    tol = 2 * lost + (2.0 ** -8 + 2000 * U32) * np.linalg.norm(want)
    assert U.dtype == torch.bfloat16 and off <= tol, (off, tol)
    return U


@pytest.mark.parametrize("m,n,kind", [(m, n, k) for m, n in SHAPES for k in ("gauss", "spikes", "rows", "rank3")
                                      if k == "gauss" or m * n < 600_000])
def test_orthogonalize(m, n, kind):
    G = _matrix(m, n, kind, m + n).astype(np.float32)
    _check(G.astype(np.float64), torch.from_numpy(G).cuda())


def test_orthogonalize_bf16_scales_and_steps():
    G = torch.from_numpy(_matrix(136, 328, "gauss", 3).astype(np.float32)).to(torch.bfloat16)
    U = _check(G.double().numpy(), G.cuda())
    # Powers of two change the exponent alone (the 1e-7 beside the norm is below it by 2^-40 either way).
    for s in (2.0 ** 60, 2.0 ** 20):
        assert torch.equal(_lib.dp_orthogonalize((G.float() * s).cuda()), _lib.dp_orthogonalize(G.float().cuda() * 2.0 ** 21))
    for steps in (1, 2, 9):
        _check(G.double().numpy(), G.cuda(), steps)
    # Five steps bring the singular values of a Gaussian matrix near 1.
    s = np.linalg.svd(host(U), compute_uv=False)
    assert 0.6 < s.min() and s.max() < 1.3


def test_zeros_and_nan():
    assert float(_lib.dp_orthogonalize(torch.zeros(136, 72, device="cuda")).abs().max()) == 0.0
    G = torch.randn(72, 136, device="cuda")
    G[3, 5] = float("nan")
    assert torch.isnan(_lib.dp_orthogonalize(G)).all()
    G[3, 5] = float("inf")
    assert torch.isnan(_lib.dp_orthogonalize(G)).any()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("m,n", [(64, 32), (32, 64), (136, 520), (520, 136), (1024, 1032)])
def test_muon_two_steps(m, n, nesterov):
    rng = np.random.default_rng(m + n)
    W0 = (rng.standard_normal((m, n)) / np.sqrt(m)).astype(np.float32)
    W, M = torch.from_numpy(W0).cuda(), torch.zeros(m, n, device="cuda")
    lr, mu, wd, gs, us = (float(np.float32(v)) for v in (0.02, 0.95, 0.1, 1 / 48, 0.7))
    for _ in range(2):
        R = rng.standard_normal((m, n)).astype(np.float32)
        Wh, Mh = host(W), host(M)
        out = _lib.dp_muon_step(W, torch.from_numpy(R).cuda(), M, lr, momentum=mu, nesterov=nesterov, weight_decay=wd,
                                grad_scale=gs, update_scale=us)
        assert out[0] is W and out[1] is M
        Wo, Mo = oracle.muon_step(Wh, R, Mh, lr, mu, nesterov, wd, gs, us)
        # One product rounded, one fused multiply and addition.
        assert np.all(np.abs(host(M) - Mo) <= 2 * U32 * (np.abs(mu * Mh) + np.abs(gs * R)))
        g = gs * R.astype(np.float64)
        lost = np.linalg.norm(_rounded_iteration(g + mu * Mo if nesterov else Mo) -
                              oracle.newton_schulz(g + mu * Mo if nesterov else Mo))
        # keep and rate are rounded to fp32, and the update is one product and one fused operation.
        tol = lr * us * (2 * lost + 2000 * U32 * np.sqrt(min(m, n))) + 3 * U32 * np.linalg.norm(Wh)
        assert np.linalg.norm(host(W) - Wo) <= tol


def test_weights_without_a_learning_rate():
    W = torch.randn(64, 128, device="cuda")
    M = torch.randn(64, 128, device="cuda")
    R = torch.randn(64, 128, device="cuda")
    W0, M0 = W.clone(), M.clone()
    _lib.dp_muon_step(W, R, M, 0.0, momentum=0.5)
    assert torch.equal(W, W0) and torch.equal(M, M0 * 0.5 + R)


def test_bits_repeat_and_surroundings_stay():
    for m, n in ((264, 520), (520, 264)):
        G = torch.randn(m, n, device="cuda")
        need = _lib.muon_workspace_size(m, n)
        ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        buf = torch.full((m + 2, n), 7.0, device="cuda", dtype=torch.bfloat16)
        first = None
        for _ in range(4):
            ws[:need] = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
            U = _lib.dp_orthogonalize(G, U=buf[1:m + 1], workspace=ws[:need])
            first = U.clone() if first is None else first
            assert torch.equal(U, first) and _lib.dp_workspace_status(ws) == _lib.DP_OK
        assert (ws[need:] == 0x5A).all() and (buf[0] == 7.0).all() and (buf[m + 1] == 7.0).all()


def test_graph_replays_follow_inputs():
    W, R, M = (torch.randn(256, 136, device="cuda") for _ in range(3))
    ws = torch.empty(_lib.muon_workspace_size(256, 136), dtype=torch.uint8, device="cuda")
    _lib.dp_muon_step(W.clone(), R, M.clone(), 0.01, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.dp_muon_step(W, R, M, 0.01, workspace=ws)
    for _ in range(3):
        R.copy_(torch.randn_like(R))
        Wc, Mc = W.clone(), M.clone()
        graph.replay()
        _lib.dp_muon_step(Wc, R, Mc, 0.01)
        assert torch.equal(W, Wc) and torch.equal(M, Mc)


def test_a_private_step_then_muon():
    """The clipped, noised gradient of a linear, taken by the optimizer as it is used."""
    X = torch.randn(4, 64, 128, device="cuda").to(torch.bfloat16)
    dY = (torch.randn(4, 64, 256, device="cuda") / 128).to(torch.bfloat16)
    G, _ = _lib.dp_linear_step(X, dY, 1.0, 0.5, 1, 2, 3)
    W = torch.randn(128, 256, device="cuda") / 11
    Wh = host(W)
    M = torch.zeros_like(W)
    _lib.dp_muon_step(W, G, M, 0.02, grad_scale=0.25)
    Wo, _ = oracle.muon_step(Wh, host(G), np.zeros((128, 256)), float(np.float32(0.02)), float(np.float32(0.95)), True, 0.0,
                             0.25, 1.0)
    moved = np.linalg.norm(Wo - Wh)
    assert np.linalg.norm(host(W) - Wo) <= 5e-3 * moved


def test_binding_refuses():
    G = torch.zeros(16, 16, device="cuda")
    with pytest.raises(ValueError):
        _lib.dp_orthogonalize(G.t()[:8].t())
    with pytest.raises(ValueError):
        _lib.dp_orthogonalize(G.reshape(4, 4, 16))
    with pytest.raises(TypeError):
        _lib.dp_orthogonalize(G.half())
    with pytest.raises(_lib.DPError):
        _lib.dp_orthogonalize(torch.zeros(16, 12, device="cuda"))
    with pytest.raises(_lib.DPError):
        _lib.dp_orthogonalize(G, steps=0)
    with pytest.raises(_lib.DPError):
        _lib.dp_muon_step(G, G, torch.zeros_like(G), 0.1)
    with pytest.raises(ValueError):
        _lib.dp_muon_step(G, torch.zeros(16, 8, device="cuda"), torch.zeros_like(G), 0.1)
