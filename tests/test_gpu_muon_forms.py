"""The Newton-Schulz products of large matrices: tiles of SM pairs, and CTAs that take several tiles.

Which form a product takes is restated here from sizes and the number of SMs, and every case says
which forms it is for.  Bounds as in the other tests of these products: twice what the library's
roundings alone cost (computed in fp64 for the same input), the fp32 additions, and a bf16 result's
half step; here also for every block of 64 x 64 by itself, where the roundings' cost is that of the
block that loses most (they are thousands of independent errors of one size)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from sample_gradient_clipping_b200 import _lib

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()


def _form(m, n, k, symmetric, sms):
    """("pair" | "single" | "split", most tiles that one CTA takes) of an m x n product over k columns."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    units = lambda t: up(m, t) * (up(m, t) + 1) // 2 if symmetric else up(m, t) * up(n, t)  # noqa: E731
    u1, u2, blocks = units(128), units(256), up(k, 64)
    if symmetric and ((u1 * 4 <= 128 and blocks >= 16) or (u1 * 2 <= sms and blocks >= 24)):
        return "split", 1
    if up(u2, sms // 2) < up(u1, sms):
        return "pair", up(u2, sms // 2)
    return "single", up(u1, sms)


def _forms(rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return _form(m, m, n, True, sms), _form(m, m, m, True, sms), _form(m, n, m, False, sms)


def _iteration(G, steps, rounded):
    """In fp64 on the device; `rounded`: with the library's fp16 planes and nothing else."""
    a, b, c = oracle.NEWTON_SCHULZ
    f16 = (lambda x: x.to(torch.float16).double()) if rounded else (lambda x: x)
    tall = G.shape[0] > G.shape[1]
    X = G.double().T if tall else G.double()
    X = X / (X.norm() + 1e-7)
    eye = torch.eye(X.shape[0], dtype=torch.float64, device=G.device)
    for _ in range(steps):
        hi = f16(X)
        if rounded:
            X = hi + f16((X - hi) * 2048) / 2048
        A = hi @ hi.T
        t = float(A.trace()) / len(A)
        delta = b * t + c * t * t if rounded else 0.0
        A = f16(A)
        X = (a + delta) * X + f16(b * A + c * (A @ A) - delta * eye) @ hi
    return X.T if tall else X


def _block_norms(x):
    pad = torch.nn.functional.pad(x, (0, -x.shape[1] % 64, 0, -x.shape[0] % 64))
    return pad.reshape(pad.shape[0] // 64, 64, -1, 64).square().sum((1, 3)).sqrt()


def _gradient(rows, cols, seed):
    """A few strong directions over noise, as a privatised gradient has."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(rows, 4) @ r(4, cols) + r(rows, cols)


PAIR, PAIRS, SINGLES = ("pair", 1), ("pair", 2), ("single", 2)
CASES = [(2312, 2440, (PAIR, PAIR, PAIRS)), (2440, 2312, (PAIR, PAIR, PAIRS)), (2824, 3000, (SINGLES, SINGLES, PAIRS)),
         (2952, 3104, (PAIRS, PAIRS, ("pair", 3))),
         (1504, 4000, (("single", 1), ("single", 1), PAIRS)), (4000, 1504, (("single", 1), ("single", 1), PAIRS)),
         (1608, 2600, (("single", 1), ("single", 1), SINGLES)), (2600, 1608, (("single", 1), ("single", 1), SINGLES))]


@pytest.mark.parametrize("rows,cols,forms", CASES, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_orthogonalize(rows, cols, forms):
    assert _forms(rows, cols) == forms
    G = _gradient(rows, cols, rows)
    want = _iteration(G, 5, False)
    lost = _iteration(G, 5, True) - want
    U = _lib.dp_orthogonalize(G)
    off = U.double() - want
    half = 2.0 ** -8 + 2000 * U32
    assert float(off.norm()) <= 2 * float(lost.norm()) + half * float(want.norm())
    assert torch.all(_block_norms(off) <= 2 * _block_norms(lost).max() + half * _block_norms(want))
    assert torch.equal(_lib.dp_orthogonalize(G), U)


@pytest.mark.parametrize("rows,cols,forms", CASES, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_muon_step(rows, cols, forms):
    R, M0 = _gradient(rows, cols, 1), _gradient(rows, cols, 2)
    W0 = _gradient(rows, cols, 3) / 64
    W, M = W0.clone(), M0.clone()
    lr, mu, wd, gs, us = (float(np.float32(v)) for v in (0.02, 0.95, 0.1, 0.25, 0.7))
    _lib.dp_muon_step(W, R, M, lr, momentum=mu, weight_decay=wd, grad_scale=gs, update_scale=us)
    Mo = mu * M0.double() + gs * R.double()
    # One product rounded, one fused multiply and addition.
    assert torch.all((M.double() - Mo).abs() <= 2 * U32 * ((mu * M0.double()).abs() + (gs * R.double()).abs()))
    u = gs * R.double() + mu * Mo
    exact = _iteration(u, 5, False)
    lost = _iteration(u, 5, True) - exact
    off = W.double() - ((1 - lr * wd) * W0.double() - lr * us * exact)
    # keep and rate are rounded to fp32, and the update is one product and one fused operation.
    tol = lr * us * (2 * _block_norms(lost).max() + 2000 * U32 * _block_norms(exact)) + 3 * U32 * _block_norms(W0.double())
    assert torch.all(_block_norms(off) <= tol)


@pytest.mark.parametrize("rows,cols", [(72, 136), (136, 72), (16, 2056), (328, 200), (200, 2000), (1096, 1096), (2312, 2440)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinities_and_nan_reach_every_value(rows, cols, value):
    """||G|| is then not a number or infinite, the mean eigenvalue is not a number, and so is all of X."""
    G = torch.randn(rows, cols, device="cuda")
    G[rows - 3, 5] = value
    assert torch.isnan(_lib.dp_orthogonalize(G)).all()
    assert torch.isnan(_lib.dp_orthogonalize(G.to(torch.bfloat16))).all()
    W = torch.zeros(rows, cols, device="cuda")
    _lib.dp_muon_step(W, G, torch.zeros_like(G), 0.1)
    assert torch.isnan(W).all()
