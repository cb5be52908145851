"""The RMS norm and its backward on rows far from size 1, where r^3 leaves fp32's range although the
gradient of h does not, against the fp64 oracle.

Bounds.  A row's sums of d products are off by at most (d/32 + 16) u of their terms' magnitudes,
u = 2^-24, and r by half of that and 3 u.  dX = r (u_j - (h r) m), m = r mean(u h): its second term
has three r and one sum beside six roundings, so it is off by at most 2.5 (d/32) + 55 u of its
magnitude, under 3 (d/32 + 24) u; the first by less.  The result's own type adds half a step."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from sample_gradient_clipping_b200 import _lib
from tests.gpu_helpers import host

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()


def _draw(B, T, d, dt, sizes, seed):
    """h with rows of the given sizes, dY, a residual gradient of dX's size, and the gain."""
    rng = np.random.default_rng(seed)
    size = rng.choice(sizes, size=(B, T, 1))
    put = lambda a: torch.from_numpy(a.astype(np.float32)).to(DT[dt]).cuda()  # noqa: E731
    h, dY = put(rng.standard_normal((B, T, d)) * size), put(rng.standard_normal((B, T, d)) / np.sqrt(T * d))
    res = put(rng.standard_normal((B, T, d)) / np.sqrt(T * d) / size)
    gain = torch.from_numpy((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)).cuda()
    return h, dY, res, gain


def _check(h, dY, res, gain, eps, dt):
    B, T, d = h.shape
    hh, yh, gh = host(h), host(dY), host(gain)
    eps64 = float(np.float32(eps))
    sums = (d / 32 + 24) * U32
    r = 1.0 / np.sqrt(np.mean(hh * hh, axis=-1, keepdims=True) + eps64)
    x, u = hh * r, np.abs(yh * gh)
    mags = r * (u + np.abs(x) * np.mean(u * np.abs(x), axis=-1, keepdims=True))
    want, per = oracle.rmsnorm_gradients(hh, gh, yh, eps64)
    if res is not None:
        want = want + host(res)
    dX, got_per, n = _lib.dp_rmsnorm_backward(h, gain, dY, eps=eps, residual_grad=res)
    tol = 3 * sums * mags + (0 if res is None else U32 * np.abs(host(res))) + HALF[dt] * (1 + 2.0 ** -10) * np.abs(want)
    assert np.all(np.isfinite(host(dX))) and np.all(np.abs(host(dX) - want) <= tol)
    mag = np.sum(np.abs(yh * x), axis=1)
    assert np.all(np.abs(host(got_per) - per) <= ((T + 8) * U32 + sums) * mag)
    dX2, _, _ = _lib.dp_rmsnorm_step(h, gain, dY, 1.0, 0.0, 0, 0, 0, eps=eps, residual_grad=res)
    assert torch.equal(dX, dX2)
    y, _ = _lib.dp_rmsnorm(h, gain, eps=eps)
    ref = oracle.rmsnorm(hh, gh, eps64)
    assert np.all(np.abs(host(y) - ref) <= (sums + HALF[dt]) * np.abs(ref))


# One to four vectors a thread, ragged ends, with the gain in registers and read again.
WIDTHS = [("bf16", 64), ("bf16", 4104), ("bf16", 16384), ("f32", 68), ("f32", 2052), ("f32", 8192)]


@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("size,eps", [(1e14, 1e-6), (3e15, 1e-6), (1e16, 1e-6), (1e-13, 0.0), (1e-15, 0.0)])
@pytest.mark.parametrize("dt,d", WIDTHS)
def test_rows_of_one_size(dt, d, size, eps, with_res):
    h, dY, res, gain = _draw(2, 5, d, dt, [size], d)
    _check(h, dY, res if with_res else None, gain, eps, dt)


@pytest.mark.parametrize("dt,d", WIDTHS)
def test_rows_of_all_sizes_together(dt, d):
    h, dY, res, gain = _draw(3, 40, d, dt, [1e-15, 1e-8, 1e-3, 1.0, 1e4, 1e9, 1e13, 1e16], d + 1)
    _check(h, dY, res, gain, 0.0, dt)
