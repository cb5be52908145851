"""Norm and Muon calls that overlap on two streams, each with its own buffers, give the bits of calls
that follow one another."""
import pytest
import torch

from sample_gradient_clipping_b200 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()


def _norms(k):
    g = torch.Generator(device="cuda").manual_seed(k)
    h, dy = (torch.randn(6, 300, 1032, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    gain = torch.randn(1032, generator=g, device="cuda")
    return lambda: _lib.dp_rmsnorm_step(h, gain, dy, 1.0, 0.5, k, 2, 3) + _lib.dp_rmsnorm(h, gain, residual=dy)


def _muon(k, m=264, n=520):
    g = torch.Generator(device="cuda").manual_seed(k)
    W, R, M = (torch.randn(m, n, generator=g, device="cuda") for _ in range(3))
    return lambda: _lib.dp_muon_step(W.clone(), R, M.clone(), 0.1) + (_lib.dp_orthogonalize(R),)


@pytest.mark.parametrize("make", [_norms, _muon, lambda k: _muon(k, 96, 1400), lambda k: _muon(k, 1400, 1608)],
                         ids=["norms", "muon", "muon, one launch", "muon, large"])
def test_overlapping_calls(make):
    calls = [make(0), make(1)]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for s, call, out in zip(streams, calls, got):
            with torch.cuda.stream(s):
                out.append(call())
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        for o in out:
            assert all(torch.equal(a, b) for a, b in zip(o, w))
