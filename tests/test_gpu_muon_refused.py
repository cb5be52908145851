"""dp_muon_step whose launches are refused on the host, through the library's fake of the launch call."""
import pytest
import torch

from sample_gradient_clipping_b200 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()


# One launch for all products, single SMs, K split among SMs, and tall matrices.
@pytest.mark.parametrize("m,n", [(64, 32), (200, 328), (328, 200), (1024, 1032)])
def test_refused_launches(m, n):
    """The call reports it.  A call whose first launch is refused has changed nothing; after any other
    the caller's copies of W and M make the same step again, bit for bit."""
    L = _lib.lib()
    W0, R, M0 = (torch.sin(k + torch.arange(m * n, device="cuda", dtype=torch.float32)).reshape(m, n) for k in range(3))
    before = _lib.kernel_launches()
    want = [t.clone() for t in _lib.dp_muon_step(W0.clone(), R, M0.clone(), 0.1)]
    for k in range(_lib.kernel_launches() - before):
        W, M = W0.clone(), M0.clone()
        try:
            assert L.dp_selftest_fail_launches(k, 1, 2) == _lib.DP_OK      # cudaErrorMemoryAllocation
            with pytest.raises(_lib.DPError) as err:
                _lib.dp_muon_step(W, R, M, 0.1)
        finally:
            L.dp_selftest_fail_launches(0, 0, 0)
        assert err.value.status == _lib.DP_ERR_CUDA
        if k == 0:
            assert torch.equal(W, W0) and torch.equal(M, M0)
        assert torch.equal(W, W0)                       # the weights are the last launch's
        W.copy_(W0)
        M.copy_(M0)
        assert all(torch.equal(a, b) for a, b in zip(_lib.dp_muon_step(W, R, M, 0.1), want))
