"""The binding refuses buffers that a linear's call would read or write past, before the library
is entered.  A stand-in for the library records what reaches it; no GPU is needed."""
import pytest
import torch

from sample_gradient_clipping_b200 import _lib

B, T, DI, DO, R = 2, 4, 8, 16, 4


class _Library:
    """Every entry point says DP_OK, every size is 256 bytes, and the calls are kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith(("_size", "_size_for")):
            return lambda *a: 256
        return lambda *a: self.calls.append((name, a)) or _lib.DP_OK


@pytest.fixture
def library(monkeypatch):
    stub = _Library()
    monkeypatch.setattr(_lib, "_lib", stub)
    monkeypatch.setattr(_lib, "_stream", lambda stream: 0)
    return stub


def _linear():
    return torch.zeros(B, T, DI), torch.zeros(B, T, DO), torch.zeros(DO, R)


BAD_SUMS = [torch.zeros(DI, R), torch.zeros(DI * DO - 1), torch.zeros(DI, DO, dtype=torch.bfloat16),
            torch.zeros(DO, DI).t(), torch.zeros(DI, 2 * DO)[:, ::2]]


@pytest.mark.parametrize("k", range(len(BAD_SUMS)))
def test_sums_that_do_not_hold_the_gradient(library, k):
    X, dY, _ = _linear()
    G = BAD_SUMS[k]
    for call in (lambda: _lib.dp_clip_accumulate(X, dY, torch.zeros(B), 1.0, G),
                 lambda: _lib.dp_linear_step(X, dY, 1.0, 0.0, 0, 0, 0, G_out=G),
                 lambda: _lib.dp_block_step([{"X": X, "dY": dY, "layer_id": 0, "G_out": G}])):
        with pytest.raises(ValueError):
            call()
    assert library.calls == []


def test_norms_and_projections_of_another_size(library):
    X, dY, P = _linear()
    G, n = torch.zeros(DI, DO), torch.zeros(B)
    for norms in (torch.zeros(B - 1), torch.zeros(B, dtype=torch.float64)):
        for call in (lambda: _lib.dp_clip_accumulate(X, dY, norms, 1.0, G),
                     lambda: _lib.dp_per_sample_norms(X, dY, norms=norms),
                     lambda: _lib.dp_linear_step(X, dY, 1.0, 0.0, 0, 0, 0, norms_out=norms),
                     lambda: _lib.dp_block_step([{"X": X, "dY": dY, "layer_id": 0, "norms_out": norms}])):
            with pytest.raises(ValueError):
                call()
    for bad in (P[1:], P.t(), P.to(torch.bfloat16), torch.zeros(R, DO).t(), torch.zeros(DO)):
        for call in (lambda: _lib.dp_clip_accumulate(X, dY, n, 1.0, G, P=bad),
                     lambda: _lib.dp_per_sample_norms(X, dY, P=bad),
                     lambda: _lib.dp_linear_step(X, dY, 1.0, 0.0, 0, 0, 0, P=bad),
                     lambda: _lib.dp_block_step([{"X": X, "dY": dY, "layer_id": 0, "P": bad}])):
            with pytest.raises(ValueError):
                call()
    assert library.calls == []


def test_buffers_that_hold_it_are_taken(library):
    """Also ones that a caller may have from elsewhere: flat, or larger than needed."""
    X, dY, P = _linear()
    n = torch.zeros(B)
    for G in (torch.zeros(DI, DO), torch.zeros(DI * DO), torch.zeros(DI + 1, DO)):
        _lib.dp_clip_accumulate(X, dY, n, 1.0, G)
        _lib.dp_linear_step(X, dY, 1.0, 0.0, 0, 0, 0, G_out=G, norms_out=n)
        _lib.dp_block_step([{"X": X, "dY": dY, "layer_id": 0, "G_out": G, "norms_out": n}])
    _lib.dp_clip_accumulate(X, dY, n, 1.0, torch.zeros(DI, R), P=P)
    _lib.dp_linear_step(X, dY, 1.0, 0.0, 0, 0, 0, G_out=torch.zeros(DI, R), P=P)
    _lib.dp_linear_step(X, dY, 1.0, 0.0, 0, 0, 0, r=R)           # P drawn by the library
    assert [name for name, _ in library.calls] == ["dp_clip_accumulate", "dp_linear_step", "dp_block_step"] * 3 + \
        ["dp_clip_accumulate", "dp_linear_step", "dp_linear_step"]
