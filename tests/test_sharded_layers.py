"""The sharded step over linears (projected ones among them), embedding tables and norm gains.

What LibraryOps asks of the library for each kind of layer is checked against a stand-in that
computes with the fp64 oracle, on two gloo ranks too.  No GPU is needed."""
import os
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import oracle
from sample_gradient_clipping_b200 import _lib, sharded

B, T, V, D, DI, DO, R, EPS = 5, 6, 11, 8, 8, 12, 4, 1e-5


class OracleLibrary:
    """The binding's functions that LibraryOps calls, by the oracle, on fp64 CPU tensors."""

    @staticmethod
    def _dtype_code(X):
        return _lib.DP_F32

    @staticmethod
    def workspace_size(*a):
        return 256

    @staticmethod
    def embedding_workspace_size(B, T, V, d, dtype_code):
        return 1000 * B

    @staticmethod
    def rmsnorm_workspace_size(B, T, d, dtype_code):
        return 500 * B

    @staticmethod
    def _fill(out, value):
        value = torch.from_numpy(np.asarray(value))
        if out is None:
            return value
        assert out.shape == value.shape
        return out.copy_(value)

    @staticmethod
    def _np(t):
        return None if t is None else t.numpy()

    def dp_per_sample_norms(self, X, dY, P=None, method="auto", norms=None, workspace=None, stream=None):
        return self._fill(norms, oracle.per_sample_norms(X.numpy(), dY.numpy(), self._np(P)))

    def dp_clip_accumulate(self, X, dY, norms, C, G_sum, P=None, workspace=None, stream=None):
        c = oracle.clip_factors(norms.numpy(), C)
        G_sum += torch.from_numpy(oracle.clipped_sum(X.numpy(), dY.numpy(), c, self._np(P))).to(G_sum.dtype)
        return G_sum

    def dp_linear_step(self, X, dY, C, sigma, seed, step, layer_id, P=None, r=0, method="auto", norms_out=None,
                       G_out=None, workspace=None, stream=None):
        assert sigma == 0
        n = oracle.per_sample_norms(X.numpy(), dY.numpy(), self._np(P))
        S = oracle.clipped_sum(X.numpy(), dY.numpy(), oracle.clip_factors(n, C), self._np(P))
        return self._fill(G_out, S), self._fill(norms_out, n)

    def _gradients(self, ids, dY, V, scale, padding_idx):
        return np.stack([oracle.embedding_gradient(ids[i].numpy(), dY[i].numpy(), V, scale, padding_idx)
                         for i in range(len(ids))])

    def dp_embedding_per_sample_norms(self, ids, dY, V, scale=1.0, padding_idx=None, norms=None, workspace=None,
                                      stream=None):
        return self._fill(norms, np.linalg.norm(self._gradients(ids, dY, V, scale, padding_idx), axis=(1, 2)))

    def dp_embedding_clip_accumulate(self, ids, dY, norms, C, G_sum, scale=1.0, padding_idx=None, workspace=None,
                                     stream=None):
        G = self._gradients(ids, dY, G_sum.shape[0], scale, padding_idx)
        G_sum += torch.from_numpy(np.tensordot(oracle.clip_factors(norms.numpy(), C), G, 1)).to(G_sum.dtype)
        return G_sum

    def dp_embedding_step(self, ids, dY, V, C, sigma, seed, step, layer_id, scale=1.0, padding_idx=None, norms_out=None,
                          G_out=None, workspace=None, stream=None):
        assert sigma == 0
        w = oracle.embedding_step(ids.numpy(), dY.numpy(), V, C, 0.0, 0, 0, 0, scale, padding_idx)
        return self._fill(G_out, w["S"]), self._fill(norms_out, w["norms"])

    def dp_rmsnorm_backward(self, H, gain, dY, eps=1e-6, residual_grad=None, dX=None, per_sample=None, norms=None,
                            workspace=None, stream=None):
        dh, per = oracle.rmsnorm_gradients(H.numpy(), gain.numpy(), dY.numpy(), eps)
        if residual_grad is not None:
            dh = dh + residual_grad.numpy()
        return self._fill(dX, dh), self._fill(per_sample, per), self._fill(norms, np.linalg.norm(per, axis=1))

    def dp_rmsnorm_clip_accumulate(self, per_sample, norms, C, G_sum, stream=None):
        G_sum += torch.from_numpy(oracle.clip_factors(norms.numpy(), C) @ per_sample.numpy()).to(G_sum.dtype)
        return G_sum

    def dp_rmsnorm_step(self, H, gain, dY, C, sigma, seed, step, layer_id, eps=1e-6, residual_grad=None, dX=None,
                        norms_out=None, G_out=None, workspace=None, stream=None):
        assert sigma == 0
        dX, per, n = self.dp_rmsnorm_backward(H, gain, dY, eps, residual_grad, dX, None, norms_out)
        return dX, self._fill(G_out, oracle.clip_factors(n.numpy(), C) @ per.numpy()), n

    def dp_block_step(self, layers, mode, C, sigma, seed, step, method, stream=None):
        assert sigma == 0 and mode == "flat"
        w = oracle.block_step([{**l, "X": l["X"].numpy(), "dY": l["dY"].numpy(), "P": self._np(l.get("P"))}
                               for l in layers], C, 0.0, seed, step, mode="flat")
        return ([self._fill(l.get("G_out"), o["S"]) for l, o in zip(layers, w["layers"])],
                [self._fill(l.get("norms_out"), o["norms"]) for l, o in zip(layers, w["layers"])], None)

    def dp_add_noise(self, G, std, seed, step, layer_id, stream=None):
        flat = G.reshape(G.shape[0], -1)          # a gain is a matrix of one column, as in the binding
        G += torch.from_numpy(oracle.noise(*flat.shape, std, seed, step, layer_id).reshape(G.shape)).to(G.dtype)
        return G


def _ops():
    ops = sharded.LibraryOps()
    ops._lib = OracleLibrary()
    return ops


def _batch(seed=0):
    rng = np.random.default_rng(seed)
    t = lambda *shape: torch.from_numpy(rng.standard_normal(shape))  # noqa: E731
    scale = torch.from_numpy(np.exp(rng.normal(0.0, 1.0, size=(B, 1, 1))))    # some samples clip, some do not
    return [{"ids": torch.from_numpy(rng.integers(-1, V, size=(B, T))), "dY": t(B, T, D) * scale, "V": V, "scale": 1.5,
             "padding_idx": 2, "layer_id": 0, "C": 2.0},
            {"H": t(B, T, D), "gain": t(D), "dY": t(B, T, D) * scale, "eps": EPS, "residual_grad": t(B, T, D),
             "layer_id": 1, "C": 3.0},
            {"X": t(B, T, DI) * scale, "dY": t(B, T, DO), "P": t(DO, R), "layer_id": 2, "C": 2.5},
            {"X": t(B, T, DI), "dY": t(B, T, DO), "layer_id": 3, "C": 4.0}]


def _share(layers, lo, hi):
    whole = ("gain", "P", "V", "scale", "padding_idx", "eps", "layer_id", "C")
    return [{k: v if k in whole else v[lo:hi].contiguous() for k, v in layer.items()} for layer in layers]


def _gradients(layers):
    """Every layer's per-sample gradients, from the oracle."""
    e, n, p, w = layers
    return [np.stack([oracle.embedding_gradient(e["ids"][i].numpy(), e["dY"][i].numpy(), V, 1.5, 2) for i in range(B)]),
            oracle.rmsnorm_gradients(n["H"].numpy(), n["gain"].numpy(), n["dY"].numpy(), EPS)[1],
            np.einsum("bti,bto,or->bir", p["X"].numpy(), p["dY"].numpy(), p["P"].numpy()),
            np.einsum("bti,bto->bio", w["X"].numpy(), w["dY"].numpy())]


def _expected(layers, mode, C, sigma):
    grads = _gradients(layers)
    norms = np.stack([np.sqrt((g.reshape(B, -1) ** 2).sum(1)) for g in grads])
    flat = np.sqrt((norms ** 2).sum(0))
    out = []
    for layer, g, n in zip(layers, grads, norms):
        bound = layer["C"] if mode == "per_layer" else C
        S = np.tensordot(oracle.clip_factors(n if mode == "per_layer" else flat, bound), g, 1)
        out.append(S + oracle.noise(S.shape[0], S.size // S.shape[0], sigma * bound, 11, 4, layer["layer_id"]).reshape(S.shape))
    return out, norms


# A flat sum over mixed layers is held in the fp32 that the library adds to; else the oracle's fp64.
# Five samples of at most 2.5 each, and noise of a few times 2: factors, sum and noise's addition are
# three roundings of values below 20, 3.6e-6 in all.
def _check(sums, norms, want, lo=0, hi=B, flat=False):
    for got, w in zip(sums, want[0]):
        assert got.shape == w.shape
        np.testing.assert_allclose(got, w, rtol=0 if flat else 1e-12, atol=4e-6 if flat else 1e-12)
    for got, w in zip(norms, want[1]):
        np.testing.assert_allclose(got, w[lo:hi], rtol=1e-12)


@pytest.fixture
def alone(monkeypatch):
    """One rank, whose all-reduce leaves every sum as it is."""
    class Done:
        def wait(self):
            pass

    monkeypatch.setattr(dist, "all_reduce", lambda G, group=None, async_op=False: Done())


@pytest.mark.parametrize("preset", [False, True])
@pytest.mark.parametrize("mode", ["per_layer", "flat"])
def test_each_kind_of_layer(alone, mode, preset):
    layers = _batch()
    want = _expected(layers, mode, 2.5, 0.8)
    if preset:
        for layer, shape in zip(layers, ((V, D), (D,), (DI, R), (DI, DO))):
            layer["G_out"] = torch.full(shape, 9.0, dtype=torch.float32 if mode == "flat" else torch.float64)
    given = [layer.get("G_out") for layer in layers]
    sums, norms = sharded.sharded_step(layers, 0.8, 11, 4, mode=mode, C=2.5, ops=_ops())
    _check(sums, norms, want, flat=mode == "flat")
    assert all(g is None or s is g for s, g in zip(sums, given))
    np.testing.assert_allclose(layers[1]["dX"], oracle.rmsnorm_step(
        layers[1]["H"].numpy(), layers[1]["gain"].numpy(), layers[1]["dY"].numpy(), 1.0, 0.0, 0, 0, 0, EPS,
        layers[1]["residual_grad"].numpy())["dX"], rtol=1e-12)


@pytest.mark.parametrize("mode", ["per_layer", "flat"])
def test_a_projected_linear_is_the_same_beside_other_kinds(alone, mode):
    """Its norms with and without a table and a gain in the block."""
    layers = _batch(1)
    _, mixed = sharded.sharded_step([dict(l) for l in layers], 0.0, 11, 4, mode=mode, C=1e9, ops=_ops())
    block, linears = sharded.sharded_step([dict(l) for l in layers[2:]], 0.0, 11, 4, mode=mode, C=1e9, ops=_ops())
    for a, b in zip(mixed[2:], linears):
        np.testing.assert_allclose(a, b, rtol=1e-12)
    assert [tuple(g.shape) for g in block] == [(DI, R), (DI, DO)]


@pytest.mark.parametrize("mode", ["per_layer", "flat"])
def test_workspaces_are_kept_and_their_status_read(alone, mode, monkeypatch):
    """A table's and a norm's status words outlive the step: the same workspace in every call of it, made
    again only where a larger batch needs more; a given one is used."""
    used = []

    class Library(OracleLibrary):
        pass

    for name in ("dp_embedding_step", "dp_embedding_per_sample_norms", "dp_embedding_clip_accumulate", "dp_rmsnorm_step",
                 "dp_rmsnorm_backward"):
        def call(self, *a, workspace=None, _real=getattr(OracleLibrary, name), **k):
            used.append(workspace)
            return _real(self, *a, **k)

        setattr(Library, name, call)
    ops = _ops()
    ops._lib = Library()
    layers = _batch()
    for small in (True, False, False):
        used.clear()
        part = _share([{k: v for k, v in l.items() if k not in ("G_out", "norms_out", "dX", "per_sample", "workspace")}
                       for l in layers], 0, 2 if small else B)
        for mine, layer in zip(part, layers):
            if "workspace" in layer:
                mine["workspace"] = layer["workspace"]
        sharded.sharded_step(part, 0.0, 0, 0, mode=mode, C=2.5, ops=ops)
        assert [("workspace" in l) for l in part] == [True, True, False, False]
        assert all(w is part[0]["workspace"] or w is part[1]["workspace"] for w in used if w is not None)
        assert part[0]["workspace"].numel() == 1000 * (2 if small else B) and part[1]["workspace"].numel() == 500 * (2 if small else B)
        if not small and layers[0].get("workspace") is not None and layers[0]["workspace"].numel() == 1000 * B:
            assert part[0]["workspace"] is layers[0]["workspace"] and part[1]["workspace"] is layers[1]["workspace"]
        for mine, layer in zip(part, layers):
            if "workspace" in mine:
                layer["workspace"] = mine["workspace"]
    monkeypatch.setattr(_lib, "dp_workspace_status", lambda ws, stream=None: ws.numel())
    assert sharded.layer_status(layers) == [1000 * B, 500 * B, None, None]


class _Untouched:
    """A library that must not be reached."""

    def __getattr__(self, name):
        if name in ("workspace_size", "_dtype_code"):
            return getattr(OracleLibrary, name)
        raise AssertionError(f"{name} was called")


@pytest.mark.parametrize("k,shape", [(0, (V - 1, D)), (0, (V + 1, D)), (1, (D, 1)), (2, (DI, DO)), (3, (DI, R)), (3, (DI,))])
def test_a_sum_of_another_shape_is_refused_before_any_call(alone, k, shape):
    layers = _batch()
    layers[k]["G_out"] = torch.zeros(shape)
    ops = sharded.LibraryOps()
    ops._lib = _Untouched()
    with pytest.raises(ValueError, match="G_out"):
        sharded.sharded_step(layers, 0.0, 0, 0, mode="flat", C=1.0, ops=ops)


def _rank(rank, world, port, mode, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE=str(world))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        lo, hi = sharded.shard_rows(B, rank, world)
        sums, norms = sharded.sharded_step(_share(_batch(), lo, hi), 0.8, 11, 4, mode=mode, C=2.5, ops=_ops())
        out[rank] = ([s.numpy() for s in sums], [n.numpy() for n in norms], (lo, hi))
        dist.barrier()
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("mode", ["per_layer", "flat"])
def test_two_ranks_match_one_device(mode):
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    out = mp.get_context("spawn").Manager().dict()
    mp.start_processes(_rank, args=(2, port, mode, out), nprocs=2, join=True, start_method="spawn")
    want = _expected(_batch(), mode, 2.5, 0.8)
    for rank in range(2):
        sums, norms, (lo, hi) = out[rank]
        _check(sums, norms, want, lo, hi, flat=mode == "flat")
    for a, b in zip(out[0][0], out[1][0]):
        assert np.array_equal(a, b)
