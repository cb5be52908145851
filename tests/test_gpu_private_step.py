"""Lookup, RMS norm, their privatised gradients, the linears' and the Muon step run together, as a
training step runs them, against per-sample gradients by automatic differentiation in fp64.

The model is z = rmsnorm(scale E[ids] + r) W with the loss sum(z dz), everything in fp32.  Bounds: every
value passes at most four sums of up to 64 terms (the norm, W's product forward and back, the sum over
a sample's tokens, which is shorter), each off by at most 64 u of its terms' magnitudes with u = 2^-24,
so about 2.5e-5 in the worst case of no cancellation; 5e-5 covers the terms' mild cancellation here."""
from __future__ import annotations

import datetime
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist

import oracle
from sample_gradient_clipping_b200 import _lib, sharded
from tests.gpu_helpers import host, rel_fro, rel_max

pytestmark = pytest.mark.gpu
TOL = 5e-5
B, T, V, D, N, SCALE, EPS = 6, 40, 50, 64, 48, 2.0, 1e-5
SIGMA, SEED, STEP = 0.5, 11, 4


@pytest.fixture(scope="module", autouse=True)
def _nccl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1,
                            timeout=datetime.timedelta(seconds=60))
    yield
    dist.destroy_process_group()


def _model(seed=0):
    g = torch.Generator().manual_seed(seed)
    p = {"E": torch.randn(V, D, generator=g), "gain": 1 + 0.2 * torch.randn(D, generator=g),
         "W": torch.randn(D, N, generator=g) / 8}
    ids = torch.randint(0, V, (B, T), generator=g)
    ids[1, 25:] = 0                                        # a padded sample
    r = torch.randn(B, T, D, generator=g)
    dz = torch.randn(B, T, N, generator=g) / 60 * torch.exp(torch.randn(B, 1, 1, generator=g))
    dz[1, 25:] = 0
    return p, ids, r, dz


def _autograd(p, ids, r, dz):
    """Sample by sample, in fp64: the gradients of E, gain and W (the padding row 0 has none)."""
    out = []
    for i in range(B):
        q = {k: v.double().requires_grad_() for k, v in p.items()}
        h = float(np.float32(SCALE)) * q["E"][ids[i]] + r[i].double()
        y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + float(np.float32(EPS))) * q["gain"]
        ((y @ q["W"]) * dz[i].double()).sum().backward()
        q["E"].grad[0] = 0
        out.append({k: v.grad.numpy() for k, v in q.items()})
    return out


def _backward(p, ids, r, dz):
    """The library's forward and backward up to the layers' inputs and output gradients."""
    E, gain, W = (p[k].cuda() for k in ("E", "gain", "W"))
    ids, r, dz = ids.cuda(), r.cuda(), dz.cuda()
    x = _lib.dp_embedding_lookup(E, ids, scale=SCALE)
    y, h = _lib.dp_rmsnorm(x, gain, eps=EPS, residual=r)
    dy = (dz.reshape(-1, N).double() @ W.double().T).float().reshape(B, T, D)
    dx, _, _ = _lib.dp_rmsnorm_backward(h, gain, dy, eps=EPS)
    return [{"ids": ids, "dY": dx, "V": V, "scale": SCALE, "padding_idx": 0, "layer_id": 0},
            {"H": h, "gain": gain, "dY": dy, "eps": EPS, "layer_id": 1},
            {"X": y, "dY": dz, "layer_id": 2}]


@pytest.mark.parametrize("mode", ["per_layer", "flat"])
def test_private_step_of_a_whole_model(mode):
    p, ids, r, dz = _model()
    grads = _autograd(p, ids, r, dz)
    names = ("E", "gain", "W")
    norms = np.array([[np.linalg.norm(g[k]) for g in grads] for k in names])     # [layer, sample]
    flat = np.sqrt((norms ** 2).sum(0))
    bounds = [float(np.float32(np.median(norms[k]))) for k in range(3)]
    C = float(np.float32(np.median(flat)))
    layers = _backward(p, ids, r, dz)
    for layer, c in zip(layers, bounds):
        layer["C"] = c
    quiet, got_n = sharded.sharded_step([dict(l) for l in layers], 0.0, SEED, STEP, mode=mode, C=C)
    noisy, _ = sharded.sharded_step([dict(l) for l in layers], SIGMA, SEED, STEP, mode=mode, C=C)
    for k, name in enumerate(names):
        std = SIGMA * (bounds[k] if mode == "per_layer" else C)
        factors = oracle.clip_factors(norms[k] if mode == "per_layer" else flat, bounds[k] if mode == "per_layer" else C)
        want = sum(c * g[name] for c, g in zip(factors, grads))
        assert rel_max(host(got_n[k]), norms[k]) <= TOL, name
        assert rel_fro(host(quiet[k]), want) <= TOL, name
        flat_shape = host(noisy[k]).reshape(want.shape[0], -1)
        z = oracle.noise(flat_shape.shape[0], flat_shape.shape[1], std, SEED, STEP, layers[k]["layer_id"])
        err = np.abs(host(noisy[k]) - host(quiet[k]) - z.reshape(want.shape))
        assert np.all(err <= 2.0 ** -23 * (np.abs(host(noisy[k])) + np.abs(host(quiet[k]))) + 1e-9), name


def test_separate_calls_make_the_sharded_step():
    """Each layer's own step gives the sharded step's sums, and the Muon step takes the linear's."""
    p, ids, r, dz = _model(1)
    layers = _backward(p, ids, r, dz)
    for layer in layers:
        layer["C"] = 0.3
    out, n = sharded.sharded_step([dict(l) for l in layers], 0.0, SEED, STEP)
    e, g, w = layers
    G0, n0 = _lib.dp_embedding_step(e["ids"], e["dY"], V, 0.3, 0.0, SEED, STEP, 0, scale=SCALE, padding_idx=0)
    dX, G1, n1 = _lib.dp_rmsnorm_step(g["H"], g["gain"], g["dY"], 0.3, 0.0, SEED, STEP, 1, eps=EPS)
    G2, n2 = _lib.dp_linear_step(w["X"], w["dY"], 0.3, 0.0, SEED, STEP, 2)
    assert torch.equal(out[0], G0) and torch.equal(out[1], G1) and torch.equal(n[0], n0) and torch.equal(n[1], n1)
    assert torch.equal(dX, e["dY"])
    assert rel_fro(host(out[2]), host(G2)) <= 1e-6 and rel_max(host(n[2]), host(n2)) <= 1e-6
    W, M = p["W"].cuda(), torch.zeros(D, N, device="cuda")
    before = host(W)
    _lib.dp_muon_step(W, G2, M, 0.02, grad_scale=1.0 / B)
    want, _ = oracle.muon_step(before, host(G2), np.zeros((D, N)), float(np.float32(0.02)), float(np.float32(0.95)), True, 0.0,
                               float(np.float32(1.0 / B)), 1.0)
    assert np.linalg.norm(host(W) - want) <= 5e-3 * np.linalg.norm(want - before)


def test_one_graph_of_a_private_step():
    """Embedding, gain and linear steps captured together with the step number on the device."""
    p, ids, r, dz = _model(2)
    e, g, w = _backward(p, ids, r, dz)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(step):
        a = _lib.dp_embedding_step(e["ids"], e["dY"], V, 0.3, 0.5, SEED, step, 0, scale=SCALE, padding_idx=0)
        b = _lib.dp_rmsnorm_step(g["H"], g["gain"], g["dY"], 0.3, 0.5, SEED, step, 1, eps=EPS)
        c = _lib.dp_linear_step(w["X"], w["dY"], 0.3, 0.5, SEED, step, 2)
        return (*a, *b, *c)

    run(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(step)
    for k in range(3):
        step.fill_(k)
        e["dY"].mul_(1.5)
        g["dY"].mul_(0.75)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = run(k)
        for i, (a, b) in enumerate(zip(got, want)):
            # The fp32 linear adds its norms with fp64 atomics, so its last bits may differ.
            assert torch.equal(a, b) if i < 5 else rel_fro(host(a), host(b)) <= 1e-6, (k, i)


def test_checked_build_gives_the_same_bits():
    """The build with device-side index checks: a clean status and the normal build's results."""
    p, ids, r, dz = _model(3)
    e, g, _ = _backward(p, ids, r, dz)
    bf = {k: v.to(torch.bfloat16) for k, v in (("dY", g["dY"]), ("H", g["H"]))}

    def run():
        out, spaces = [], []

        def ws(n):
            spaces.append(torch.zeros(n, dtype=torch.uint8, device="cuda"))
            return spaces[-1]

        out += [_lib.dp_embedding_lookup(p["E"].cuda(), e["ids"], scale=SCALE, out_dtype=torch.bfloat16)]
        out += _lib.dp_embedding_step(e["ids"], e["dY"], V, 0.3, 0.5, SEED, STEP, 0, workspace=ws(
            _lib.embedding_workspace_size(B, T, V, D, _lib.DP_F32)))
        out += _lib.dp_rmsnorm(bf["H"], g["gain"], residual=bf["dY"])
        out += _lib.dp_rmsnorm_step(bf["H"], g["gain"], bf["dY"], 0.3, 0.5, SEED, STEP, 1, workspace=ws(
            _lib.rmsnorm_workspace_size(B, T, D)))
        for m, n in ((D, N), (200, 328), (328, 200)):
            G = torch.sin(torch.arange(m * n, device="cuda", dtype=torch.float32)).reshape(m, n)
            out += [_lib.dp_orthogonalize(G, workspace=ws(_lib.muon_workspace_size(m, n)))]
            out += _lib.dp_muon_step(G.clone(), G, G.clone(), 0.1, workspace=ws(_lib.muon_workspace_size(m, n)))
        assert all(_lib.dp_workspace_status(s) == _lib.DP_OK for s in spaces)
        return out

    want = run()
    with _lib.using(_lib.debug_lib()):
        got = run()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refused_launches_are_reported_and_the_next_call_is_whole():
    """Each launch of each call refused in turn, on the host: the call reports it and enqueues no
    more, and the same call then gives the bits of an undisturbed one."""
    p, ids, r, dz = _model(4)
    e, g, _ = _backward(p, ids, r, dz)
    G = torch.sin(torch.arange(200 * 328, device="cuda", dtype=torch.float32)).reshape(200, 328)
    calls = [lambda: _lib.dp_embedding_step(e["ids"], e["dY"], V, 0.3, 0.5, SEED, STEP, 0),
             lambda: (_lib.dp_embedding_lookup(p["E"].cuda(), e["ids"]),),
             lambda: _lib.dp_rmsnorm(g["H"], g["gain"]),
             lambda: _lib.dp_rmsnorm_step(g["H"], g["gain"], g["dY"], 0.3, 0.5, SEED, STEP, 1),
             lambda: (_lib.dp_orthogonalize(G),), lambda: (_lib.dp_orthogonalize(G[:64].contiguous()),)]
    for call in calls:
        n = _lib.kernel_launches()
        want = call()
        n = _lib.kernel_launches() - n
        for k in range(n):
            try:
                assert _lib.lib().dp_selftest_fail_launches(k, 1, 2) == _lib.DP_OK     # cudaErrorMemoryAllocation
                with pytest.raises(_lib.DPError) as err:
                    call()
                assert err.value.status == _lib.DP_ERR_CUDA and "memory" in str(err.value)
            finally:
                _lib.lib().dp_selftest_fail_launches(0, 0, 0)
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
