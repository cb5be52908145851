"""The sharded step over a projected and a plain linear, a table and a gain on one GPU (a one-rank
NCCL group) against the oracle: the bounds of the linears' own tests (norms 1e-3 and sums 5e-3 in
bf16), which the table's and the gain's fp32 sums of bf16 values are far below."""
import datetime
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist

import oracle
from sample_gradient_clipping_b200 import _lib, sharded
from tests.gpu_helpers import TOL, host, rel_fro, rel_max

pytestmark = pytest.mark.gpu
B, T, V, D, DI, DO, R, EPS = 4, 96, 40, 64, 128, 96, 16, 1e-5


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


def _layers(seed=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda *shape: (torch.randn(*shape, generator=g) / 8).to(torch.bfloat16)  # noqa: E731
    ids = torch.randint(-1, V, (B, T), generator=g)
    P = oracle.round_to("bf16", oracle.projection(DO, R, 7, 2))
    return [{"ids": ids, "dY": t(B, T, D), "V": V, "scale": 2.0, "padding_idx": 3, "layer_id": 0},
            {"H": t(B, T, D) * 8, "gain": 1 + 0.2 * torch.randn(D, generator=g), "dY": t(B, T, D), "eps": EPS, "layer_id": 1},
            {"X": t(B, T, DI), "dY": t(B, T, DO), "P": torch.from_numpy(P).to(torch.bfloat16), "layer_id": 2},
            {"X": t(B, T, DI), "dY": t(B, T, DO), "layer_id": 3}]


def _cuda(layers):
    return [{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in layer.items()} for layer in layers]


def _gradients(layers):
    e, n, p, w = [{k: host(v) if isinstance(v, torch.Tensor) else v for k, v in layer.items()} for layer in layers]
    return [np.stack([oracle.embedding_gradient(e["ids"][i].astype(np.int64), e["dY"][i], V, 2.0, 3) for i in range(B)]),
            oracle.rmsnorm_gradients(n["H"], n["gain"], n["dY"], float(np.float32(EPS)))[1],
            np.einsum("bti,bto,or->bir", p["X"], p["dY"], p["P"]), np.einsum("bti,bto->bio", w["X"], w["dY"])]


@pytest.mark.parametrize("preset", [False, True])
@pytest.mark.parametrize("mode", ["per_layer", "flat"])
def test_projected_linear_in_a_mixed_step(mode, preset):
    layers = _layers()
    grads = _gradients(layers)
    norms = np.stack([np.sqrt((g.reshape(B, -1) ** 2).sum(1)) for g in grads])
    flat = np.sqrt((norms ** 2).sum(0))
    bounds = [float(np.float32(np.median(n))) for n in norms]
    C = float(np.float32(np.median(flat)))
    mine = _cuda(layers)
    behind = []
    for layer, c, g in zip(mine, bounds, grads):
        layer["C"] = c
        if preset:                                     # with values behind each sum, left as they were
            buf = torch.full((g[0].size + 4096,), 7.0, device="cuda")
            layer["G_out"] = buf[:g[0].size].view(g.shape[1:])
            behind.append(buf[g[0].size:])
    sums, got_n = sharded.sharded_step(mine, 0.0, 5, 6, mode=mode, C=C)
    torch.cuda.synchronize()
    for k, g in enumerate(grads):
        c = oracle.clip_factors(norms[k] if mode == "per_layer" else flat, bounds[k] if mode == "per_layer" else C)
        assert sums[k].shape == g.shape[1:]
        assert rel_max(host(got_n[k]), norms[k]) <= TOL["bf16"]["norm"], k
        assert rel_fro(host(sums[k]), np.tensordot(c, g, 1)) <= TOL["bf16"]["sum"], k
    assert all(bool((b == 7.0).all()) for b in behind)


def test_projected_linear_beside_others_and_alone():
    """Its norms and its flat sum agree with the block of linears' (under a bound that clips nothing)."""
    layers = _cuda(_layers(1))
    mixed, n = sharded.sharded_step([dict(l) for l in layers], 0.0, 5, 6, mode="flat", C=1e6)
    outs, _, _ = _lib.dp_block_step([dict(l, norms_out=torch.empty(B, device="cuda")) for l in layers[2:]], mode="flat",
                                    C=1e6)
    for a, b in zip(mixed[2:], outs):
        assert a.shape == b.shape and rel_fro(host(a), host(b)) <= 2 * TOL["bf16"]["sum"]


@pytest.mark.parametrize("mode", ["per_layer", "flat"])
def test_an_id_past_the_table_is_reported_after_the_step(mode):
    layers = _cuda(_layers(2))
    for layer in layers:
        layer["C"] = 1.0
    sharded.sharded_step(layers, 0.0, 5, 6, mode=mode, C=1.0)
    assert sharded.layer_status(layers) == [_lib.DP_OK, _lib.DP_OK, None, None]
    spaces = [layer.get("workspace") for layer in layers]
    good = layers[0]["ids"][2, 7].item()
    layers[0]["ids"][2, 7] = V
    sharded.sharded_step(layers, 0.0, 5, 6, mode=mode, C=1.0)
    assert sharded.layer_status(layers) == [_lib.DP_ERR_INVALID_ARG, _lib.DP_OK, None, None]
    assert all(a is b for a, b in zip(spaces, [layer.get("workspace") for layer in layers]))
    layers[0]["ids"][2, 7] = good
    sharded.sharded_step(layers, 0.0, 5, 6, mode=mode, C=1.0)
    assert sharded.layer_status(layers) == [_lib.DP_OK, _lib.DP_OK, None, None]
