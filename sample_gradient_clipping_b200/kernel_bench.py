"""Times one entry point of the library on its own, for profiling a single kernel.

    python -m sample_gradient_clipping_b200.kernel_bench --op noise --rows 8192 --cols 8192
    python -m sample_gradient_clipping_b200.kernel_bench --op norms --method explicit \\
        --B 8 --T 2048 --d-in 4096 --d-out 4096

Ops: ``noise`` (dp_add_noise on an fp32 [rows, cols] buffer), ``projection``
(dp_projection_matrix, bf16 [rows, cols]), ``philox`` (dp_philox_blocks, rows*cols/4 blocks),
``norms`` (dp_per_sample_norms) and ``clip_accumulate`` (dp_clip_accumulate) on seeded bf16
inputs [B, T, d], ``lookup`` and ``embedding`` (dp_embedding_lookup, dp_embedding_step with a table
of ``rows`` rows of width ``d-in``, ids as frequent as 1 / rank), ``rmsnorm_step`` (dp_rmsnorm_step of
[B, T, d-in] with a residual gradient) and ``muon`` (dp_muon_step of fp32 [rows, cols]).  Prints one JSON line: microseconds per call (CUDA events around ``--iters``
calls after ``--warmup`` calls) and the algorithmic bytes or flops per second.
"""
from __future__ import annotations

import argparse
import json


def main(argv=None):
    import torch

    from . import _lib, inputs

    ap = argparse.ArgumentParser()
    ap.add_argument("--op", required=True, choices=["noise", "projection", "philox", "norms", "clip_accumulate",
                                                   "lookup", "embedding", "rmsnorm_step", "muon"])
    ap.add_argument("--rows", type=int, default=8192)
    ap.add_argument("--cols", type=int, default=8192)
    ap.add_argument("--B", type=int, default=8)
    ap.add_argument("--T", type=int, default=2048)
    ap.add_argument("--d-in", type=int, default=4096)
    ap.add_argument("--d-out", type=int, default=4096)
    ap.add_argument("--method", default="auto", choices=list(_lib.METHODS))
    ap.add_argument("--sigma", type=float, default=1.0)
    ap.add_argument("--iters", type=int, default=20)
    ap.add_argument("--warmup", type=int, default=3)
    a = ap.parse_args(argv)
    _lib.lib()
    dev = torch.device("cuda")
    rows, cols = a.rows, a.cols
    if a.op == "noise":
        G = torch.zeros(rows, cols, dtype=torch.float32, device=dev)
        call = lambda k: _lib.dp_add_noise(G, 0.5, 7, k, 3)
        work, unit = 8.0 * rows * cols, "GB/s"      # read and write fp32
    elif a.op == "projection":
        P = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
        call = lambda k: _lib.dp_projection_matrix(P, 7 + k, 3)
        work, unit = 2.0 * rows * cols, "GB/s"
    elif a.op == "philox":
        nblk = rows * cols // 4
        out = torch.empty(nblk, 4, dtype=torch.int32, device=dev)
        call = lambda k: _lib.dp_philox_blocks(nblk, 7, k, 3, 0, out=out)
        work, unit = 16.0 * nblk, "GB/s"
    elif a.op in ("lookup", "embedding"):
        gen = torch.Generator(device=dev).manual_seed(1)
        u = torch.rand(a.B, a.T, generator=gen, device=dev, dtype=torch.float64)
        ids = (rows ** u).long().clamp(1, rows) - 1
        tokens = a.B * a.T * a.d_in * 2.0
        if a.op == "lookup":
            W = torch.randn(rows, a.d_in, generator=gen, device=dev).to(torch.bfloat16)
            Y = torch.empty(a.B, a.T, a.d_in, dtype=torch.bfloat16, device=dev)
            call = lambda k: _lib.dp_embedding_lookup(W, ids, out=Y)
            work = 2 * tokens
        else:
            dY = torch.randn(a.B, a.T, a.d_in, generator=gen, device=dev).to(torch.bfloat16)
            G = torch.empty(rows, a.d_in, dtype=torch.float32, device=dev)
            ws = torch.empty(_lib.embedding_workspace_size(a.B, a.T, rows, a.d_in), dtype=torch.uint8, device=dev)
            call = lambda k: _lib.dp_embedding_step(ids, dY, rows, 1.0, a.sigma, 7, k, 3, G_out=G, workspace=ws)
            work = tokens + 4.0 * rows * a.d_in
        unit = "GB/s"
    elif a.op == "rmsnorm_step":
        H, dY, res = (torch.randn(a.B, a.T, a.d_in, device=dev).to(torch.bfloat16) for _ in range(3))
        gain = torch.ones(a.d_in, device=dev)
        ws = torch.empty(_lib.rmsnorm_workspace_size(a.B, a.T, a.d_in), dtype=torch.uint8, device=dev)
        dX = torch.empty_like(H)
        call = lambda k: _lib.dp_rmsnorm_step(H, gain, dY, 1.0, a.sigma, 7, k, 3, residual_grad=res, dX=dX, workspace=ws)
        work, unit = 8.0 * a.B * a.T * a.d_in, "GB/s"
    elif a.op == "muon":
        W, R, M = (torch.randn(rows, cols, device=dev) for _ in range(3))
        ws = torch.empty(_lib.muon_workspace_size(rows, cols), dtype=torch.uint8, device=dev)
        call = lambda k: _lib.dp_muon_step(W, R, M, 1e-3, workspace=ws)
        m, n = float(min(rows, cols)), float(max(rows, cols))
        work, unit = 5 * (3 * m * m * n + m ** 3), "TFLOP/s"    # X X^T and A^2 are symmetric
    else:
        w = inputs.custom("kernel_bench", B=a.B, T=a.T, d_in=a.d_in, d_out=a.d_out, C=1.0, sigma=0.0, seed=1)
        d = inputs.generate(w)
        X, dY = d["X"]["in"].to(dev), d["dY"]["linear"].to(dev)
        ws = torch.empty(_lib.workspace_size(a.B, a.T, a.d_in, a.d_out, 0, _lib.DP_BF16, a.method),
                         dtype=torch.uint8, device=dev)
        n = torch.empty(a.B, dtype=torch.float32, device=dev)
        flops = 2.0 * a.B * a.T * a.d_in * a.d_out
        if a.op == "norms":
            call = lambda k: _lib.dp_per_sample_norms(X, dY, method=a.method, norms=n, workspace=ws)
        else:
            _lib.dp_per_sample_norms(X, dY, method=a.method, norms=n, workspace=ws)
            G = torch.zeros(a.d_in, a.d_out, dtype=torch.float32, device=dev)
            call = lambda k: _lib.dp_clip_accumulate(X, dY, n, 1.0, G, workspace=ws)
        work, unit = flops, "TFLOP/s"
    for k in range(a.warmup):
        call(k)
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for k in range(a.iters):
        call(a.warmup + k)
    e1.record()
    torch.cuda.synchronize()
    us = e0.elapsed_time(e1) * 1e3 / a.iters
    rate = work / (us * 1e-6) / (1e9 if unit == "GB/s" else 1e12)
    print(json.dumps({"op": a.op, "us_per_call": us, "rate": rate, "unit": unit,
                      "shape": {"rows": rows, "cols": cols} if a.op in ("noise", "projection", "philox", "muon")
                      else {"B": a.B, "T": a.T, "rows": rows, "d": a.d_in}
                      if a.op in ("lookup", "embedding", "rmsnorm_step")
                      else {"B": a.B, "T": a.T, "d_in": a.d_in, "d_out": a.d_out, "method": a.method}}))


if __name__ == "__main__":
    main()
