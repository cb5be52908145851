"""Sample-sharded DP-SGD step over several GPUs, one process per GPU.

Each sample's gradient, norm and clip factor depend on that sample alone, so the batch splits
across ranks with no exchange for the norms.  A step is then:

1. every rank forms the clipped sum of its own samples for every linear, without noise;
2. one fp32 all-reduce (sum) per linear;
3. every rank adds the same Gaussian noise, drawn from the (seed, step, layer) Philox counter,
   to the reduced sum.  The counter is deterministic, so no message carries the noise, and it
   is added exactly once to the global sum, as in the one-GPU step.

The all-reduce of linear l is issued as soon as its sum is enqueued, so it overlaps the next
linear's kernels.  With flat (whole-block) clipping the clip factor of a sample needs only
that sample's norms over the block's linears, which live on the same rank.

A layer is a linear (X, dY), an embedding table (ids, dY, V) or the gain of an RMS norm (H, gain,
dY), each with its own entry points of the library.

``ops`` supplies the per-rank compute.  The default is the CUDA library; there is no CPU
path in the product.  Tests substitute their own ops to check this orchestration on CPU
ranks with the gloo backend.
"""
from __future__ import annotations

import math


class LibraryOps:
    """The per-rank compute of a sharded step: the CUDA library through its C ABI."""

    def __init__(self, method="auto"):
        from . import _lib

        self._lib = _lib
        self.method = method
        self._ws = None   # one workspace, grown to the largest linear seen

    def _workspace(self, X, dY, P=None):
        import torch

        B, T, d_in, d_out = (int(v) for v in (X.shape[0], X.shape[1], X.shape[2], dY.shape[2]))
        r = int(P.shape[1]) if P is not None else 0
        need = self._lib.workspace_size(B, T, d_in, d_out, r, self._lib._dtype_code(X), self.method)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=X.device)
        return self._ws

    def local_sum(self, layer, C, seed, step, stream=None):
        """Clipped sum of this rank's samples for one layer (sigma = 0, so no noise)."""
        if "ids" in layer:
            G, n = self._lib.dp_embedding_step(layer["ids"], layer["dY"], layer["V"], C, 0.0, seed, step,
                                               layer["layer_id"], norms_out=layer.get("norms_out"),
                                               G_out=layer.get("G_out"), stream=stream, **self._embedding(layer, stream))
            layer["G_out"], layer["norms_out"] = G, n
            return G
        if "gain" in layer:
            layer["dX"], G, n = self._lib.dp_rmsnorm_step(layer["H"], layer["gain"], layer["dY"], C, 0.0, seed, step,
                                                          layer["layer_id"], dX=layer.get("dX"),
                                                          norms_out=layer.get("norms_out"), G_out=layer.get("G_out"),
                                                          stream=stream, **self._norm(layer, stream))
            layer["G_out"], layer["norms_out"] = G, n
            return G
        P = layer.get("P")
        G, n = self._lib.dp_linear_step(layer["X"], layer["dY"], C, 0.0, seed, step, layer["layer_id"], P=P,
                                        method=self.method, norms_out=layer.get("norms_out"),
                                        G_out=layer.get("G_out"), workspace=self._workspace(layer["X"], layer["dY"], P),
                                        stream=stream)
        layer["G_out"], layer["norms_out"] = G, n
        return G

    def local_block_sums(self, layers, C, seed, step, stream=None):
        """Flat clipping over the block on this rank's samples, without noise."""
        if any("ids" in layer or "gain" in layer for layer in layers):
            return self._mixed_sums(layers, C, stream)
        outs, norms, flat = self._lib.dp_block_step(layers, mode="flat", C=C, sigma=0.0, seed=seed, step=step,
                                                    method=self.method, stream=stream)
        for layer, G, n in zip(layers, outs, norms):
            layer["G_out"], layer["norms_out"] = G, n
        return outs, flat

    @staticmethod
    def _kept_workspace(layer, need, stream):
        """The layer's workspace, made where it has none of `need` bytes and kept in its dict, as its
        sums are: its status word can then be read after the step (layer_status)."""
        import contextlib

        import torch

        ws, device = layer.get("workspace"), layer["dY"].device
        if need and (ws is None or ws.numel() * ws.element_size() < need or ws.device != device):
            with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
                ws = layer["workspace"] = torch.empty(need, dtype=torch.uint8, device=device)
        return ws

    def _embedding(self, layer, stream=None):
        B, T, d = (int(v) for v in layer["dY"].shape)
        need = self._lib.embedding_workspace_size(B, T, int(layer["V"]), d, self._lib._dtype_code(layer["dY"]))
        return {"scale": layer.get("scale", 1.0), "padding_idx": layer.get("padding_idx"),
                "workspace": self._kept_workspace(layer, need, stream)}

    def _norm(self, layer, stream=None):
        B, T, d = (int(v) for v in layer["dY"].shape)
        need = self._lib.rmsnorm_workspace_size(B, T, d, self._lib._dtype_code(layer["dY"]))
        return {"eps": layer.get("eps", 1e-6), "residual_grad": layer.get("residual_grad"),
                "workspace": self._kept_workspace(layer, need, stream)}

    @staticmethod
    def _sum_shape(layer):
        if "ids" in layer:
            return int(layer["V"]), int(layer["dY"].shape[2])
        if "gain" in layer:
            return tuple(layer["gain"].shape)
        P = layer.get("P")
        return int(layer["X"].shape[2]), int((layer["dY"] if P is None else P).shape[-1])

    def _mixed_sums(self, layers, C, stream):
        """Flat clipping over linears, tables and gains: every layer's norms first, then each
        layer's sum with the factors of the combined norms."""
        import contextlib

        import torch

        for layer in layers:
            G, shape = layer.get("G_out"), self._sum_shape(layer)
            if G is not None and (tuple(G.shape) != shape or G.dtype != torch.float32):
                raise ValueError(f"G_out of layer {layer['layer_id']} must be {torch.float32} of shape {list(shape)}, "
                                 f"got {G.dtype} {list(G.shape)}")
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            for layer in layers:
                if "ids" in layer:
                    n = self._lib.dp_embedding_per_sample_norms(layer["ids"], layer["dY"], layer["V"],
                                                                norms=layer.get("norms_out"), **self._embedding(layer))
                elif "gain" in layer:
                    layer["dX"], layer["per_sample"], n = self._lib.dp_rmsnorm_backward(
                        layer["H"], layer["gain"], layer["dY"], dX=layer.get("dX"), norms=layer.get("norms_out"),
                        **self._norm(layer))
                else:
                    P = layer.get("P")
                    n = self._lib.dp_per_sample_norms(layer["X"], layer["dY"], P=P, method=self.method,
                                                      norms=layer.get("norms_out"),
                                                      workspace=self._workspace(layer["X"], layer["dY"], P))
                layer["norms_out"] = n
            flat = torch.stack([layer["norms_out"] for layer in layers]).double().square().sum(0).sqrt().float()
            for layer in layers:
                G = layer.get("G_out")
                if G is None:
                    G = torch.empty(self._sum_shape(layer), dtype=torch.float32, device=layer["dY"].device)
                G.zero_()
                if "ids" in layer:
                    self._lib.dp_embedding_clip_accumulate(layer["ids"], layer["dY"], flat, C, G, **self._embedding(layer))
                elif "gain" in layer:
                    self._lib.dp_rmsnorm_clip_accumulate(layer["per_sample"], flat, C, G)
                else:
                    P = layer.get("P")
                    self._lib.dp_clip_accumulate(layer["X"], layer["dY"], flat, C, G, P=P,
                                                 workspace=self._workspace(layer["X"], layer["dY"], P))
                layer["G_out"] = G
        return [layer["G_out"] for layer in layers], flat

    def add_noise(self, G, std, seed, step, layer_id, stream=None):
        self._lib.dp_add_noise(G, std, seed, step, layer_id, stream=stream)


def sharded_step(layers, sigma, seed, step, mode="per_layer", C=None, group=None, ops=None, stream=None):
    """One privatised step of a block whose batch is split across the ranks of ``group``.

    ``layers``: this rank's shard, dicts with X [B_r, T, d_in], dY [B_r, T, d_out], layer_id, C
    (per-layer bound) and optional G_out / norms_out / P (a projection [d_out, r], the same on every
    rank: the linear's sum is then that of the projected gradients, [d_in, r]).  Instead of X: ids [B_r, T] and V (and scale,
    padding_idx) for an embedding table; H [B_r, T, d] and gain [d] (and eps, residual_grad) for an
    RMS norm, whose dX is then put into the dict.  The workspace of a table or a norm is kept in its
    dict too (or given there): layer_status reads it.  ``mode``: "per_layer" (each linear its
    own C_l, noise sigma * C_l) or "flat" (bound ``C`` for the whole block, noise sigma * C).
    Every rank returns the same noisy global sums, one per linear, and its own samples' norms.
    """
    import contextlib

    import torch
    import torch.distributed as dist

    if ops is None:
        ops = LibraryOps()
    if mode not in ("per_layer", "flat"):
        raise ValueError(f"unknown clipping mode {mode!r}")
    if mode == "flat" and not (C is not None and C > 0 and math.isfinite(C)):
        raise ValueError("flat clipping needs a finite bound C > 0")
    # NCCL orders a collective after the work already on the *current* stream, so the
    # library calls run on the current stream (``stream``, when given, becomes it).
    ctx = torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()
    with ctx:
        pending = []
        if mode == "per_layer":
            for layer in layers:
                G = ops.local_sum(layer, layer["C"], seed, step)
                pending.append((layer, G, dist.all_reduce(G, group=group, async_op=True), sigma * layer["C"]))
        else:
            outs, _ = ops.local_block_sums(layers, C, seed, step)
            for layer, G in zip(layers, outs):
                pending.append((layer, G, dist.all_reduce(G, group=group, async_op=True), sigma * C))
        results = []
        for layer, G, work, std in pending:
            work.wait()          # NCCL: the current stream waits; gloo: the host waits
            if std != 0.0:
                ops.add_noise(G, std, seed, step, layer["layer_id"])
            results.append(G)
    return results, [layer.get("norms_out") for layer in layers]


def layer_status(layers, stream=None):
    """What the kernels of a step recorded, layer by layer: the dp_status of each layer's workspace, None
    for a layer that keeps none (linears).  DP_ERR_INVALID_ARG: a token id past the table's end, whose
    tokens are missing from this rank's sum; DP_ERR_TIMEOUT: an in-kernel wait ran out, and the sum is
    invalid.  Synchronises the stream (``stream``, or the current one)."""
    from . import _lib

    return [_lib.dp_workspace_status(layer["workspace"], stream) if layer.get("workspace") is not None else None
            for layer in layers]


def shard_rows(batch, rank, world):
    """The contiguous slice of a batch dimension of size ``batch`` that ``rank`` owns."""
    per, extra = divmod(batch, world)
    start = rank * per + min(rank, extra)
    return start, start + per + (1 if rank < extra else 0)
