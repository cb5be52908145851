"""The RMS norm, its backward and the gain's privatised gradient against the fp64 oracle.

Bounds.  A row's sums of d products are off by at most (d/32 + 16) u of their terms' magnitudes
(a thread adds at most d/32 of them, then the warps are joined), u = 2^-24; the mean square has no
cancellation, so 1/rms is off by half of that and a few roundings.  dX adds two terms, each with a
handful of roundings, and is rounded to its type (bf16: half a step, at most 2^-8 of the value).
A column's sum over T rows is fp32 inside a block: at most T u of the terms' magnitudes."""
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
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()


def _draw(B, T, d, dt, seed, n=3):
    rng = np.random.default_rng(seed)
    out = []
    for k in range(n):
        a = rng.standard_normal((B, T, d)) * (1.0 if k == 0 else np.exp(rng.standard_normal((B, 1, 1))) / np.sqrt(T * d))
        t = torch.from_numpy(a.astype(np.float32)).to(DT[dt])
        out += [t.double().numpy(), t.cuda()]
    gain = (1.0 + 0.3 * rng.standard_normal(d)).astype(np.float32)
    return (*out, gain.astype(np.float64), torch.from_numpy(gain).cuda())


# Rows of one to four vectors a lane, a warp, a block of 128 to 512 threads; ragged ends.
WIDTHS = [("bf16", d) for d in (8, 256, 264, 1024, 1032, 2048, 2056, 4096, 4104, 8200, 16384)] + \
         [("f32", d) for d in (4, 128, 132, 512, 516, 1028, 2052, 8192)]


@pytest.mark.parametrize("dt,d", WIDTHS)
@pytest.mark.parametrize("rows", [1, 5])
def test_forward(dt, d, rows):
    x_h, x, r_h, r, gain_h, gain = _draw(1, rows, d, dt, d + rows, n=2)
    y, h = _lib.dp_rmsnorm(x, gain, eps=EPS)
    assert h is x
    rel = (d / 32 + 24) * U32 + HALF[dt]
    want = oracle.rmsnorm(x_h, gain_h, float(np.float32(EPS)))
    assert np.all(np.abs(host(y) - want) <= rel * np.abs(want))
    y, h = _lib.dp_rmsnorm(x, gain, eps=EPS, residual=r * 100)
    r_h = host(r * 100)
    # One fp32 addition, then the type's rounding.
    assert np.all(np.abs(host(h) - (x_h + r_h)) <= (U32 + HALF[dt]) * np.abs(x_h + r_h))
    want = oracle.rmsnorm(host(h), gain_h, float(np.float32(EPS)))
    assert np.all(np.abs(host(y) - want) <= rel * np.abs(want))


def test_forward_many_rows_and_extremes():
    x_h, x, gain_h, gain = _draw(40, 777, 64, "bf16", 3, n=1)
    y, _ = _lib.dp_rmsnorm(x, gain, eps=EPS)
    want = oracle.rmsnorm(x_h, gain_h, float(np.float32(EPS)))
    assert np.all(np.abs(host(y) - want) <= (64 / 32 + 24) * U32 * np.abs(want) + HALF["bf16"] * np.abs(want))
    z = torch.zeros(3, 64, device="cuda")
    g64 = gain.clone()
    assert float(_lib.dp_rmsnorm(z, g64, eps=EPS)[0].abs().max()) == 0.0          # rows of zeros
    z[1, 5] = float("nan")
    y, _ = _lib.dp_rmsnorm(z, g64, eps=EPS)
    assert torch.isnan(y[1]).all() and float(y[0].abs().max()) == 0.0 == float(y[2].abs().max())
    assert _lib.dp_rmsnorm(torch.empty(0, 64, device="cuda"), g64)[0].shape == (0, 64)


def _bounds(h, gain, dY, ref, C, dt, T, d, res):
    r = 1.0 / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + float(np.float32(EPS)))
    u = np.abs(dY * gain)
    sums = (d / 32 + 24) * U32
    mags = r * u + np.abs(h) * r ** 3 * np.mean(u * np.abs(h), axis=-1, keepdims=True)
    dX = 2 * sums * mags + (0 if res is None else U32 * np.abs(res)) + HALF[dt] * (1 + 2.0 ** -10) * np.abs(ref["dX"])
    mag = np.sum(np.abs(dY * h) * r, axis=1)
    per = ((T + 8) * U32 + sums) * mag
    norm = np.linalg.norm(per, axis=1) + 12 * U32 * ref["norms"]
    rel_c = np.where(ref["norms"] > C, norm / np.maximum(ref["norms"], 1e-300), 0.0)
    S = (ref["c"][:, None] * (per + (rel_c[:, None] + 4 * U32) * mag)).sum(0) + U32 * np.abs(ref["out"]) + 1e-11
    return dX, per, norm, S


@pytest.mark.parametrize("dt,d", WIDTHS)
@pytest.mark.parametrize("B,T,sigma", [(1, 1, 0.0), (3, 37, 0.7)])
def test_step(dt, d, B, T, sigma):
    if d > 4200 and T > 1:
        T = 9
    h_h, h, y_h, y, r_h, r, gain_h, gain = _draw(B, T, d, dt, d + T)
    C = 0.8
    for res_h, res in ((None, None), (r_h, r)):
        ref = oracle.rmsnorm_step(h_h, gain_h, y_h, float(np.float32(C)), float(np.float32(sigma)), 5, 6, 7,
                                  float(np.float32(EPS)), residual_grad=res_h)
        dX, G, n = _lib.dp_rmsnorm_step(h, gain, y, C, sigma, 5, 6, 7, eps=EPS, residual_grad=res)
        bX, bper, bn, bS = _bounds(h_h, gain_h, y_h, ref, C, dt, T, d, res_h)
        assert np.all(np.abs(host(dX) - ref["dX"]) <= bX + 1e-30)
        assert np.all(np.abs(host(n) - ref["norms"]) <= bn + 1e-30)
        assert np.all(np.abs(host(G) - ref["out"]) <= bS)
        # The unprivatised backward and the accumulation of given norms make the same step.
        dX2, per, n2 = _lib.dp_rmsnorm_backward(h, gain, y, eps=EPS, residual_grad=res)
        assert torch.equal(dX, dX2) and torch.equal(n, n2)
        assert np.all(np.abs(host(per) - ref["per_sample"]) <= bper + 1e-30)
        S = torch.ones(d, device="cuda")
        _lib.dp_rmsnorm_clip_accumulate(per, n, C, S)
        assert np.all(np.abs(host(S) - 1.0 - ref["S"]) <= bS + U32 * (1.0 + np.abs(ref["S"])))


@pytest.mark.parametrize("B,T,d,dt", [
    # parts of a sample: 7, 2 and 4 of many bytes, 32, 37, one a row, and more than a row each
    (300, 20, 256, "bf16"), (64, 2, 2056, "bf16"), (32, 4, 4096, "bf16"), (16, 32, 2048, "bf16"), (64, 40, 128, "bf16"),
    (2, 486, 396, "f32"), (1, 700, 132, "f32"), (1, 2500, 64, "f32"),
])
def test_parts_of_a_sample(B, T, d, dt):
    h_h, h, y_h, y, gain_h, gain = _draw(B, T, d, dt, B + T + d, n=2)
    C = 0.8
    ref = oracle.rmsnorm_step(h_h, gain_h, y_h, float(np.float32(C)), 0.0, 0, 0, 0, float(np.float32(EPS)))
    dX, G, n = _lib.dp_rmsnorm_step(h, gain, y, C, 0.0, 0, 0, 0, eps=EPS)
    bX, bper, bn, bS = _bounds(h_h, gain_h, y_h, ref, C, dt, T, d, None)
    assert np.all(np.abs(host(dX) - ref["dX"]) <= bX + 1e-30)
    assert np.all(np.abs(host(n) - ref["norms"]) <= bn + 1e-30)
    # (the samples' terms are added in fp64, so more of them add no rounding)
    assert np.all(np.abs(host(G) - ref["out"]) <= bS)
    _, per, n2 = _lib.dp_rmsnorm_backward(h, gain, y, eps=EPS)
    assert torch.equal(n, n2) and np.all(np.abs(host(per) - ref["per_sample"]) <= bper + 1e-30)


def test_many_samples():
    h_h, h, y_h, y, gain_h, gain = _draw(2500, 3, 40, "f32", 8, n=2)
    ref = oracle.rmsnorm_step(h_h, gain_h, y_h, 0.5, 0.0, 0, 0, 0, float(np.float32(EPS)))
    dX, G, n = _lib.dp_rmsnorm_step(h, gain, y, 0.5, 0.0, 0, 0, 0, eps=EPS)
    bX, bper, bn, bS = _bounds(h_h, gain_h, y_h, ref, 0.5, "f32", 3, 40, None)
    assert np.all(np.abs(host(dX) - ref["dX"]) <= bX) and np.all(np.abs(host(n) - ref["norms"]) <= bn)
    assert np.all(np.abs(host(G) - ref["out"]) <= bS)


def test_offsets_past_32_bits():
    d, B, T = 4096, 5, 106_000
    H = torch.zeros(B, T, d, dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros_like(H)
    H[4, -1, ::2] = 2.0
    H[4, -1, 1::2] = -2.0
    dY[4, -1] = 1.0
    gain = torch.full((d,), 3.0, device="cuda")
    dX, G, n = _lib.dp_rmsnorm_step(H, gain, dY, 1e6, 0.0, 0, 0, 0, eps=1e-5)
    # r = 1/2 up to eps, u.h sums to zero: dX = r g dy, and the gain's gradient is dy h r = +-1.
    assert torch.all((dX[4, -1] - 1.5).abs() <= 2 ** -8 * 1.5) and float(dX[:4].abs().max()) == 0.0
    assert torch.all((G.abs() - 1.0).abs() <= 1e-5) and float(G[0]) > 0 > float(G[1]) and float(n[:4].max()) == 0.0
    assert abs(float(n[4]) - 64.0) <= 1e-3
    del dX
    Y, _ = _lib.dp_rmsnorm(H, gain, eps=1e-5, Y=dY)
    assert torch.all((Y[4, -1].abs() - 3.0).abs() <= 2 ** -8 * 3.0) and float(Y[4, -2].abs().max()) == 0.0


def test_as_many_rows_as_are_taken():
    """2^31 - 1 rows of one sample: row numbers next to the end of 32 bits.  (32 GiB a tensor; dY is h.)"""
    d, T = 8, 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 80 * 2 ** 30:
        pytest.skip("needs 80 GiB of free device memory")
    h = torch.ones(1, T, d, dtype=torch.bfloat16, device="cuda")
    dX = torch.full_like(h, 5.0)
    gain = torch.arange(1, d + 1, dtype=torch.float32, device="cuda")
    _, per, n = _lib.dp_rmsnorm_backward(h, gain, h, eps=0.0, dX=dX)
    # r = 1: dX = gain - its mean, exact in bf16, and every row adds 1 to the gain's gradient, exact in
    # a part's fp32 sum (under 2^24 rows) and in the fp64 sum of the parts.
    want = (gain - gain.mean()).to(torch.bfloat16)
    for rows in (dX[0, :1000], dX[0, T // 2:T // 2 + 1000], dX[0, -1000:]):
        assert torch.all(rows == want)
    assert torch.all(dX[0].view(-1, 8)[::4096] == want)
    assert torch.all(per == float(np.float32(T)))
    assert abs(float(n) - T * np.sqrt(d)) <= 4 * U32 * T * np.sqrt(d)


def test_gradients_against_differences():
    """The backward of the forward that is called, by central differences in fp32."""
    h_h, h, y_h, y, gain_h, gain = _draw(1, 2, 16, "f32", 9, n=2)
    y = y * 100
    dX, per, _ = _lib.dp_rmsnorm_backward(h, gain, y, eps=EPS)
    f = lambda hh, g: float((_lib.dp_rmsnorm(hh, g, eps=EPS)[0].double() * y.double()).sum())  # noqa: E731
    e = 2.0 ** -7
    # Each output is off by at most 8 u of itself, and both ends of a difference are divided by 2 e;
    # the third derivative of a normalised value in one h is at most 15 (|h| about 1), over 6.
    out = _lib.dp_rmsnorm(h, gain, eps=EPS)[0]
    tol = 8 * U32 * float((out * y).abs().sum()) / e + 2.5 * e * e * float((y * gain).abs().sum())
    for t, j in ((0, 0), (1, 7), (0, 15)):
        up, dn = h.clone(), h.clone()
        up[0, t, j] += e
        dn[0, t, j] -= e
        assert abs((f(up, gain) - f(dn, gain)) / (2 * e) - float(dX[0, t, j])) <= tol
        gu, gd = gain.clone(), gain.clone()
        gu[j] += e
        gd[j] -= e
        assert abs((f(h, gu) - f(h, gd)) / (2 * e) - float(per[0, j])) <= tol


def test_bits_repeat_and_surroundings_stay():
    _, h, _, y, _, r, _, gain = _draw(6, 150, 1032, "bf16", 10)
    need = _lib.rmsnorm_workspace_size(6, 150, 1032)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    buf = torch.full((8, 150, 1032), 3.0, device="cuda", dtype=torch.bfloat16)
    first = None
    for _ in range(4):
        ws[:need] = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
        out = _lib.dp_rmsnorm_step(h, gain, y, 1.0, 0.5, 1, 2, 3, residual_grad=r, workspace=ws[:need], dX=buf[1:7])
        first = [o.clone() for o in out] if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(out, first))
        assert _lib.dp_workspace_status(ws) == _lib.DP_OK
    assert (ws[need:] == 0x5A).all() and (buf[0] == 3.0).all() and (buf[7] == 3.0).all()


def test_graph_replays_follow_inputs_and_step():
    _, h, _, y, _, gain = _draw(4, 60, 512, "bf16", 11, n=2)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.empty(_lib.rmsnorm_workspace_size(4, 60, 512), dtype=torch.uint8, device="cuda")
    dX, G, n = torch.empty_like(h), torch.empty(512, device="cuda"), torch.empty(4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.dp_rmsnorm_step(h, gain, y, 1.0, 0.8, 5, step, 1, workspace=ws, dX=dX, G_out=G, norms_out=n)
    for k in range(3):
        step.fill_(k)
        h.copy_(torch.randn_like(h))
        graph.replay()
        want = _lib.dp_rmsnorm_step(h, gain, y, 1.0, 0.8, 5, k, 1)
        assert all(torch.equal(a, b) for a, b in zip((dX, G, n), want)), k


def test_binding_refuses():
    x = torch.zeros(2, 3, 16, device="cuda")
    g = torch.ones(16, device="cuda")
    with pytest.raises(ValueError):
        _lib.dp_rmsnorm(x, g.to(torch.bfloat16))
    with pytest.raises(ValueError):
        _lib.dp_rmsnorm(x, g, residual=x[:1])
    with pytest.raises(ValueError):
        _lib.dp_rmsnorm(x.transpose(0, 1), g)
    with pytest.raises(ValueError):
        _lib.dp_rmsnorm(x, g, H_out=torch.empty_like(x))
    with pytest.raises(_lib.DPError):
        _lib.dp_rmsnorm(x, g, Y=x)
    with pytest.raises(_lib.DPError):
        _lib.dp_rmsnorm_step(x, g, x + 1, 1.0, 0.0, 0, 0, 0, dX=x)
    with pytest.raises(ValueError):
        _lib.dp_rmsnorm_step(x, g, x[:1], 1.0, 0.0, 0, 0, 0)
    with pytest.raises(_lib.DPError) as e:
        _lib.dp_rmsnorm(torch.zeros(1, 8196, device="cuda"), torch.ones(8196, device="cuda"))
    assert e.value.status == _lib.DP_ERR_UNSUPPORTED
