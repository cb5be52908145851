"""The embedding's lookup and privatised gradient against the fp64 oracle.

Bounds.  A group's rows are added in fp32: m additions are off by at most m u of the sum of the
terms' magnitudes, u = 2^-24.  A row of S adds its groups times their factors (one product and one
addition each, and the factor's own rounding).  Norms are the root of fp32 squares added over a
chunk (8 or 4 squares a lane, 5 additions over the warp: at most 13 roundings, half of that after
the root) and then in fp64."""
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


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _lib.lib()


def _draw(B, T, V, d, dt, seed, index="int64", lo=0, spread=1.0):
    rng = np.random.default_rng(seed)
    ids = np.minimum((V - lo) ** rng.random((B, T)) - 1 + lo, V - 1).astype(np.int64)
    dY = rng.standard_normal((B, T, d)) * np.exp(spread * rng.standard_normal((B, 1, 1))) / np.sqrt(T * d)
    dYt = torch.from_numpy(dY.astype(np.float32)).to(DT[dt])
    return ids, torch.from_numpy(ids).to(getattr(torch, index)).cuda(), dYt.double().numpy(), dYt.cuda()


def _bounds(ids, dY, V, C, scale, padding_idx, ref):
    """(norms' absolute bounds [B], S's absolute bounds [V, d]) by the reasoning above."""
    B, T, d = dY.shape
    keep = (ids >= 0) & (ids < V) & (ids != (-1 if padding_idx is None else padding_idx))
    mags = [oracle.embedding_gradient(ids[i], np.abs(dY[i]), V, abs(scale), padding_idx) for i in range(B)]
    most = [np.bincount(ids[i][keep[i]], minlength=V).max() if keep[i].any() else 0 for i in range(B)]
    norm = np.array([(m + 2) * U32 * np.linalg.norm(g) + 10 * U32 * n for m, g, n in zip(most, mags, ref["norms"])])
    S = np.zeros((V, d))
    groups = np.zeros(V)
    for i in range(B):
        rel_c = norm[i] / ref["norms"][i] if ref["norms"][i] > C else 0.0
        S += ref["c"][i] * mags[i] * ((most[i] + 4) * U32 + rel_c)
        groups += np.bincount(ids[i][keep[i]], minlength=V) > 0
    total = sum(c * m for c, m in zip(ref["c"], mags))
    # The additions over a row's groups, and the one rounding of the stored value.
    S += (groups[:, None] + 2) * U32 * total + U32 * np.abs(ref["out"]) + 1e-11
    return norm, S


def _check(B, T, V, d, dt, seed, C=1.0, sigma=0.0, scale=1.0, padding_idx=None, index="int64", ids=None, **kw):
    ids_h, ids_d, dY_h, dY_d = _draw(B, T, V, d, dt, seed, index, **kw)
    if ids is not None:
        ids_h = ids(ids_h)
        ids_d = torch.from_numpy(ids_h).to(ids_d.dtype).cuda()
    # The C ABI takes C, sigma and scale in fp32; the oracle gets the values that reach it.
    C, sigma, scale = (float(np.float32(v)) for v in (C, sigma, scale))
    ref = oracle.embedding_step(ids_h, dY_h, V, C, sigma, 7, 3, 2, scale=scale, padding_idx=padding_idx)
    G, n = _lib.dp_embedding_step(ids_d, dY_d, V, C, sigma, 7, 3, 2, scale=scale, padding_idx=padding_idx)
    bn, bS = _bounds(ids_h, dY_h, V, C, scale, padding_idx, ref)
    assert np.all(np.abs(host(n) - ref["norms"]) <= bn + 1e-300)
    err = np.abs(host(G) - ref["out"])
    assert np.all(err <= bS), float(np.max(err / bS))
    return ids_d, dY_d, G, n, ref, bn, bS


SHAPES = [
    # B, T, V, d: one token; one row; every id the same; lengths about a warp and a block; long
    # groups and heavy rows; more than one chunk with a ragged last one; ids of 1, 2 and 3 digits.
    (1, 1, 1, 8), (1, 1, 70000, 16), (3, 5, 1, 8), (2, 31, 7, 24), (2, 33, 7, 264), (4, 16, 512, 64),
    (5, 333, 40, 136), (2, 700, 3, 520), (9, 257, 255, 72), (9, 257, 256, 72), (3, 129, 65535, 40), (3, 129, 65536, 40),
    (70, 40, 11, 16), (1, 4099, 300, 32), (16, 1031, 261, 104),
    # more tokens than a pass of the sort keeps in registers, in one digit and in three
    (5, 9001, 200, 8), (1, 70001, 70000, 8),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_step_matches_the_oracle(shape, dt):
    B, T, V, d = shape
    _check(B, T, V, d, dt, seed=sum(shape), sigma=0.7 if V * d < 2_000_000 else 0.0, scale=0.5,
           index="int32" if d % 16 else "int64")


@pytest.mark.parametrize("V", [511, 512, 2 ** 18 - 1, 2 ** 18])
@pytest.mark.parametrize("B,T", [(2, 300), (2, 2500)])
def test_tables_at_the_ends_of_the_sorts_digits(V, B, T):
    """Where the digits' width or number changes; uniform ids, the first and last ones among them."""
    ids = np.random.default_rng(V + T).integers(0, V, (B, T))
    ids[0, :4] = ids[-1, -4:] = (V - 1, 0, 255, 256)
    _check(B, T, V, 8, "bf16", seed=V, ids=lambda _: ids, padding_idx=256)


@pytest.mark.parametrize("first", [0, 5, 17, 31])
def test_group_and_row_lengths_around_the_thresholds(first):
    """Groups of 1 to 130 tokens of one id, alone and as rows of several samples, at every phase of the
    windows of 16 and 32 positions in which the order is read."""
    lengths = [1, 2, 15, 16, 17, 18, 31, 32, 33, 47, 48, 49, 63, 64, 65, 66, 96, 130]
    T = first + sum(lengths)
    one = np.concatenate([np.arange(first)] + [np.full(n, first + k) for k, n in enumerate(lengths)])
    rng = np.random.default_rng(first)
    # Two samples with the same ids in different orders, and one that has each id once or not at all.
    ids = np.stack([rng.permutation(one), rng.permutation(one), np.arange(T) % 60])
    _check(3, T, 60, 72, "bf16", seed=first, ids=lambda _: ids, sigma=0.3)


def test_offsets_past_32_bits():
    """A table, an output and a gradient of more than 2^31 elements: the far rows are found."""
    d, V, N = 4096, 530_000, 530_000
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    far = [V - 1, V - 2, 524_288, 262_144, 1]
    for k, v in enumerate(far):
        W[v] = k + 1
    y = _lib.dp_embedding_lookup(W, torch.tensor(far, device="cuda"))
    assert [float(r.min()) for r in y] == [float(r.max()) for r in y] == [1, 2, 3, 4, 5]
    ids = torch.zeros(1, N, dtype=torch.int32, device="cuda")
    ids[0, -3:] = torch.tensor([7, 9, 7], dtype=torch.int32)
    W.zero_()
    dY = W.view(1, N, d)
    dY[0, -3:] = torch.tensor([[1.0], [2.0], [4.0]], device="cuda").to(torch.bfloat16)
    G, n = _lib.dp_embedding_step(ids, dY, 12, 1000.0, 0.0, 0, 0, 0)
    assert abs(float(n[0]) - np.sqrt(d * 29.0)) <= 1e-3
    assert float(G[7].min()) == float(G[7].max()) == 5.0 and float(G[9].min()) == 2.0 == float(G[9].max())
    assert float(G[:7].abs().max()) == 0.0
    # and the output of a lookup past 2^31 elements
    Y = _lib.dp_embedding_lookup(torch.arange(12, device="cuda").to(torch.bfloat16)[:, None].expand(12, d).contiguous(), ids, out=dY)
    assert [float(v) for v in Y[0, -4:, 0]] == [0.0, 7.0, 9.0, 7.0]


def test_narrow_fp32_rows():
    _check(3, 50, 9, 4, "f32", seed=1)
    _check(3, 50, 9, 132, "f32", seed=2, sigma=1.0)


def test_padding_negative_and_outside_ids_belong_to_no_row():
    def ids(x):
        x = x.copy()
        x[0, 10:] = 0          # padding
        x[1, :] = 0            # a sample of padding alone: norm 0
        x[2, ::3] = -1
        x[3, ::2] = -100
        return x

    ids_d, dY_d, G, n, ref, bn, bS = _check(5, 64, 12, 40, "bf16", seed=5, padding_idx=0, ids=ids, sigma=0.0)
    assert float(n[1]) == 0.0 and float(G[0].abs().max()) == 0.0
    # Their gradients are not read as numbers: NaN and infinity there change nothing.
    bad = dY_d.clone()
    bad[ids_d <= 0] = float("nan")
    bad[1] = float("inf")
    G2, n2 = _lib.dp_embedding_step(ids_d, bad, 12, 1.0, 0.0, 7, 3, 2, scale=1.0, padding_idx=0)
    assert torch.equal(G, G2) and torch.equal(n, n2)
    # An id past the table is skipped too, and reported.
    past = ids_d.clone()
    past[ids_d < 0] = 12
    ws = torch.empty(_lib.embedding_workspace_size(5, 64, 12, 40), dtype=torch.uint8, device="cuda")
    G3, n3 = _lib.dp_embedding_step(past, dY_d, 12, 1.0, 0.0, 7, 3, 2, padding_idx=0, workspace=ws)
    assert torch.equal(G, G3) and torch.equal(n, n3)
    assert _lib.dp_workspace_status(ws) == _lib.DP_ERR_INVALID_ARG
    past[ids_d < 0] = 2 ** 33 + 1
    G3, n3 = _lib.dp_embedding_step(past, dY_d, 12, 1.0, 0.0, 7, 3, 2, padding_idx=0, workspace=ws)
    assert torch.equal(G, G3) and _lib.dp_workspace_status(ws) == _lib.DP_ERR_INVALID_ARG
    _lib.dp_embedding_step(ids_d, dY_d, 12, 1.0, 0.0, 7, 3, 2, padding_idx=0, workspace=ws)
    assert _lib.dp_workspace_status(ws) == _lib.DP_OK


def test_no_token_at_all():
    ids = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    dY = torch.randn(2, 9, 16, device="cuda")
    G, n = _lib.dp_embedding_step(ids, dY, 5, 1.0, 1.0, 1, 2, 3)
    assert float(n.abs().max()) == 0.0
    z = oracle.noise(5, 16, 1.0, 1, 2, 3)
    assert np.all(np.abs(host(G) - z) <= U32 * np.abs(z) + 1e-11)


def test_infinite_bound_is_the_plain_gradient():
    ids_d, dY_d, G, n, *_ = _check(4, 100, 30, 64, "f32", seed=9, C=float("inf"))


def test_norms_and_accumulate_make_the_step():
    ids_h, ids_d, dY_h, dY_d = _draw(6, 300, 50, 264, "bf16", 11)
    G, n = _lib.dp_embedding_step(ids_d, dY_d, 80, 0.9, 0.0, 0, 0, 0, scale=2.0, padding_idx=3)
    n2 = _lib.dp_embedding_per_sample_norms(ids_d, dY_d, 80, scale=2.0, padding_idx=3)
    assert torch.equal(n, n2)
    S = torch.zeros(80, 264, device="cuda")
    _lib.dp_embedding_clip_accumulate(ids_d, dY_d, n, 0.9, S, scale=2.0, padding_idx=3)
    assert torch.equal(S, G)
    # Accumulating a second time adds the same sum; rows without a token keep what they held.
    S[60:] = float("nan")
    _lib.dp_embedding_clip_accumulate(ids_d, dY_d, n, 0.9, S, scale=2.0, padding_idx=3)
    assert torch.equal(S[:50], G[:50] + G[:50]) and torch.isnan(S[60:]).all()
    # Flat norms of several layers clip this table's gradient as one vector with theirs.
    flat = torch.sqrt(n * n + 4.0)
    F = torch.zeros(80, 264, device="cuda")
    _lib.dp_embedding_clip_accumulate(ids_d, dY_d, flat, 0.9, F, scale=2.0, padding_idx=3)
    want = sum(min(1.0, float(np.float32(0.9)) / f) * oracle.embedding_gradient(i, y, 80, 2.0, 3)
               for f, i, y in zip(host(flat), ids_h, dY_h))
    assert np.linalg.norm(host(F) - want) <= 300 * U32 * np.linalg.norm(want) * 4


def test_bits_repeat_and_surroundings_stay():
    ids_h, ids_d, dY_h, dY_d = _draw(8, 500, 90, 328, "bf16", 12)
    need = _lib.embedding_workspace_size(8, 500, 90, 328)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    buf = torch.full((92, 328), 7.0, device="cuda")
    first = None
    for _ in range(4):
        ws[:need] = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")   # whatever was there before
        G, n = _lib.dp_embedding_step(ids_d, dY_d, 90, 1.0, 0.5, 1, 2, 3, workspace=ws[:need], G_out=buf[1:91])
        first = (G.clone(), n.clone()) if first is None else first
        assert torch.equal(G, first[0]) and torch.equal(n, first[1])
    assert (ws[need:] == 0x5A).all() and (buf[0] == 7.0).all() and (buf[91] == 7.0).all()


def test_graph_replays_follow_inputs_and_step():
    ids_h, ids_d, dY_h, dY_d = _draw(4, 200, 64, 128, "bf16", 13)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.empty(_lib.embedding_workspace_size(4, 200, 64, 128), dtype=torch.uint8, device="cuda")
    G = torch.empty(64, 128, device="cuda")
    n = torch.empty(4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.dp_embedding_step(ids_d, dY_d, 64, 1.0, 0.8, 5, step, 1, workspace=ws, G_out=G, norms_out=n)
    for k in range(3):
        step.fill_(k)
        ids_d.copy_(torch.randint(0, 64, ids_d.shape, device="cuda"))
        dY_d.copy_(torch.randn_like(dY_d) / 100)
        graph.replay()
        want, wn = _lib.dp_embedding_step(ids_d, dY_d, 64, 1.0, 0.8, 5, k, 1)
        assert torch.equal(G, want) and torch.equal(n, wn), k


def test_two_streams_at_once():
    a = _draw(8, 400, 64, 256, "bf16", 14)
    b = _draw(8, 400, 64, 256, "bf16", 15)
    want = [_lib.dp_embedding_step(x[1], x[3], 64, 1.0, 0.3, 5, 0, 1) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got.append([_lib.dp_embedding_step(x[1], x[3], 64, 1.0, 0.3, 5, 0, 1, stream=s) for x, s in zip((a, b), streams)])
    torch.cuda.synchronize()
    for pair in got:
        for (G, n), (Gw, nw) in zip(pair, want):
            assert torch.equal(G, Gw) and torch.equal(n, nw)


@pytest.mark.parametrize("wdt,odt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("N,V,d", [(1, 1, 8), (7, 3, 24), (1000, 333, 1032), (33, 70000, 64)])
def test_lookup(wdt, odt, N, V, d):
    rng = np.random.default_rng(N + d)
    W = torch.from_numpy(rng.standard_normal((V, d)).astype(np.float32)).to(DT[wdt])
    ids = torch.from_numpy(rng.integers(-2, V + 2, N))
    for index in (torch.int64, torch.int32):
        got = _lib.dp_embedding_lookup(W.cuda(), ids.to(index).cuda(), scale=1.1, out_dtype=DT[odt])
        inside = (ids >= 0) & (ids < V)
        # The scale reaches the library in fp32, the product is rounded in fp32, then to the output.
        want = W.double()[ids.clamp(0, V - 1)] * float(np.float32(1.1)) * inside[:, None]
        half = 2 * U32 + (2.0 ** -8 if odt == "bf16" else 0.0)
        assert got.dtype == DT[odt] and bool(((got.cpu().double() - want).abs() <= half * want.abs()).all())
    if odt == wdt == "f32":
        w4 = torch.randn(5, 12, device="cuda")
        i4 = torch.tensor([[4, 0], [2, 2]], device="cuda")
        assert torch.equal(_lib.dp_embedding_lookup(w4, i4), w4[i4])


def test_lookup_of_no_token():
    assert _lib.dp_embedding_lookup(torch.ones(3, 8, device="cuda"), torch.empty(0, 5, dtype=torch.int64, device="cuda")).shape == (0, 5, 8)


def test_binding_refuses():
    ids = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    dY = torch.zeros(2, 3, 16, device="cuda")
    args = (4, 1.0, 0.0, 0, 0, 0)
    with pytest.raises(ValueError):
        _lib.dp_embedding_step(ids.cpu(), dY, *args)
    with pytest.raises(ValueError):
        _lib.dp_embedding_step(ids[:, :2], dY, *args)
    with pytest.raises(ValueError):
        _lib.dp_embedding_step(ids, dY.transpose(0, 1).contiguous().transpose(0, 1), *args)
    with pytest.raises(TypeError):
        _lib.dp_embedding_step(ids.to(torch.int16), dY, *args)
    with pytest.raises(TypeError):
        _lib.dp_embedding_step(ids, dY.half(), *args)
    with pytest.raises(ValueError):
        _lib.dp_embedding_step(ids, dY, *args, G_out=torch.zeros(4, 8, device="cuda"))
    with pytest.raises(_lib.DPError):
        _lib.dp_embedding_step(ids, dY[..., :6].contiguous(), *args)
    with pytest.raises(_lib.DPError):
        _lib.dp_embedding_step(ids, dY, *args, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
