"""The embedding, RMS norm and Muon entry points without a GPU: workspace sizes, and bad arguments
refused on the host before the device is touched."""
import math

import pytest

from sample_gradient_clipping_b200 import _lib, build

E, W, U = _lib.DP_ERR_INVALID_ARG, _lib.DP_ERR_WORKSPACE, _lib.DP_ERR_UNSUPPORTED
FAKE, ODD = 0x10000, 0x10004          # never dereferenced: every case fails on the host
BF16, F32, I32, I64 = _lib.DP_BF16, _lib.DP_F32, _lib.DP_I32, _lib.DP_I64


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def _embedding(L, **kw):
    a = dict(ids=FAKE, it=I64, dY=FAKE, dt=BF16, B=2, T=4, V=9, d=16, scale=1.0, pad=-1, C=1.0, sigma=1.0, step=0,
             norms=None, G=FAKE, ws=FAKE, ws_bytes=1 << 30)
    dev = kw.pop("dev", False)
    a.update(kw)
    entry = L.dp_embedding_step_dev_step if dev else L.dp_embedding_step
    return entry(a["ids"], a["it"], a["dY"], a["dt"], a["B"], a["T"], a["V"], a["d"], a["scale"], a["pad"], a["C"],
                 a["sigma"], 0, a["step"], 0, a["norms"], a["G"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(ids=None), E), (dict(dY=None), E), (dict(G=None), E), (dict(ws=None), E), (dict(ids=ODD), E),
    (dict(ids=FAKE + 2, it=I32), E), (dict(dY=ODD), E), (dict(G=ODD), E), (dict(ws=FAKE + 16), E), (dict(it=2), E),
    (dict(dt=5), E), (dict(B=0), E), (dict(T=0), E), (dict(V=0), E), (dict(V=2**31 - 1, d=8), E), (dict(d=0), E),
    (dict(d=12), E), (dict(dt=F32, d=6), E), (dict(B=1 << 16, T=1 << 15), E), (dict(V=1 << 30, d=24), E),
    (dict(scale=math.inf), E), (dict(scale=math.nan), E), (dict(C=0.0), E), (dict(C=math.nan), E), (dict(sigma=-1.0), E),
    (dict(sigma=math.inf), E), (dict(C=math.inf), E), (dict(ws_bytes=300), W), (dict(dev=True, step=None), E),
    (dict(dev=True, step=ODD), E),
])
def test_embedding_step_rejects_on_host(L, kw, want):
    assert _embedding(L, **kw) == want


def test_embedding_pieces_reject_on_host(L):
    ws = 1 << 30

    def norms(**k):
        a = dict(dict(ids=FAKE, dY=FAKE, d=16, norms=FAKE, ws=FAKE, n=ws), **k)
        return L.dp_embedding_per_sample_norms(a["ids"], I64, a["dY"], BF16, 2, 4, 9, a["d"], 1.0, -1, a["norms"],
                                               a["ws"], a["n"], None)

    assert norms(ids=None) == norms(dY=ODD) == norms(d=12) == norms(norms=None) == norms(ws=ODD) == E
    assert norms(n=100) == W

    def acc(**k):
        a = dict(dict(norms=FAKE, C=1.0, G=FAKE, n=ws), **k)
        return L.dp_embedding_clip_accumulate(FAKE, I64, FAKE, BF16, 2, 4, 9, 16, 1.0, -1, a["norms"], a["C"], a["G"],
                                              FAKE, a["n"], None)

    assert acc(norms=None) == acc(C=0.0) == acc(C=math.nan) == acc(G=None) == acc(G=ODD) == E
    assert acc(n=100) == W

    def lookup(**k):
        a = dict(dict(W=FAKE, wdt=BF16, ids=FAKE, it=I64, scale=1.0, N=5, V=9, d=16, Y=FAKE, ydt=BF16), **k)
        return L.dp_embedding_lookup(a["W"], a["wdt"], a["ids"], a["it"], a["scale"], a["N"], a["V"], a["d"], a["Y"],
                                     a["ydt"], None)

    for k in (dict(W=None), dict(W=ODD), dict(wdt=3), dict(ids=None), dict(ids=ODD), dict(it=7), dict(scale=math.inf),
              dict(N=0), dict(N=1 << 31), dict(V=0), dict(d=12), dict(d=12, wdt=F32), dict(d=6, wdt=F32, ydt=F32),
              dict(Y=None), dict(Y=ODD), dict(ydt=9)):
        assert lookup(**k) == E, k


def test_embedding_workspace_size(L):
    f = L.dp_embedding_workspace_size
    N, V, d = 8 * 2048, 32000, 4096
    longs = N // 17 + 1                                   # fp32 sums of groups of more than 16 tokens
    want = N * 17 + 8 * V + N * 8 * 4 + longs * (d * 4 + 8)
    assert want <= f(8, 2048, V, d, BF16) < want + 8192
    assert f(8, 2048, V, 12, BF16) == 0 and f(8, 2048, V, 12, F32) > 0 and f(0, 1, 1, 8, BF16) == 0


def _norm_step(L, **kw):
    a = dict(H=FAKE, gain=FAKE, dY=FAKE + 64, res=None, dt=BF16, B=2, T=4, d=16, eps=1e-6, C=1.0, sigma=1.0, step=0,
             dX=FAKE + 128, norms=None, G=FAKE, ws=FAKE, ws_bytes=1 << 30)
    dev = kw.pop("dev", False)
    a.update(kw)
    entry = L.dp_rmsnorm_step_dev_step if dev else L.dp_rmsnorm_step
    return entry(a["H"], a["gain"], a["dY"], a["res"], a["dt"], a["B"], a["T"], a["d"], a["eps"], a["C"], a["sigma"], 0,
                 a["step"], 0, a["dX"], a["norms"], a["G"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(H=None), E), (dict(gain=None), E), (dict(dY=None), E), (dict(dX=None), E), (dict(G=None), E), (dict(ws=None), E),
    (dict(H=ODD), E), (dict(gain=ODD), E), (dict(dY=ODD), E), (dict(dX=ODD), E), (dict(G=ODD), E), (dict(res=ODD), E),
    (dict(ws=FAKE + 16), E), (dict(dX=FAKE), E), (dict(dX=FAKE + 64), E), (dict(res=FAKE + 128), E), (dict(dt=4), E),
    (dict(B=0), E), (dict(T=0), E), (dict(d=0), E), (dict(d=12), E), (dict(B=65536), E), (dict(B=60000, T=60000), E),
    (dict(eps=-1.0), E), (dict(eps=math.nan), E), (dict(eps=math.inf), E), (dict(C=0.0), E), (dict(C=math.inf), E),
    (dict(sigma=math.nan), E), (dict(d=16392), U), (dict(dt=F32, d=8196), U), (dict(ws_bytes=300), W),
    (dict(dev=True, step=None), E), (dict(dev=True, step=ODD), E),
])
def test_rmsnorm_step_rejects_on_host(L, kw, want):
    assert _norm_step(L, **kw) == want


def test_rmsnorm_pieces_reject_on_host(L):
    def fwd(**k):
        a = dict(dict(X=FAKE, res=FAKE + 64, gain=FAKE, dt=BF16, rows=3, d=16, eps=1e-6, H=FAKE + 128, Y=FAKE + 256), **k)
        return L.dp_rmsnorm(a["X"], a["res"], a["gain"], a["dt"], a["rows"], a["d"], a["eps"], a["H"], a["Y"], None)

    for k in (dict(X=None), dict(X=ODD), dict(gain=None), dict(gain=ODD), dict(res=ODD), dict(H=None), dict(H=ODD),
              dict(Y=None), dict(Y=ODD), dict(Y=FAKE), dict(Y=FAKE + 64), dict(H=FAKE), dict(H=FAKE + 64),
              dict(H=FAKE + 256), dict(rows=0), dict(rows=1 << 31), dict(d=12), dict(eps=-1.0), dict(dt=2)):
        assert fwd(**k) == E, k
    assert fwd(d=16392) == U

    def bwd(**k):
        a = dict(dict(per=FAKE, norms=FAKE, n=1 << 30), **k)
        return L.dp_rmsnorm_backward(FAKE, FAKE, FAKE + 64, None, BF16, 2, 4, 16, 1e-6, FAKE + 128, a["per"], a["norms"],
                                     FAKE, a["n"], None)

    assert bwd(per=None) == bwd(per=ODD) == bwd(norms=None) == E and bwd(n=10) == W

    def acc(**k):
        a = dict(dict(per=FAKE, norms=FAKE, B=2, d=16, C=1.0, G=FAKE), **k)
        return L.dp_rmsnorm_clip_accumulate(a["per"], a["norms"], a["B"], a["d"], a["C"], a["G"], None)

    for k in (dict(per=None), dict(per=ODD), dict(norms=None), dict(B=0), dict(d=0), dict(d=6), dict(C=0.0), dict(C=math.nan),
              dict(G=None), dict(G=ODD)):
        assert acc(**k) == E, k
    assert acc(d=16388) == acc(d=2**31 - 4) == U


def test_rmsnorm_workspace_size(L):
    f = L.dp_rmsnorm_workspace_size
    # 148 x 2 blocks of rows, one partial column sum each, and a gradient a sample.
    parts = 8 * 37 * 4096 * 4
    assert parts + 8 * 4096 * 4 <= f(8, 2048, 4096, BF16) < parts + 8 * 4096 * 4 + 4096
    assert f(8, 2048, 12, BF16) == 0 and f(8, 2048, 16392, BF16) == 0 and f(1, 1, 4, F32) > 0


def test_muon_rejects_on_host(L):
    def ortho(**k):
        a = dict(dict(G=FAKE, dt=F32, m=64, n=32, steps=5, U=FAKE + 64, ws=FAKE, n_ws=1 << 30), **k)
        return L.dp_orthogonalize(a["G"], a["dt"], a["m"], a["n"], a["steps"], a["U"], a["ws"], a["n_ws"], None)

    for k in (dict(G=None), dict(G=ODD), dict(dt=3), dict(m=0), dict(m=12), dict(n=4), dict(n=36), dict(steps=0),
              dict(steps=33), dict(U=None), dict(U=ODD), dict(U=FAKE), dict(ws=None), dict(ws=FAKE + 16),
              dict(m=131072, n=131080), dict(m=65544, n=65544), dict(m=8, n=2**30 + 8)):
        assert ortho(**k) == E, k
    assert ortho(n_ws=1000) == W

    def muon(**k):
        a = dict(dict(W=FAKE, R=FAKE + 64, M=FAKE + 128, m=64, n=32, lr=0.1, mu=0.9, wd=0.0, gs=1.0, us=1.0, steps=5,
                      ws=FAKE, n_ws=1 << 30), **k)
        return L.dp_muon_step(a["W"], a["R"], a["M"], a["m"], a["n"], a["lr"], a["mu"], 1, a["wd"], a["gs"], a["us"],
                              a["steps"], a["ws"], a["n_ws"], None)

    for k in (dict(W=None), dict(W=ODD), dict(R=None), dict(R=ODD), dict(R=FAKE), dict(M=None), dict(M=ODD), dict(M=FAKE),
              dict(M=FAKE + 64), dict(m=12), dict(lr=-1.0), dict(lr=math.inf), dict(lr=math.nan), dict(mu=1.0),
              dict(mu=-0.1), dict(mu=math.nan), dict(wd=-1.0), dict(wd=math.inf), dict(gs=math.nan), dict(us=math.inf),
              dict(steps=0), dict(steps=33), dict(ws=None), dict(ws=FAKE + 16)):
        assert muon(**k) == E, k
    assert muon(n_ws=1000) == W


def test_muon_workspace_size(L):
    f = L.dp_muon_workspace_size
    assert 8 * 64 * 32 + 4 * 32 * 32 <= f(64, 32) < 8 * 64 * 32 + 4 * 32 * 32 + 16384
    assert f(64, 32) == f(32, 64) and f(64, 12) == 0 and f(0, 8) == 0
