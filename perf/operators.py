"""Cases of the operators around the privatised linears: the embedding table and the RMS norm's
gain (a transformer's other parameters, clipped and noised per sample like its linears) and the
Muon step that applies a privatised gradient.

Every case is one call a private training step makes:

  lookup    y = scale * W[ids]
  embedding the privatised gradient of that lookup's table: per-sample norms, clipped sum, noise
  norm      h = x + residual, y = h / rms(h) * gain
  norm_step the backward of that norm: dh, and the privatised gradient of the gain
  ortho     five Newton-Schulz products on a momentum matrix
  muon      momentum, orthogonalisation and weight update of one linear

Plain forms are elementary torch operations in 32 bits (the noise in 64, as it is defined),
rounded once at the end.
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)  # a, b, c of the orthogonalising quintic
STEPS = 5
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # The repository's smallest workload (4 samples of 16 tokens, 64 wide, fp32): launch latency.
        {"name": "lookup tiny", "op": "lookup", "B": 4, "T": 16, "V": 512, "d": 64, "dt": "f32", "scale": 8.0, "index": "int32"},
        # The tokens of the Llama-7B block workload.
        {"name": "lookup 8x2048 4096", "op": "lookup", "B": 8, "T": 2048, "V": 32000, "d": 4096, "dt": "bf16", "scale": 1.0,
         "index": "int64"},
        {"name": "embedding tiny", "op": "embedding", "B": 4, "T": 16, "V": 512, "d": 64, "dt": "f32", "scale": 8.0, "sigma": 1.0,
         "pad": 0.0, "index": "int32"},
        # A small vocabulary (bytes): long groups of the same token in every sample, a ragged width,
        # padded tails, one shard of a batch (its noise is added after the all-reduce).
        {"name": "embedding bytes", "op": "embedding", "B": 16, "T": 1031, "V": 261, "d": 1032, "dt": "bf16", "scale": 1.0,
         "sigma": 0.0, "pad": 0.3, "index": "int64"},
        # The GPT-2 workload's batch with its usual vocabulary.
        {"name": "embedding 32x512 768", "op": "embedding", "B": 32, "T": 512, "V": 50257, "d": 768, "dt": "bf16", "scale": 1.0,
         "sigma": 0.8, "pad": 0.0, "index": "int64"},
        # The Llama-7B workload's batch: the table's gradient is 0.5 GB.
        {"name": "embedding 8x2048 4096", "op": "embedding", "B": 8, "T": 2048, "V": 32000, "d": 4096, "dt": "bf16", "scale": 1.0,
         "sigma": 1.0, "pad": 0.1, "index": "int64"},
        # A few rows (a short prompt), and the Llama-13B workload's rows with their residual.
        {"name": "norm 4 rows", "op": "norm", "B": 1, "T": 4, "d": 4096, "dt": "bf16", "res": True},
        {"name": "norm 4x2048 5120", "op": "norm", "B": 4, "T": 2048, "d": 5120, "dt": "bf16", "res": True},
        # Odd sizes in fp32, no residual branch; the Llama-7B workload's rows with it.
        {"name": "norm_step ragged", "op": "norm_step", "B": 7, "T": 333, "d": 1028, "dt": "f32", "res": False, "sigma": 0.5},
        {"name": "norm_step 8x2048 4096", "op": "norm_step", "B": 8, "T": 2048, "d": 4096, "dt": "bf16", "res": True, "sigma": 1.0},
        # A projected gradient of the RoBERTa workload (r = 128), and a linear of the Llama-7B block.
        {"name": "ortho 1024x128", "op": "ortho", "m": 1024, "n": 128, "dt": "f32"},
        {"name": "muon 4096x11008", "op": "muon", "m": 4096, "n": 11008, "lr": 1e-3, "wd": 0.01, "nesterov": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, q):
    return max(q, _log(rng, lo / q, hi / q) * q)


def draw(rng):
    op = rng.choice(["lookup", "embedding", "embedding", "norm", "norm_step", "norm_step", "ortho", "muon"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    q = 8 if dt == "bf16" else 4
    if op in ("ortho", "muon"):
        m, n = _width(rng, 64, 4096, 8), _width(rng, 64, 4096, 8)
        if op == "ortho":
            return {"op": op, "m": m, "n": n, "dt": dt}
        return {"op": op, "m": m, "n": n, "lr": 10 ** rng.uniform(-4, -2.7), "wd": rng.choice([0.0, 0.01]),
                "nesterov": rng.random() < 0.5}
    B, T = _log(rng, 1, 64), _log(rng, 1, 2048)
    T = max(1, min(T, 16384 // B))
    d = _width(rng, 64, 5120, q)
    c = {"op": op, "B": B, "T": T, "d": d, "dt": dt}
    if op in ("lookup", "embedding"):
        c["V"] = _log(rng, 2, 32000)
        c["scale"] = rng.choice([1.0, math.sqrt(d)])
        c["index"] = rng.choice(["int32", "int64"])
        if op == "embedding":
            c["sigma"] = rng.choice([0.0, round(rng.uniform(0.3, 2.0), 2)])
            c["pad"] = rng.choice([0.0, round(rng.uniform(0.05, 0.9), 2)])
        return c
    c["res"] = rng.random() < 0.5
    if op == "norm_step":
        c["sigma"] = rng.choice([0.0, round(rng.uniform(0.3, 2.0), 2)])
    return c


# ----------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, dt=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def _ids(case, g):
    """Token ids with frequencies falling like 1 / rank, as text has them; the first row of the
    table is the padding token, and a share of the samples ends in it."""
    B, T, V = case["B"], case["T"], case["V"]
    u = torch.rand(B, T, generator=g, device="cuda", dtype=torch.float64)
    ids = torch.clamp(torch.exp(u * math.log(V)).long(), 1, V) - 1
    if case.get("pad"):
        keep = (T * (1.0 - case["pad"] * torch.rand(B, 1, generator=g, device="cuda"))).ceil()
        ids = torch.where(torch.arange(T, device="cuda")[None, :] < keep, ids, torch.zeros_like(ids))
    return ids.to(torch.int32 if case["index"] == "int32" else torch.int64)


def _sample_scales(g, B):
    """Samples whose gradient norms spread around the bound: some are clipped, some are not."""
    return torch.exp(torch.randn(B, 1, 1, generator=g, device="cuda"))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": dict(case), "seed": int(seed)}
    if op in ("ortho", "muon"):
        m, n = case["m"], case["n"]
        # A few strong directions over noise, as a privatised gradient has.
        k = min(8, m, n)
        R = _normal(g, m, k) @ _normal(g, k, n) * (2.0 / math.sqrt(k)) + _normal(g, m, n)
        if op == "ortho":
            s["G"] = R.to(DT[case["dt"]])
        else:
            s["R"] = R
            s["M"] = _normal(g, m, n, std=2.0)
            s["W"] = _normal(g, m, n, std=1.0 / math.sqrt(m))
        return s
    B, T, d, dt = case["B"], case["T"], case["d"], DT[case["dt"]]
    if op in ("lookup", "embedding"):
        s["ids"] = _ids(case, g)
        if op == "lookup":
            s["W"] = _normal(g, case["V"], d, dt=dt)
        else:
            std = 1.0 / (case["scale"] * math.sqrt(T * d))
            s["dY"] = (_normal(g, B, T, d, std=std) * _sample_scales(g, B)).to(dt)
        return s
    s["X"] = _normal(g, B, T, d, dt=dt)
    s["gain"] = 1.0 + 0.2 * _normal(g, d)
    if case["res"]:
        s["res"] = _normal(g, B, T, d, std=2.0 if op == "norm" else 0.02, dt=dt)
    if op == "norm_step":
        s["dY"] = (_normal(g, B, T, d, std=1.0 / math.sqrt(T * d)) * _sample_scales(g, B)).to(dt)
    return s


# ---------------------------------------------------------------------------- the plain forms
def _philox(j, layer, step, key):
    """Philox4x32-10 words of blocks j (int64 tensor), as int64 tensors of 32-bit values."""
    mask = 0xFFFFFFFF
    k0, k1 = key & mask, (key >> 32) & mask
    x0, x1 = j & mask, torch.full_like(j, layer)
    x2, x3 = torch.full_like(j, step & mask), torch.zeros_like(j)
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((b >> 32) & mask) ^ x1 ^ k0, b & mask, ((a >> 32) & mask) ^ x3 ^ k1, a & mask
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return x0, x1, x2, x3


def _noise(n, layer, step, key):
    """The first n standard normals of the noise stream, fp64."""
    j = torch.arange((n + 3) // 4, device="cuda", dtype=torch.int64)
    x0, x1, x2, x3 = _philox(j, layer, step, key)
    z = []
    for a, b in ((x0, x1), (x2, x3)):
        r = torch.sqrt(-2.0 * torch.log((a.double() + 1.0) * 2.0 ** -32))
        t = b.double() * (2.0 * math.pi * 2.0 ** -32)
        z += [r * torch.cos(t), r * torch.sin(t)]
    return torch.stack(z, dim=1).reshape(-1)[:n]


def _plus_noise(S, std, layer, step, key):
    if std == 0.0:
        return S.float()
    return (S.double() + std * _noise(S.numel(), layer, step, key).reshape(S.shape)).float()


def _clip(n, C):
    return torch.where(n <= C, torch.ones_like(n), C / n)


def _plain_lookup(W, ids, scale):
    inside = (ids >= 0) & (ids < W.shape[0])
    rows = W[torch.where(inside, ids, torch.zeros_like(ids)).long()].float() * scale
    return torch.where(inside[..., None], rows, torch.zeros_like(rows)).to(W.dtype)


def _plain_embedding(ids, dY, V, C, sigma, seed, step, layer, scale, padding_idx):
    B, T, d = dY.shape
    flat = ids.reshape(-1).long()
    used = torch.nonzero((flat >= 0) & (flat < V) & (flat != padding_idx))[:, 0]
    sample = used // T
    groups, of = torch.unique(sample * V + flat[used], return_inverse=True)
    rows = torch.zeros(groups.numel(), d, device=dY.device).index_add_(0, of, dY.reshape(B * T, d)[used].float()) * scale
    owner = groups // V
    norms = torch.sqrt(torch.zeros(B, device=dY.device).index_add_(0, owner, (rows * rows).sum(1)))
    S = torch.zeros(V, d, device=dY.device).index_add_(0, groups % V, rows * _clip(norms, C)[owner][:, None])
    return _plus_noise(S, float(sigma) * C, layer, step, seed), norms


def _plain_norm(X, gain, res):
    h = X if res is None else (X.float() + res.float()).to(X.dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * gain
    return y.to(X.dtype), h


def _plain_norm_step(H, gain, dY, res, C, sigma, seed, step, layer):
    h, dy = H.float(), dY.float()
    inv = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    xhat, gy = h * inv, dy * gain
    dx = inv * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))
    if res is not None:
        dx = dx + res.float()
    per = (dy * xhat).sum(1)
    norms = torch.sqrt((per * per).sum(1))
    S = (per * _clip(norms, C)[:, None]).sum(0)
    return dx.to(H.dtype), _plus_noise(S, float(sigma) * C, layer, step, seed), norms


def _plain_ortho(G):
    X = G.float()
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (torch.sqrt((X * X).sum()) + 1e-7)
    a, b, c = NS
    for _ in range(STEPS):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.T if tall else X


def _plain_muon(W, R, M, lr, momentum, nesterov, wd, grad_scale, update_scale):
    g = R * grad_scale
    M.mul_(momentum).add_(g)
    U = _plain_ortho(g + momentum * M if nesterov else M)
    W.mul_(1.0 - lr * wd).sub_(U * (lr * update_scale))
    return W, M


LAYER, STEP, BOUND, MU, GRAD_SCALE, UPDATE_SCALE = 3, 11, 1.0, 0.95, 1.0 / 64, 1.0


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        from sample_gradient_clipping_b200 import _lib

        if op == "lookup":
            return _lib.dp_embedding_lookup(s["W"], s["ids"], scale=c["scale"])
        if op == "embedding":
            return _lib.dp_embedding_step(s["ids"], s["dY"], c["V"], BOUND, c["sigma"], s["seed"], STEP, LAYER, scale=c["scale"],
                                          padding_idx=0 if c["pad"] else None)
        if op == "norm":
            return _lib.dp_rmsnorm(s["X"], s["gain"], eps=EPS, residual=s.get("res"))
        if op == "norm_step":
            return _lib.dp_rmsnorm_step(s["X"], s["gain"], s["dY"], BOUND, c["sigma"], s["seed"], STEP, LAYER, eps=EPS,
                                        residual_grad=s.get("res"))
        if op == "ortho":
            return _lib.dp_orthogonalize(s["G"], steps=STEPS)
        # The weights and the momentum are updated in place, here and in the plain form.
        return _lib.dp_muon_step(s["W"], s["R"], s["M"], c["lr"], momentum=MU, nesterov=c["nesterov"], weight_decay=c["wd"],
                                 grad_scale=GRAD_SCALE, update_scale=UPDATE_SCALE, steps=STEPS)
    if op == "lookup":
        return _plain_lookup(s["W"], s["ids"], c["scale"])
    if op == "embedding":
        return _plain_embedding(s["ids"], s["dY"], c["V"], BOUND, c["sigma"], s["seed"], STEP, LAYER, c["scale"],
                                0 if c["pad"] else -1)
    if op == "norm":
        return _plain_norm(s["X"], s["gain"], s.get("res"))
    if op == "norm_step":
        return _plain_norm_step(s["X"], s["gain"], s["dY"], s.get("res"), BOUND, c["sigma"], s["seed"], STEP, LAYER)
    if op == "ortho":
        return _plain_ortho(s["G"]).to(torch.bfloat16)
    return _plain_muon(s["W"], s["R"], s["M"], c["lr"], MU, c["nesterov"], c["wd"], GRAD_SCALE, UPDATE_SCALE)


# ------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("ortho", "muon"):
        m, n = min(case["m"], case["n"]), max(case["m"], case["n"])
        # A = X X^T and A^2 are symmetric (half the products each); (bA + cA^2) X is whole.
        flops = STEPS * (m * m * n + m * m * m + 2.0 * m * m * n)
        if op == "ortho":
            return {"bytes": m * n * (2 + (4 if case["dt"] == "f32" else 2)), "flops": flops}
        return {"bytes": m * n * 4 * 5, "flops": flops}  # R, M, W read; M, W written
    N, d = case["B"] * case["T"], case["d"]
    e = 2 if case["dt"] == "bf16" else 4
    if op in ("lookup", "embedding"):
        idx = N * (4 if case["index"] == "int32" else 8)
        if op == "lookup":
            return {"bytes": idx + (N + min(N, case["V"])) * d * e, "flops": N * d}
        # dY read once, the table's gradient written once.
        return {"bytes": idx + N * d * e * (1.0 - case["pad"] / 2) + case["V"] * d * 4 + case["B"] * 4, "flops": 4.0 * N * d}
    if op == "norm":
        return {"bytes": N * d * e * (4 if case["res"] else 2) + d * 4, "flops": 5.0 * N * d}
    return {"bytes": N * d * e * (4 if case["res"] else 3) + d * 8 + case["B"] * 4, "flops": 14.0 * N * d}


# --------------------------------------------------------------------------- 64-bit definitions
def _exact_noise(n, layer, step, key):
    """z_k from the counter's definition, words held as (n, 4) and multiplied in 16-bit halves."""
    blocks = -(-n // 4)
    ctr = torch.zeros(4, blocks, dtype=torch.int64, device="cuda")
    ctr[0] = torch.arange(blocks, device="cuda")
    ctr[1], ctr[2] = layer, step % 2 ** 32
    keys = [key % 2 ** 32, key // 2 ** 32]

    def wide(x, k):
        lo, hi = (x % 65536) * k, (x // 65536) * k  # both below 2^48
        mid = hi + lo // 65536
        return mid // 65536, (mid % 65536) * 65536 + lo % 65536

    for r in range(10):
        h0, l0 = wide(ctr[0], 0xD2511F53)
        h2, l2 = wide(ctr[2], 0xCD9E8D57)
        ctr = torch.stack([h2 ^ ctr[1] ^ ((keys[0] + r * 0x9E3779B9) % 2 ** 32), l2,
                           h0 ^ ctr[3] ^ ((keys[1] + r * 0xBB67AE85) % 2 ** 32), l0])
    u = ctr.double()
    rad = torch.sqrt(-2 * torch.log((u[0::2] + 1) / 2.0 ** 32))
    ang = 2 * math.pi * (u[1::2] / 2.0 ** 32)
    out = torch.empty(blocks, 4, dtype=torch.float64, device="cuda")
    out[:, 0::2] = (rad * torch.cos(ang)).T
    out[:, 1::2] = (rad * torch.sin(ang)).T
    return out.flatten()[:n]


def _exact_ortho(X):
    X = X.double()
    U = X / (X.norm() + 1e-7)
    a, b, c = NS
    for _ in range(STEPS):
        if U.shape[0] <= U.shape[1]:
            K = U.matmul(U.mT)
            KU = K.matmul(U)
            U = a * U + b * KU + c * K.matmul(KU)
        else:
            K = U.mT.matmul(U)
            UK = U.matmul(K)
            U = a * U + b * UK + c * UK.matmul(K)
    return U


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ortho":
        return _exact_ortho(s["G"])
    if op == "muon":
        g = s["R"].double() * GRAD_SCALE
        M = MU * s["M"].double() + g
        U = _exact_ortho(g + MU * M if case["nesterov"] else M)
        return s["W"].double() * (1 - case["lr"] * case["wd"]) - case["lr"] * UPDATE_SCALE * U, M
    if op == "lookup":
        return s["W"].double().index_select(0, s["ids"].flatten().long()).reshape(case["B"], case["T"], case["d"]) * case["scale"]
    C = BOUND
    if op == "embedding":
        V, d = case["V"], case["d"]
        S = torch.zeros(V, d, dtype=torch.float64, device="cuda")
        norms = []
        for i in range(case["B"]):  # one sample's whole gradient at a time
            ids, dy = s["ids"][i].long(), s["dY"][i].double()
            if case["pad"]:
                dy = dy * (ids != 0).double()[:, None]
            here, at = torch.unique(ids, return_inverse=True)
            G = torch.zeros(here.numel(), d, dtype=torch.float64, device="cuda").index_add_(0, at, dy) * case["scale"]
            n = G.norm()
            norms.append(n)
            S[here] += G * torch.clamp(C / n, max=1.0)
        if case["sigma"]:
            S += (case["sigma"] * C) * _exact_noise(V * d, LAYER, STEP, s["seed"]).reshape(V, d)
        return S, torch.stack(norms)
    X, g = s["X"], s["gain"].double()
    if op == "norm":
        h = X.double() if not case["res"] else X.double() + s["res"].double()
        f = h.to(X.dtype).double()  # the norm is taken of the stored sum, which its backward reads
        return g * f / torch.sqrt(f.square().mean(-1, keepdim=True) + EPS), h
    h, dy = X.double(), s["dY"].double()
    rms = torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
    # d/dh of sum(dy g h / rms): the direct term, less what flows through rms.
    dh = dy * g / rms - h * (dy * g * h).sum(-1, keepdim=True) / (case["d"] * rms ** 3)
    if case["res"]:
        dh = dh + s["res"].double()
    per = torch.einsum("btd,btd->bd", dy, h / rms)
    norms = per.norm(dim=1)
    S = torch.clamp(C / norms, max=1.0) @ per
    if case["sigma"]:
        S = S + case["sigma"] * C * _exact_noise(case["d"], LAYER, STEP, s["seed"])
    return dh, S, norms
