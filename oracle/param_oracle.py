"""fp64 oracle of the parameters beside the linears (embedding table, RMS norm gain) and of the
Muon step.  Plain numpy, one sample's whole gradient at a time; shares no code with the library."""
from __future__ import annotations

import numpy as np

from .dp_oracle import clip_factors, noise

__all__ = ["embedding_gradient", "embedding_step", "rmsnorm", "rmsnorm_gradients", "rmsnorm_step", "newton_schulz",
           "muon_step", "NEWTON_SCHULZ"]

# x <- a x + b x^3 + c x^5 on every singular value (the Muon optimiser's published coefficients).
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def embedding_gradient(ids_i, dY_i, V, scale=1.0, padding_idx=None):
    """One sample's gradient of the table [V, d]: row v sums scale * dY over the tokens with id v.
    Ids outside [0, V) and the padding index name no row."""
    G = np.zeros((V, dY_i.shape[1]))
    for t, v in enumerate(np.asarray(ids_i).tolist()):
        if 0 <= v < V and v != padding_idx:
            G[v] += float(scale) * np.asarray(dY_i[t], dtype=np.float64)
    return G


def _privatise(gradients, C, sigma, seed, step, layer_id):
    """Norms, clip factors, clipped sum and noise of per-sample gradients of any one shape."""
    norms = np.array([np.sqrt(np.sum(g * g)) for g in gradients])
    c = clip_factors(norms, C)
    S = np.zeros_like(gradients[0])
    for ci, g in zip(c, gradients):
        S += ci * g
    flat = S.reshape(-1, S.shape[-1])
    z = (noise(flat.shape[0], flat.shape[1], float(sigma) * float(C), seed, step, layer_id).reshape(S.shape)
         if sigma != 0 else np.zeros_like(S))
    return {"norms": norms, "c": c, "S": S, "noise": z, "out": S + z}


def embedding_step(ids, dY, V, C, sigma, seed, step, layer_id, scale=1.0, padding_idx=None):
    return _privatise([embedding_gradient(ids[i], dY[i], V, scale, padding_idx) for i in range(len(ids))], C, sigma,
                      seed, step, layer_id)


def rmsnorm(h, gain, eps):
    """y = h / sqrt(mean(h^2) + eps) * gain over the last axis."""
    h = np.asarray(h, dtype=np.float64)
    return h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * gain


def rmsnorm_gradients(h, gain, dY, eps):
    """(gradient of h, per-sample gradients of the gain [B, d]) of sum(dY * rmsnorm(h))."""
    h, dY, gain = (np.asarray(v, dtype=np.float64) for v in (h, dY, gain))
    r = 1.0 / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
    u = dY * gain
    dh = r * u - h * r ** 3 * np.mean(u * h, axis=-1, keepdims=True)
    return dh, np.sum(dY * h * r, axis=1)


def rmsnorm_step(h, gain, dY, C, sigma, seed, step, layer_id, eps, residual_grad=None):
    dh, per = rmsnorm_gradients(h, gain, dY, eps)
    out = _privatise(list(per), C, sigma, seed, step, layer_id)
    out["dX"] = dh if residual_grad is None else dh + np.asarray(residual_grad, dtype=np.float64)
    out["per_sample"] = per
    return out


def newton_schulz(G, steps=5):
    """X = G / (||G|| + 1e-7), then `steps` times X <- a X + b X X^T X + c (X X^T)^2 X."""
    a, b, c = NEWTON_SCHULZ
    X = np.asarray(G, dtype=np.float64)
    X = X / (np.linalg.norm(X) + 1e-7)
    for _ in range(steps):
        if X.shape[0] <= X.shape[1]:
            A = X @ X.T
            X = a * X + (b * A + c * (A @ A)) @ X
        else:
            A = X.T @ X
            X = a * X + X @ (b * A + c * (A @ A))
    return X


def muon_step(W, R, M, lr, momentum, nesterov, weight_decay, grad_scale, update_scale, steps=5):
    """(W, M): M <- momentum M + g, g = grad_scale R; U orthogonalises g + momentum M (nesterov) or M;
    W <- (1 - lr weight_decay) W - lr update_scale U."""
    g = float(grad_scale) * np.asarray(R, dtype=np.float64)
    M = float(momentum) * np.asarray(M, dtype=np.float64) + g
    U = newton_schulz(g + float(momentum) * M if nesterov else M, steps)
    return (1.0 - float(lr) * float(weight_decay)) * np.asarray(W, dtype=np.float64) - float(lr) * float(update_scale) * U, M
