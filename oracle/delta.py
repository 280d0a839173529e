"""fp64 oracle of the gated delta rule and of the layer norms' backward passes.

Gated delta rule, per value head, S [Dk, Dv]:
    S <- exp(g) S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q,
token by token; the adjoint is the same loop backwards with the states kept.
"""
from __future__ import annotations

import numpy as np


def _per_value_head(x, hv):
    return np.repeat(np.asarray(x, np.float64), hv // x.shape[1], axis=1)


def sequence(q, k, v, g, beta, scale, state, do=None, dstate=None):
    """One sequence: q, k [T, Hk, Dk], v [T, Hv, Dv], g, beta [T, Hv], state
    [Hv, Dk, Dv]. Returns (o, last state), and with do a dict of gradients
    (q, k, v, g, beta, initial_state) too; dstate is the last state's gradient."""
    T, hv, dv = v.shape
    hk, dk = k.shape[1:]
    qq, kk = _per_value_head(q, hv), _per_value_head(k, hv)
    v, g, beta = (np.asarray(x, np.float64) for x in (v, g, beta))
    S = np.array(state, np.float64)
    o = np.zeros((T, hv, dv))
    kept = []
    with np.errstate(invalid="ignore"):
        for t in range(T):
            Sd = np.exp(g[t])[:, None, None] * S
            miss = v[t] - np.einsum("hkv,hk->hv", Sd, kk[t])
            u = beta[t][:, None] * miss
            S = Sd + kk[t][:, :, None] * u[:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S, qq[t])
            if do is not None:
                kept.append((Sd, miss, u, S))
    if do is None:
        return o, S
    do = np.asarray(do, np.float64)
    D = np.zeros_like(S) if dstate is None else np.array(dstate, np.float64)
    dq, dk_, dv_ = np.zeros((T, hv, dk)), np.zeros((T, hv, dk)), np.zeros((T, hv, dv))
    dg, db = np.zeros((T, hv)), np.zeros((T, hv))
    for t in range(T - 1, -1, -1):
        Sd, miss, u, S1 = kept[t]
        dq[t] = scale * np.einsum("hkv,hv->hk", S1, do[t])
        D = D + scale * qq[t][:, :, None] * do[t][:, None, :]
        du = np.einsum("hkv,hk->hv", D, kk[t])
        db[t] = (du * miss).sum(-1)
        dm = beta[t][:, None] * du
        dv_[t] = dm
        dk_[t] = np.einsum("hkv,hv->hk", D, u) - np.einsum("hkv,hv->hk", Sd, dm)
        D = D - kk[t][:, :, None] * dm[:, None, :]
        dg[t] = (D * Sd).sum((-1, -2))
        D = D * np.exp(g[t])[:, None, None]
    shared = lambda x: x.reshape(T, hk, hv // hk, dk).sum(2)  # noqa: E731
    return o, S, {"q": shared(dq), "k": shared(dk_), "v": dv_, "g": dg, "beta": db, "initial_state": D}


def gated_delta(q, k, v, g, beta, scale, state=None, cu=None, do=None, dstate=None):
    """All sequences: [Bt, T, ...] inputs, or with cu (N + 1 offsets) N
    sequences packed in [1, T, ...]. Rows of o and of the gradients that no
    sequence covers are NaN."""
    if cu is None:
        spans = [((b, slice(None)), b) for b in range(v.shape[0])]
    else:
        spans = [((0, slice(cu[i], cu[i + 1])), i) for i in range(len(cu) - 1)]
    n, hv, dk, dv = len(spans), v.shape[2], k.shape[3], v.shape[3]
    state = np.zeros((n, hv, dk, dv)) if state is None else np.asarray(state, np.float64)
    o, last = np.full(v.shape, np.nan), np.zeros((n, hv, dk, dv))
    grads = None
    if do is not None:
        grads = {m: np.full(x.shape, np.nan) for m, x in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta))}
        grads["initial_state"] = np.zeros((n, hv, dk, dv))
    for at, i in spans:
        args = (q[at], k[at], v[at], g[at], beta[at], scale, state[i])
        if do is None:
            o[at], last[i] = sequence(*args)
            continue
        o[at], last[i], gr = sequence(*args, do=do[at], dstate=None if dstate is None else dstate[i])
        for m in ("q", "k", "v", "g", "beta"):
            grads[m][at] = gr[m]
        grads["initial_state"][i] = gr["initial_state"]
    return (o, last) if do is None else (o, last, grads)


def layer_norm_backward(dz, x, gamma, eps):
    """Norm over the last axis: (z - beta, mean, rstd, dx, dgamma, dbeta)."""
    x, dz, gamma = (np.asarray(a, np.float64) for a in (x, dz, gamma))
    mu = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    xhat = (x - mu) * rstd
    h = dz * gamma
    dx = rstd * (h - h.mean(-1, keepdims=True) - xhat * (h * xhat).mean(-1, keepdims=True))
    others = tuple(range(x.ndim - 1))
    return xhat * gamma, mu[..., 0], rstd[..., 0], dx, (dz * xhat).sum(others), dz.sum(others)
