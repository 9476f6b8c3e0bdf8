"""CPU oracle of the operators for long histories and drafted candidates (numpy, fp64).

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``; it imports nothing from the CUDA package.

* windowed causal attention over packed rows: row i of a user sees j <= i with j > i - window or
  j < n_sinks, padding left out; its gradients, written out from the explicit mask;
* the same for one new token over a cache;
* trees of drafted tokens over a cached history;
* rotary positions with several axes.

Query heads share key heads: head h reads key head h // (H // Hkv). Each attention also returns
what its tolerance is made of: the sums of absolute values over which a rounding of the weights
spreads.
"""

from __future__ import annotations

import numpy as np


def f64(x) -> np.ndarray:
    return np.asarray(x.detach().double().cpu().numpy() if hasattr(x, "detach") else x,
                      dtype=np.float64)


def window_mask(L: int, window: int, n_sinks: int, valid=None) -> np.ndarray:
    i, j = np.arange(L)[:, None], np.arange(L)[None, :]
    m = (j <= i) & ((j > i - window) | (j < n_sinks))
    if valid is not None:
        ok = np.asarray(valid).astype(bool)
        m &= ok[None, :] & ok[:, None]
    return m


def tree_mask(parent, n_hist: int) -> np.ndarray:
    """[n, n_hist + n]: the history, the ancestors and the token itself."""
    n = len(parent)
    m = np.zeros((n, n_hist + n), dtype=bool)
    m[:, :n_hist] = True
    for i in range(n):
        j = i
        while j >= 0:
            m[i, n_hist + j] = True
            j = int(parent[j])
    return m


def _expand(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def masked(q, k, v, mask, scale):
    """Softmax attention under an explicit mask: (out [n,H,d], lse [n,H], P [H,n,m], A [n,H,d]),
    A = P |V|. Keys that no row sees may hold anything; rows without a key give 0 and -inf."""
    q, k, v = f64(q).copy(), f64(k).copy(), f64(v).copy()
    seen, live = mask.any(0), mask.any(1)
    k[~seen] = 0.0
    v[~seen] = 0.0
    q[~live] = 0.0
    H = q.shape[1]
    k, v = _expand(k, H), _expand(v, H)
    S = scale * np.einsum("nhd,mhd->hnm", q, k)
    S = np.where(mask, S, -np.inf)
    top = np.where(live, S.max(-1, initial=-np.inf), 0.0)
    P = np.where(mask, np.exp(S - top[..., None]), 0.0)
    total = P.sum(-1)
    P /= np.where(live, total, 1.0)[..., None]
    with np.errstate(divide="ignore"):
        lse = np.where(live, top + np.log(total), -np.inf)
    return (np.einsum("hnm,mhd->nhd", P, v), lse.T, P, np.einsum("hnm,mhd->nhd", P, np.abs(v)))


def gradients(q, k, v, dout, mask, scale):
    """(dq, dk, dv) and the sums of their tolerances (see the tests): with e a relative rounding of
    the weights P and dS, and of O in rowsum(dO * O)."""
    Hkv = k.shape[1]
    out, _, P, _ = masked(q, k, v, mask, scale)
    q, k, v, do = f64(q).copy(), f64(k).copy(), f64(v).copy(), f64(dout).copy()
    seen, live = mask.any(0), mask.any(1)
    k[~seen] = 0.0
    v[~seen] = 0.0
    q[~live] = 0.0
    do[~live] = 0.0
    H = q.shape[1]
    ke, ve = _expand(k, H), _expand(v, H)
    dP = np.einsum("nhd,mhd->hnm", do, ve)
    D = (do * out).sum(-1).T[..., None]
    E = (np.abs(do) * np.abs(out)).sum(-1).T[..., None]
    dS = P * (dP - D)
    soft = np.abs(dS) + P * E                       # spread of the bf16 roundings
    hard = P * (np.abs(dP) + np.abs(D) + E)         # spread of the fp32 arithmetic

    def shared(x):
        m = x.shape[0]
        return x.reshape(m, Hkv, H // Hkv, -1).sum(2)

    dq = scale * np.einsum("hnm,mhd->nhd", dS, ke)
    dk = shared(scale * np.einsum("hnm,nhd->mhd", dS, q))
    dv = shared(np.einsum("hnm,nhd->mhd", P, do))
    tq = [scale * np.einsum("hnm,mhd->nhd", w, np.abs(ke)) for w in (soft, hard)]
    tk = [shared(scale * np.einsum("hnm,nhd->mhd", w, np.abs(q))) for w in (soft, hard)]
    tv = [shared(np.einsum("hnm,nhd->mhd", P, np.abs(do)))] * 2
    return (dq, dk, dv), (tq, tk, tv)


def rope_axes(x, positions, sections, base=10000.0, per_axis=False, sign=1.0) -> np.ndarray:
    """Rotation of [T, H, d] by positions [T, A]; pairs past the sections stay. Angles are formed in
    extended precision: in fp64 a position of 2^31 would leave 2^-22 of a radian in doubt."""
    x = f64(x)
    half = x.shape[2] // 2
    pos = np.asarray(positions).astype(np.longdouble)
    base = np.longdouble(base)
    y = x.copy()
    j = 0
    for a, n in enumerate(sections):
        for i in range(n):
            theta = base ** (-(np.longdouble(i) / n if per_axis else np.longdouble(j) / half))
            c = np.cos(pos[:, a] * theta).astype(np.float64)[:, None]
            s = sign * np.sin(pos[:, a] * theta).astype(np.float64)[:, None]
            y[..., j] = x[..., j] * c - x[..., j + half] * s
            y[..., j + half] = x[..., j] * s + x[..., j + half] * c
            j += 1
    return y
