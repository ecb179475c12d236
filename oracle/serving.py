"""Plain fp64 definitions of the serving operators (numpy, token by token, row by row).

Test infrastructure only; shares no code with the kernels.  Inputs are numpy arrays whose
values are exactly those the kernels get (bf16 values widened), outputs are float64.
"""

from __future__ import annotations

import numpy as np


def delta_rule(q, k, v, log_alpha, beta, cu, pool, slot):
    """The gated delta rule over packed sequences; returns (o [T,Hv,dv], pool after)."""
    Hv, dv = v.shape[1:]
    heads = np.arange(Hv) // (Hv // q.shape[1])
    o = np.zeros((v.shape[0], Hv, dv))
    out = np.array(pool, dtype=np.float64)
    for b in range(len(cu) - 1):
        S = out[slot[b]].copy()
        for t in range(cu[b], cu[b + 1]):
            kt, qt = k[t][heads].astype(np.float64), q[t][heads].astype(np.float64)
            S *= np.exp(log_alpha[t].astype(np.float64))[:, None, None]
            u = beta[t][:, None].astype(np.float64) * (v[t] - np.einsum("hk,hkv->hv", kt, S))
            S += kt[:, :, None] * u[:, None, :]
            o[t] = np.einsum("hk,hkv->hv", qt, S)
        out[slot[b]] = S
    return o, out


def attend(q, k, v, parent, cu, k_cache, v_cache, table, ctx, prefix_pages, prefix_len, scale):
    """Returns (o [T,Hq,D], lse [T,Hq], a [T,Hq,D]) with a = sum_j p_j |v_j|, the size of
    the terms whose sum o is (what a rounding of the weights acts on)."""
    T, Hq, D = q.shape
    page, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    o, a = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)

    def cached(cache, pages, length):
        return np.array([cache[pages[p // page], p % page] for p in range(length)],
                        dtype=np.float64).reshape(length, Hkv, D)

    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        K = [cached(k_cache, prefix_pages, prefix_len), cached(k_cache, table[b], ctx[b])]
        V = [cached(v_cache, prefix_pages, prefix_len), cached(v_cache, table[b], ctx[b])]
        for i in range(n):
            path, at = [], i
            while at >= 0 and k is not None:
                path.append(cu[b] + at)
                at = parent[cu[b] + at] if parent is not None else at - 1
            own = [] if k is None else path[::-1]
            Ki = np.concatenate(K + ([k[own].astype(np.float64)] if own else []))
            Vi = np.concatenate(V + ([v[own].astype(np.float64)] if own else []))
            if not len(Ki):
                continue
            for h in range(Hq):
                s = scale * (Ki[:, h // G] @ q[cu[b] + i, h].astype(np.float64))
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                lse[cu[b] + i, h] = m + np.log(z)
                o[cu[b] + i, h] = (p / z) @ Vi[:, h // G]
                a[cu[b] + i, h] = (p / z) @ np.abs(Vi[:, h // G])
    return o, lse, a


def cache_append(k, v, cu, k_cache, v_cache, table, ctx, path=None, path_len=None):
    """Returns (k_cache, v_cache, new_len) after the call."""
    k_cache, v_cache, page = k_cache.copy(), v_cache.copy(), k_cache.shape[1]
    new_len = np.array(ctx).copy()
    for b in range(len(cu) - 1):
        rows = (range(cu[b + 1] - cu[b]) if path is None
                else [int(x) for x in path[b][:path_len[b]]])
        for j, r in enumerate(rows):
            p = int(ctx[b]) + j
            k_cache[table[b][p // page], p % page] = k[cu[b] + r]
            v_cache[table[b][p // page], p % page] = v[cu[b] + r]
        new_len[b] += len(rows)
    return k_cache, v_cache, new_len
