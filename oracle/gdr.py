"""Head-gated delta rule and state-cache pages in 64 bits, token by token (numpy) — test infrastructure.

One value head, state S [dk, dv]:  S' = e^g S;  u = beta (v - S'^T k);  S = S' + k u^T;  o = S^T q.
Value head h reads key head h // (Hv // Hk).
"""
import numpy as np


def _rep(x, Hv):
    return np.repeat(np.asarray(x, np.float64), Hv // x.shape[1], axis=1)


def forward(q, k, v, g, beta, cu, s0=None):
    """q, k [T, Hk, dk]; v [T, Hv, dv]; g, beta [T, Hv]; cu [N + 1]; s0 [N, Hv, dk, dv] or None.
    Returns out [T, Hv, dv] (zeros at tokens of no sequence) and the final states."""
    v = np.asarray(v, np.float64)
    Hv, dv = v.shape[1:]
    q, k = _rep(q, Hv), _rep(k, Hv)
    a, beta = np.exp(np.asarray(g, np.float64)), np.asarray(beta, np.float64)
    N, dk = len(cu) - 1, q.shape[-1]
    S = np.zeros((N, Hv, dk, dv)) if s0 is None else np.array(s0, np.float64)
    out = np.zeros_like(v)
    for n in range(N):
        s = S[n]
        for t in range(cu[n], cu[n + 1]):
            s = a[t][:, None, None] * s
            u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", s, k[t]))
            s = s + k[t][:, :, None] * u[:, None, :]
            out[t] = np.einsum("hkv,hk->hv", s, q[t])
        S[n] = s
    return out, S


def backward(q, k, v, g, beta, cu, d_out, s0=None, d_final=None):
    """Reverse mode of `forward`: dict dq, dk, dv, dg, dbeta, d_initial_state."""
    Hk = q.shape[1]
    v, d_out = np.asarray(v, np.float64), np.asarray(d_out, np.float64)
    Hv, dv = v.shape[1:]
    q, k = _rep(q, Hv), _rep(k, Hv)
    a, beta = np.exp(np.asarray(g, np.float64)), np.asarray(beta, np.float64)
    N, dk = len(cu) - 1, q.shape[-1]
    r = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dg": np.zeros_like(a),
         "dbeta": np.zeros_like(a)}
    dS = np.zeros((N, Hv, dk, dv)) if d_final is None else np.array(d_final, np.float64)
    for n in range(N):
        s = np.zeros((Hv, dk, dv)) if s0 is None else np.array(s0[n], np.float64)
        kept = []
        for t in range(cu[n], cu[n + 1]):
            sd = a[t][:, None, None] * s
            e = v[t] - np.einsum("hkv,hk->hv", sd, k[t])
            s = sd + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
            kept.append((sd, e, s))
        d = dS[n]
        for t in reversed(range(cu[n], cu[n + 1])):
            sd, e, s = kept[t - cu[n]]
            r["dq"][t] = np.einsum("hkv,hv->hk", s, d_out[t])
            d = d + q[t][:, :, None] * d_out[t][:, None, :]
            du = np.einsum("hkv,hk->hv", d, k[t])
            r["dbeta"][t] = (du * e).sum(-1)
            r["dv"][t] = beta[t][:, None] * du
            r["dk"][t] = np.einsum("hkv,hv->hk", d, beta[t][:, None] * e) - np.einsum("hkv,hv->hk", sd, r["dv"][t])
            d = d - k[t][:, :, None] * r["dv"][t][:, None, :]
            r["dg"][t] = (d * sd).sum((-1, -2))
            d = a[t][:, None, None] * d
        dS[n] = d
    for x in ("dq", "dk"):
        r[x] = r[x].reshape(r[x].shape[0], Hk, Hv // Hk, dk).sum(2)
    r["d_initial_state"] = dS
    return r


def decode(q, k, v, g, beta, pages, index=None):
    """[N, T, H, ...] tokens on pages[index]; returns (out with zeros at idle rows, pages)."""
    pages = np.array(pages, np.float64)
    out = np.zeros(v.shape)
    for n in range(len(q)):
        p = n if index is None else int(index[n])
        if p < 0 or p >= len(pages) or (index is not None and p in [int(x) for x in index[:n]]):
            continue
        out[n], s = forward(q[n], k[n], v[n], g[n], beta[n], [0, q.shape[1]], pages[p][None])
        pages[p] = s[0]
    return out, pages


def fork(cache, refs, parents):
    cache, refs = np.array(cache), np.array(refs)
    free = np.flatnonzero(refs == 0)
    old = cache.copy()
    live = refs > 0
    children = np.full(len(parents), -1, np.int32)
    for i, p in enumerate(parents):
        if i >= len(free) or not (p == -1 or (0 <= p < len(live) and live[p])):
            continue
        children[i] = free[i]
        refs[free[i]] = 1
        cache[:, free[i]] = 0 if p == -1 else old[:, p]
    return cache, refs, children


def copy(cache, src, dst):
    cache = np.array(cache)
    old = cache.copy()
    P = cache.shape[1]
    for i, (s, d) in enumerate(zip(src, dst)):
        if not (-1 <= s < P and -1 <= d < P) or d == -1:
            continue
        if any(dst[j] == d for j in range(i)):
            continue
        if any(j != i and dst[j] >= 0 and dst[j] == s and src[j] != dst[j] for j in range(len(src))):
            continue
        cache[:, d] = 0 if s == -1 else old[:, s]
    return cache


def compact(cache, refs, table):
    cache, refs, table = np.array(cache), np.array(refs), np.array(table)
    m = int((refs > 0).sum())
    to = np.where(refs > 0, np.arange(len(refs)), -1)
    movers = [p for p in range(m, len(refs)) if refs[p] > 0]
    holes = [p for p in range(m) if refs[p] <= 0]
    for s, d in zip(movers, holes):
        cache[:, d] = cache[:, s]
        refs[d], refs[s] = refs[s], 0
        to[s] = d
    table = np.array([-1 if t == -1 or not 0 <= t < len(to) else to[t] for t in table], np.int32)
    return cache, refs, table, m
