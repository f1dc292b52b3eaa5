"""A bound on fp32's error in kda_tree_verify and kda_tree_commit that stays small on deep trees.

serving_model.tree_run bounds the error by the recurrence on absolute values, which grows with every level of the tree: past
some 30 levels it exceeds the outputs themselves.  Here the error is followed through the equations that the tree's nodes
satisfy, with the signs that the inputs have: with L = I + C,

    L U = R,  R = beta (V - X),       O = Y + D U,       S' = Diag(P) S + sum_t w_t u_t^T  over the accepted path,

an error e in the residual of the first equation moves U by at most |L^-1| e, and keys of norm 1 with beta <= 1 and
alpha <= 1 keep the entries of L^-1 near 1 however deep the tree is.

Roundings, each at most u = 2^-24 of its value; g(n) = n u for a product or a sum that a value passes n of:
  * a key or query decayed along its path: one product a level; c, d and the products with the state are sums of d_k terms
    (any order: at most d_k of them), and beta's product with c: a = d_k + depth + 4 in all, of the sum of the absolute terms;
  * R: v - x and beta: 2 of beta (|v| + |x|);
  * the sum over the other nodes: at most K terms, K + 2 of |C| |U| + |R|;
  * the diagonal blocks (16 nodes) through their inverses M: a column is a substitution of at most 16 products and sums,
    (L + E) M_j = e_j with |E| <= g(17) |L|, so M is off by at most g(17) |L^-1| |L| |M| and M r by that times |r|, and
    by g(17) |M| |r| for its own product, where |r| <= |R| + |C| |U| (what the block's right-hand side is made of); L times
    that is a residual of the same equation;
  * O: K + 2 of |Y| + |D| |U|; S': 2 depth + 4 of its absolute terms.
Every bound is taken twice: once for the first-order terms left out (products of two bounds, below 1e-3 of either), which
the factor covers many times over.
"""
from __future__ import annotations

import numpy as np

from serving_model import U


def _paths(parents):
    """above [K][K]: s is an ancestor of t; depth [K]."""
    K = len(parents)
    above, depth = np.zeros((K, K), dtype=bool), np.ones(K, dtype=int)
    for t, p in enumerate(parents):
        if p >= 0:
            above[t] = above[p]
            above[t, p] = True
            depth[t] = depth[p] + 1
    return above, depth


def bounds(S, q, k, v, alpha, beta, parents, u):
    """Bounds eo, eu [K][dv] and a function es(last) -> [dk][dv] on what fp32 may be off by, for one (sequence, head).

    S [dk][dv]; q, k, alpha [K][dk]; v [K][dv]; beta [K]; u [K][dv]: the exact write vectors."""
    K, dk = k.shape
    S, q, k, v, alpha, beta = (np.asarray(a, dtype=np.float64) for a in (S, q, k, v, alpha, beta))
    above, depth = _paths(parents)
    P = np.ones((K, dk))  # decays from the root through t
    G = np.zeros((K, K, dk))  # G[t, s]: decays after the ancestor s through t
    for t, p in enumerate(parents):
        P[t] = alpha[t] * (P[p] if p >= 0 else 1.0)
        if p >= 0:
            G[t] = alpha[t] * G[p]
            G[t, p] = alpha[t]
    C = beta[:, None] * np.einsum("si,tsi,ti->ts", k, G, k)
    D = np.einsum("si,tsi,ti->ts", k, G, q) + np.diag((k * q).sum(-1))
    aC = np.abs(beta)[:, None] * np.einsum("si,tsi,ti->ts", np.abs(k), G, np.abs(k))
    aD = np.einsum("si,tsi,ti->ts", np.abs(k), G, np.abs(q)) + np.diag((np.abs(k) * np.abs(q)).sum(-1))
    aX, aY = (P * np.abs(k)) @ np.abs(S), (P * np.abs(q)) @ np.abs(S)
    X = (P * k) @ S
    R = beta[:, None] * (v - X)
    L = np.eye(K) + C
    aU, aL = np.abs(u), np.abs(L)
    dep = depth[:, None].astype(float)
    a = (dk + dep + 4) * U
    # residuals of L U = R
    res = a * np.abs(beta)[:, None] * aX + 2 * U * np.abs(beta)[:, None] * (np.abs(v) + np.abs(X))
    res += a * (aC @ aU) + (K + 2) * U * (np.abs(C) @ aU + np.abs(R))
    rhs = np.abs(R) + np.abs(C) @ aU
    for m in range(0, K, 16):
        b = slice(m, min(m + 16, K))
        M = np.abs(np.linalg.inv(L[b, b]))
        res[b] += 17 * U * aL[b, b] @ (M @ (aL[b, b] @ (M @ rhs[b])) + M @ rhs[b])
    eu = 2 * np.abs(np.linalg.inv(L)) @ res
    eo = 2 * (a * aY + a * (aD @ aU) + (K + 2) * U * (aY + np.abs(D) @ aU)) + np.abs(D) @ eu

    def es(last):
        path, t = [], last
        while t >= 0:
            path.append(t)
            t = parents[t]
        n, out = len(path), P[last][:, None] * np.abs(S)
        err = np.zeros_like(out)
        for t in path:
            w = np.abs(k[t]) * (G[last, t] if t != last else 1.0)
            out = out + np.outer(w, aU[t])
            err = err + np.outer(w, eu[t])
        return err + 2 * (2 * n + 4) * U * out

    return eo, eu, es
