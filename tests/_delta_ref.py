"""The gated delta rule in 64 bits (numpy), token by token from its definition in
include/r9q.h, with a bound for what fp32 kernels may be off.

The bound.  A token multiplies an error that the state has by exp(g) (1 - beta k k^T), which
for beta from 0 to 2 and |k| <= 1 does not lengthen a row.  What it adds itself: S k is a sum
of D products, off by at most 2^-19 |S| |k| (the row's 2-norm; partial sums of up to sixteen
terms and then a tree, or a tensor core's sums of two 11-bit parts of every factor), g's exponential by
2^-22, and the sums for u and S as much again: in all 2^-18 (|S| + beta |v|).  So
  E <- exp(g) E + 2^-18 (exp(g) |S| + beta |v|)
bounds every element of the row.  An output is scale S q with S rounded to 11 bits at least:
scale (E + 2^-11 |S|) + 2^-8 |o|, the last its rounding to bf16."""
import numpy as np


def unit(x, eps):
    x = x.astype(np.float64)
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + eps)


def token(S, E, q, k, v, g, beta, scale, eps):
    """One token: S [Hv][D][D], E [Hv][D]; q, k [Hk][D], v [Hv][D], g, beta [Hv] -> S, E, o, and o's bound."""
    ratio = v.shape[0] // k.shape[0]
    q, k = (np.repeat(unit(x, eps), ratio, 0) for x in (q, k))
    a = np.exp(g.astype(np.float64))[:, None]
    S = np.where(a[..., None] == 0, 0.0, a[..., None] * S)
    u = beta.astype(np.float64)[:, None] * (v.astype(np.float64) - np.einsum("hvk,hk->hv", S, k))
    E = a * E + 2.0 ** -18 * (np.linalg.norm(S, axis=-1) + np.abs(beta[:, None] * v))
    S = S + u[..., None] * k[:, None]
    o = scale * np.einsum("hvk,hk->hv", S, q)
    return S, E, o, scale * (E + 2.0 ** -11 * np.linalg.norm(S, axis=-1)) + 2.0 ** -8 * 1.01 * np.abs(o)


def chain(S, q, k, v, g, beta, scale, eps=1e-6, E=None):
    """Tokens one after another: the state, its bound [Hv][D], outputs [n][Hv][D] and theirs."""
    E = np.zeros(v.shape[1:]) if E is None else E
    o, w = np.zeros(v.shape), np.zeros(v.shape)
    for t in range(len(v)):
        S, E, o[t], w[t] = token(S, E, q[t], k[t], v[t], g[t], beta[t], scale, eps)
    return S, E, o, w


def tree(S, q, k, v, g, beta, parents, scale, eps=1e-6):
    """Every node from its parent's state: outputs and their bounds (zeros where there is no node)."""
    after = {-1: (S, np.zeros(v.shape[1:]))}
    o, w = np.zeros(v.shape), np.zeros(v.shape)
    for i, p in enumerate(parents):
        if p >= -1:
            s, e, o[i], w[i] = token(*after[p], q[i], k[i], v[i], g[i], beta[i], scale, eps)
            after[i] = (s, e)
    return o, w
