"""Cross attention to an encoder's states, and its gradients -- oracle (test
infrastructure).

Not for the product path; see the package docstring.

q [B, Lq, H, D] over k, v [B or 1, Lk, Hk, D]; head h reads key head
h // (H // Hk).  Queries from q_len[b] on and keys from kv_len[b] on do not
exist: such a query's O is 0 and its LSE -inf, and what they hold is not read."""

from __future__ import annotations

import numpy as np


def _pairs(q, k, q_len, kv_len):
    B, Lq, H, _ = q.shape
    Bk, Lk, Hk, _ = k.shape
    for b in range(B):
        e = b if Bk == B else 0
        m = Lq if q_len is None else min(max(int(q_len[b]), 0), Lq)
        n = Lk if kv_len is None else min(max(int(kv_len[e]), 0), Lk)
        if m > 0 and n > 0:
            for h in range(H):
                yield b, e, h, h // (H // Hk), m, n


def forward(q, k, v, scale, q_len=None, kv_len=None):
    """(O, LSE [B, H, Lq], weight, score): weight is the row's sum of p |v|,
    score [B, H, Lq] its largest scale * sum |q| |k|, for error bounds."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, Lq, H, D = q.shape
    O, W = np.zeros((B, Lq, H, D)), np.zeros((B, Lq, H, D))
    lse, score = np.full((B, H, Lq), -np.inf), np.zeros((B, H, Lq))
    for b, e, h, j, m, n in _pairs(q, k, q_len, kv_len):
        x = scale * (q[b, :m, h] @ k[e, :n, j].T)
        top = x.max(1)
        p = np.exp(x - top[:, None])
        total = p.sum(1)
        p /= total[:, None]
        O[b, :m, h] = p @ v[e, :n, j]
        W[b, :m, h] = p @ np.abs(v[e, :n, j])
        lse[b, h, :m] = top + np.log(total)
        score[b, h, :m] = scale * (np.abs(q[b, :m, h]) @ np.abs(k[e, :n, j]).T).max(1)
    return O, lse, W, score


def backward(q, k, v, do, scale, q_len=None, kv_len=None):
    """((dq, dk, dv), their error scales): the scales are the sums of absolute
    terms, with |dP| + |delta| in dS's place."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    out = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    bound = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    a = np.abs
    for b, e, h, j, m, n in _pairs(q, k, q_len, kv_len):
        Q, K, V, G = q[b, :m, h], k[e, :n, j], v[e, :n, j], do[b, :m, h]
        x = scale * (Q @ K.T)
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        dp = G @ V.T
        delta = (p * dp).sum(1, keepdims=True)
        ds = p * (dp - delta) * scale
        s = p * (a(G) @ a(V).T + (p * (a(G) @ a(V).T)).sum(1, keepdims=True)) * scale
        out[0][b, :m, h] = ds @ K
        out[1][e, :n, j] += ds.T @ Q
        out[2][e, :n, j] += p.T @ G
        bound[0][b, :m, h] = s @ a(K)
        bound[1][e, :n, j] += s.T @ a(Q)
        bound[2][e, :n, j] += p.T @ a(G)
    return tuple(out), tuple(bound)
