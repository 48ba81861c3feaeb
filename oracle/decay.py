"""Decay attention and its gradients -- oracle (test infrastructure).

Not for the product path; see the package docstring.

Per (b, h), g = exp(log_decay[h]): S_t = g S_{t-1} + k_t v_t^T,
o_t = scale q_t S_t, evaluated token by token in float64.  Gradients by the
adjoint recurrence R_t = X_t + scale q_t dO_t^T, dk_t = R_t v_t,
dv_t = R_t^T k_t, X_{t-1} = g R_t, dq_t = scale S_t dO_t.  Tokens past a
sequence's length are padding: output and gradients 0, state untouched.

Each output also comes with a scale for error bounds: the same sum with every
product replaced by its absolute value, which bounds what rounding a factor of
each product by a relative r can change (by r times that sum)."""

from __future__ import annotations

import numpy as np


def _decay(log_decay):
    return np.exp(np.minimum(np.asarray(log_decay, dtype=np.float64), 0.0))


def decay_attention(q, k, v, log_decay, scale, state=None, lens=None):
    """[B, L, H, D] inputs -> (O, S, O_abs, S_abs)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, L, H, D = q.shape
    g = _decay(log_decay)[:, None, None]
    S = np.zeros((B, H, D, D)) if state is None else np.array(state, dtype=np.float64)
    A = np.abs(S)
    O, Oa = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        n = L if lens is None else min(max(int(lens[b]), 0), L)
        for t in range(n):
            kv = k[b, t, :, :, None] * v[b, t, :, None, :]
            S[b] = g * S[b] + kv
            A[b] = g * A[b] + np.abs(kv)
            O[b, t] = scale * np.einsum("hd,hde->he", q[b, t], S[b])
            Oa[b, t] = scale * np.einsum("hd,hde->he", np.abs(q[b, t]), A[b])
    return O, S, Oa, A


def decay_attention_backward(q, k, v, do, log_decay, scale, state=None, dstate=None, lens=None):
    """-> ((dq, dk, dv, d_state_in), (their absolute sums))."""
    q, k, v, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, do))
    B, L, H, D = q.shape
    g = _decay(log_decay)[:, None, None]
    S = np.zeros((B, H, D, D)) if state is None else np.array(state, dtype=np.float64)
    R = np.zeros((B, H, D, D)) if dstate is None else np.array(dstate, dtype=np.float64)
    A, Ra = np.abs(S), np.abs(R)
    out = [np.zeros_like(q) for _ in range(6)]
    dq, dk, dv, dqa, dka, dva = out
    for b in range(B):
        n = L if lens is None else min(max(int(lens[b]), 0), L)
        for t in range(n):
            kv = k[b, t, :, :, None] * v[b, t, :, None, :]
            S[b] = g * S[b] + kv
            A[b] = g * A[b] + np.abs(kv)
            dq[b, t] = scale * np.einsum("hde,he->hd", S[b], do[b, t])
            dqa[b, t] = scale * np.einsum("hde,he->hd", A[b], np.abs(do[b, t]))
        for t in range(n - 1, -1, -1):
            w = scale * q[b, t, :, :, None] * do[b, t, :, None, :]
            R[b] += w
            Ra[b] += np.abs(w)
            dk[b, t] = np.einsum("hde,he->hd", R[b], v[b, t])
            dv[b, t] = np.einsum("hde,hd->he", R[b], k[b, t])
            dka[b, t] = np.einsum("hde,he->hd", Ra[b], np.abs(v[b, t]))
            dva[b, t] = np.einsum("hde,hd->he", Ra[b], np.abs(k[b, t]))
            R[b] *= g
            Ra[b] *= g
    return (dq, dk, dv, R), (dqa, dka, dva, Ra)
