"""fp64 CPU oracle of linear attention with one decay per head and of causal
softmax attention.

TEST INFRASTRUCTURE ONLY, under the same rule as the rest of ``oracle/``: only
``tests/`` may use it; the HIP library never does.

Linear attention, per value head j with query/key head i = j // (Hv / Hk), one
token at a time:

    S_t = exp(g_j) S_{t-1} + k_t v_t^T
    o_t = scale S_t^T q_t

Softmax attention, per query head h with key head h // (Hq / Hkv), one query at
a time: query t of lq sees the first lk - lq + t + 1 of the lk keys,

    o_t = sum_s exp(a_s) v_s / sum_s exp(a_s),   a_s = scale q_t . k_s

and o_t = 0 when it sees none.

Each function also returns the same sums over absolute values, which bound what
rounding a term can do to its output.
"""
from __future__ import annotations

import numpy as np


def _f64(*arrays):
    return [np.asarray(a, dtype=np.float64) for a in arrays]


def linattn(q, k, v, g, S0=None, scale=1.0):
    """One sequence: q, k [L, Hk, dk], v [L, Hv, dv], g [Hv], S0 [Hv, dk, dv].
    Returns (o [L, Hv, dv], S, |o| bound, |S| bound)."""
    q, k, v, g = _f64(q, k, v, g)
    L, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    r = Hv // Hk
    S = np.zeros((Hv, dk, dv)) if S0 is None else np.array(S0, dtype=np.float64)
    A = np.abs(S)
    lam = np.exp(g)[:, None, None]
    o, ao = np.empty((L, Hv, dv)), np.empty((L, Hv, dv))
    for t in range(L):
        kt, qt = np.repeat(k[t], r, axis=0), np.repeat(q[t], r, axis=0)
        S = lam * S + kt[:, :, None] * v[t][:, None, :]
        A = lam * A + np.abs(kt)[:, :, None] * np.abs(v[t])[:, None, :]
        o[t] = scale * np.einsum("hk,hkv->hv", qt, S)
        ao[t] = abs(scale) * np.einsum("hk,hkv->hv", np.abs(qt), A)
    return o, S, ao, A


def attn(q, k, v, scale):
    """One sequence: q [lq, Hq, D], k, v [lk, Hkv, D].  Returns (o [lq, Hq, D],
    sum_s p_s |v_s|, the largest sum_d |scale q_d k_d| of a visible score)."""
    q, k, v = _f64(q, k, v)
    lq, Hq, D = q.shape
    lk, Hkv = k.shape[:2]
    o, ao = np.zeros((lq, Hq, D)), np.zeros((lq, Hq, D))
    big = np.zeros((lq, Hq, 1))
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
        for t in range(lq):
            n = min(lk, lk - lq + t + 1)
            if n <= 0:
                continue
            a = scale * (kh[:n] @ q[t, h])
            p = np.exp(a - a.max())
            p /= p.sum()
            o[t, h], ao[t, h] = p @ vh[:n], p @ np.abs(vh[:n])
            big[t, h] = abs(scale) * (np.abs(kh[:n]) @ np.abs(q[t, h])).max()
    return o, ao, big
