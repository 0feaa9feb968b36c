"""Plain fp64 CPU oracle for the attention layer and the AdamW step.

TEST INFRASTRUCTURE ONLY.  Only the test suite, ``__graft_entry__.smoke()`` and
the CPU-baseline leg of ``bench.py`` may import this module.  The product path
(the CUDA library and its Python binding) never calls it and shares no code
with it.  Everything is evaluated from the definitions in float64, one sequence
and one head at a time; roundings of the device are tolerances of the tests.
"""
from __future__ import annotations

import numpy as np

from .model_oracle import _f64


def rope_angles(positions, inv_freq) -> np.ndarray:
    """[T, R/2] angles: position times frequency."""
    return _f64(positions)[:, None] * _f64(inv_freq)[None, :]


def rotate(y, ang, back: bool = False) -> np.ndarray:
    """Pairs (i, i + R/2) of y [T, H, D] turned by ang [T, R/2] (by -ang with ``back``)."""
    h = ang.shape[1]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1.0 if back else 1.0)
    a, b = y[..., :h], y[..., h:2 * h]
    return np.concatenate([a * c - b * s, b * c + a * s, y[..., 2 * h:]], -1)


def head_norm(x, g, eps: float):
    """(x r g, r) of x [T, H, D] with r = 1 / sqrt(mean(x^2) + eps); g None: (x, 1)."""
    X = _f64(x)
    if g is None:
        return X, np.ones(X.shape[:-1] + (1,))
    r = 1.0 / np.sqrt(np.mean(X * X, -1, keepdims=True) + eps)
    return X * r * _f64(g), r


def qk_norm_rope(x, g, positions, inv_freq, eps: float) -> np.ndarray:
    y, _ = head_norm(x, g, eps)
    return rotate(y, rope_angles(positions, inv_freq))


def qk_norm_rope_bwd(dz, x, g, positions, inv_freq, eps: float):
    """(dx, dg or None)."""
    dy = rotate(_f64(dz), rope_angles(positions, inv_freq), back=True)
    if g is None:
        return dy, None
    _, r = head_norm(x, g, eps)
    n = _f64(x) * r
    dn = dy * _f64(g)
    return r * (dn - n * np.mean(dn * n, -1, keepdims=True)), (dy * n).sum((0, 1))


def sequences(q_offsets, k_offsets=None, k_lens=None):
    """[(first query, queries, first key, keys)] of each sequence."""
    qo = [int(x) for x in q_offsets]
    ko = qo if k_offsets is None else [int(x) for x in k_offsets]
    n = [ko[i + 1] - ko[i] for i in range(len(qo) - 1)] if k_lens is None else [int(x) for x in k_lens]
    return [(qo[i], qo[i + 1] - qo[i], ko[i], n[i]) for i in range(len(qo) - 1)]


def attention(q, k, v, seqs, causal: bool, scale: float, dout=None) -> dict:
    """softmax(q k^T scale) v for q [Tq, Hq, D], k, v [Tk, Hkv, D]; query i of n sees keys
    j <= i + (keys - n) under ``causal``.  A query that sees nothing gives zeros and lse = -inf.
    Returns out, lse [Hq, Tq], and with ``dout`` the gradients and, for tolerances, the sums of
    absolute terms of each result."""
    Q, K, V = _f64(q), _f64(k), _f64(v)
    Hq, Hkv = Q.shape[1], K.shape[1]
    G = Hq // Hkv
    R = {"out": np.zeros(Q.shape), "lse": np.full((Hq, Q.shape[0]), np.nan), "out_abs": np.zeros(Q.shape),
         "s_abs": np.zeros((Hq, Q.shape[0]))}
    if dout is not None:
        G_ = _f64(dout)
        R.update(dq=np.zeros(Q.shape), dk=np.zeros(K.shape), dv=np.zeros(V.shape), dq_abs=np.zeros(Q.shape),
                 dk_abs=np.zeros(K.shape), dv_abs=np.zeros(V.shape))
    for q0, nq, k0, nk in seqs:
        for h in range(Hq):
            a, b, c = Q[q0:q0 + nq, h], K[k0:k0 + nk, h // G], V[k0:k0 + nk, h // G]
            s = a @ b.T * scale
            seen = np.ones((nq, nk), bool)
            if causal:
                seen = np.arange(nk)[None, :] <= np.arange(nq)[:, None] + (nk - nq)
            s = np.where(seen, s, -np.inf)
            m = s.max(1, initial=-np.inf)
            e = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None]), 0.0)
            z = e.sum(1)
            p = e / np.where(z > 0, z, 1.0)[:, None]
            R["out"][q0:q0 + nq, h] = p @ c
            R["out_abs"][q0:q0 + nq, h] = p @ np.abs(c)
            with np.errstate(divide="ignore"):
                R["lse"][h, q0:q0 + nq] = m + np.log(z)
            sa = np.where(seen, np.abs(a) @ np.abs(b).T * scale, 0.0)
            R["s_abs"][h, q0:q0 + nq] = sa.max(1, initial=0.0)
            if dout is not None:
                d = G_[q0:q0 + nq, h]
                dp = d @ c.T
                mean = (p * dp).sum(1, keepdims=True)
                ds = p * (dp - mean) * scale
                # every term that enters ds, whatever cancels between them
                dsa = p * (np.abs(d) @ np.abs(c).T + (p * (np.abs(d) @ np.abs(c).T)).sum(1, keepdims=True)) * scale
                R["dq"][q0:q0 + nq, h] = ds @ b
                R["dq_abs"][q0:q0 + nq, h] = dsa @ np.abs(b)
                R["dk"][k0:k0 + nk, h // G] += ds.T @ a
                R["dk_abs"][k0:k0 + nk, h // G] += dsa.T @ np.abs(a)
                R["dv"][k0:k0 + nk, h // G] += p.T @ d
                R["dv_abs"][k0:k0 + nk, h // G] += p.T @ np.abs(d)
    return R


def adamw(p, g, m, v, step: int, lr: float, beta1: float, beta2: float, eps: float, weight_decay: float,
          grad_scale: float = 1.0):
    """(p, m, v) after one step, and the update's parts for tolerances: (update, denominator)."""
    p, g, m, v = (_f64(x) for x in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v / (1 - beta2 ** step)) + eps
    u = lr / (1 - beta1 ** step) * m / den
    return p * (1 - lr * weight_decay) - u, m, v, u, den
