"""fp64 oracle of the training-step operators beside the linear layers:
attention and its gradient, the per-head norm and rotation of queries and
keys and its gradient, and the distillation loss on a teacher's top logits
with its gradient.

Plain numpy from the definitions, one head (or row) at a time; test
infrastructure only, sharing no code with the package.
"""

from __future__ import annotations

import numpy as np


def _sequences(cu, tokens):
    if cu is None:
        return [(0, tokens)]
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def attention(q, k, v, causal, scale, cu_q=None, cu_k=None):
    """q [tokens, heads, d], k, v [key tokens, key heads, d] -> (o, lse [heads,
    tokens], w) with w = sum_j P_ij |v_j| (what a rounding of P is measured
    by). Rows outside every sequence are 0, -inf and 0."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    group = q.shape[1] // k.shape[1]
    o, w = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((q.shape[1], q.shape[0]), -np.inf)
    for (q0, q1), (k0, k1) in zip(_sequences(cu_q, q.shape[0]), _sequences(cu_k, k.shape[0])):
        for h in range(q.shape[1]):
            p, z = _probabilities(q[q0:q1, h], k[k0:k1, h // group], causal, scale)
            lse[h, q0:q1] = z
            o[q0:q1, h] = p @ v[k0:k1, h // group]
            w[q0:q1, h] = p @ np.abs(v[k0:k1, h // group])
    return o, lse, w


def _probabilities(q, k, causal, scale):
    """Softmax rows (all 0 where the mask leaves nothing) and log-sum-exps."""
    lq, lk = len(q), len(k)
    s = scale * (q @ k.T)
    seen = np.ones((lq, lk), dtype=bool)
    if causal:
        seen = np.arange(lk)[None] <= np.arange(lq)[:, None] + (lk - lq)
    p = np.zeros((lq, lk))
    z = np.full(lq, -np.inf)
    for i in range(lq):
        if seen[i].any():
            top = s[i, seen[i]].max()
            e = np.exp(s[i, seen[i]] - top)
            z[i] = top + np.log(e.sum())
            p[i, seen[i]] = e / e.sum()
    return p, z


def attention_backward(q, k, v, do, causal, scale, cu_q=None, cu_k=None):
    """(dq, dk, dv) and, for each, how far it moves when every P, dS and O
    that enters it moves by one part of itself: sums of magnitudes."""
    q, k, v, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, do))
    group = q.shape[1] // k.shape[1]
    grads = [np.zeros_like(x) for x in (q, k, v)]
    sizes = [np.zeros_like(x) for x in (q, k, v)]
    for (q0, q1), (k0, k1) in zip(_sequences(cu_q, q.shape[0]), _sequences(cu_k, k.shape[0])):
        for h in range(q.shape[1]):
            g = h // group
            qh, kh, vh, dh = q[q0:q1, h], k[k0:k1, g], v[k0:k1, g], do[q0:q1, h]
            p, _ = _probabilities(qh, kh, causal, scale)
            o = p @ vh
            delta = (dh * o).sum(axis=1, keepdims=True)
            ds = p * (dh @ vh.T - delta)
            # a rounding of dS, and one of O within delta
            moved = np.abs(ds) + p * (np.abs(dh) * np.abs(o)).sum(axis=1, keepdims=True)
            grads[0][q0:q1, h] = scale * (ds @ kh)
            grads[1][k0:k1, g] += scale * (ds.T @ qh)
            grads[2][k0:k1, g] += p.T @ dh
            sizes[0][q0:q1, h] = scale * (moved @ np.abs(kh))
            sizes[1][k0:k1, g] += scale * (moved.T @ np.abs(qh))
            sizes[2][k0:k1, g] += p.T @ np.abs(dh)
    return grads, sizes


def _turn(x, cos, sin, interleaved):
    """x [..., d] with the pairs of its first 2 len(cos) entries turned."""
    y = x.copy()
    r = 2 * cos.shape[-1]
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def qk_norm_rope(x, wq, wk, cos, sin, pos, heads_q, heads_kv, eps, interleaved):
    """x [tokens, (heads_q + 2 heads_kv) d] -> q, k, v [tokens, heads, d]."""
    x = np.asarray(x, dtype=np.float64)
    x = x.reshape(len(x), heads_q + 2 * heads_kv, -1)
    c, s = (np.asarray(t, dtype=np.float64)[pos][:, None] for t in (cos, sin))
    out = []
    for lo, hi, w in ((0, heads_q, wq), (heads_q, heads_q + heads_kv, wk)):
        part = x[:, lo:hi]
        n = part / np.sqrt((part ** 2).mean(axis=-1, keepdims=True) + eps)
        out.append(_turn(n * np.asarray(w, dtype=np.float64), c, s, interleaved))
    return out[0], out[1], x[:, heads_q + heads_kv:].copy()


def qk_norm_rope_backward(x, wq, wk, cos, sin, pos, dq, dk, dv, eps, interleaved):
    """(dx, dwq, dwk) of qk_norm_rope."""
    heads_q, heads_kv = dq.shape[1], dk.shape[1]
    x = np.asarray(x, dtype=np.float64)
    x = x.reshape(len(x), heads_q + 2 * heads_kv, -1)
    c, s = (np.asarray(t, dtype=np.float64)[pos][:, None] for t in (cos, sin))
    dx, dw = [], []
    for lo, hi, w, dy in ((0, heads_q, wq, dq), (heads_q, heads_q + heads_kv, wk, dk)):
        part, w = x[:, lo:hi], np.asarray(w, dtype=np.float64)
        r = 1.0 / np.sqrt((part ** 2).mean(axis=-1, keepdims=True) + eps)
        dn = _turn(np.asarray(dy, dtype=np.float64), c, -s, interleaved)
        dw.append((dn * part * r).sum(axis=(0, 1)))
        g = dn * w
        dx.append(r * g - part * r ** 3 * (g * part).mean(axis=-1, keepdims=True))
    dx.append(np.asarray(dv, dtype=np.float64))
    return np.concatenate(dx, axis=1).reshape(len(x), -1), dw[0], dw[1]


def distill_topk(logits, ids, teacher, tau, inv_norm):
    """losses [M] = tau^2 KL(p || q) and dlogits = tau (q - p) inv_norm: p the
    softmax of the row's teacher logits / tau over its listed entries (id in
    [0, V); the others are empty places), q the softmax of the logits / tau
    over all V. A row without entries gives 0."""
    z = np.asarray(logits, dtype=np.float64) / tau
    t = np.asarray(teacher, dtype=np.float64) / tau
    m, v = z.shape
    losses, dz = np.zeros(m), np.zeros((m, v))
    for i in range(m):
        has = (ids[i] >= 0) & (ids[i] < v)
        if not has.any():
            continue
        e = np.exp(t[i, has] - t[i, has].max())
        log_p = t[i, has] - t[i, has].max() - np.log(e.sum())
        p = e / e.sum()
        top = z[i].max()
        total = np.exp(z[i] - top).sum()
        log_q = z[i] - top - np.log(total)
        losses[i] = tau ** 2 * (p * (log_p - log_q[ids[i][has]])).sum()
        dz[i] = np.exp(log_q)
        np.subtract.at(dz[i], ids[i][has], p)
        dz[i] *= tau * inv_norm
    return losses, dz
