"""fp64 oracle of the operators around a block and of the optimizer's step: the
norms before and after a block with its gate and residual and their gradient,
attention with capped, biased and ranged scores and its gradient, AdamW with
states in 32 bits, and what its 8-bit states hold.

Plain numpy from the definitions; test infrastructure only, sharing no code
with the package.
"""

from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def block_norms(x, y, gate, w_post, w_pre, residual_scale, block_scale, eps):
    """(h, n) and the sizes of their terms; n is None without w_pre."""
    x, y, gate, w_post, w_pre = (_f64(t) for t in (x, y, gate, w_post, w_pre))
    h, size = residual_scale * x, np.abs(residual_scale * x)
    if y is not None:
        b = y
        if w_post is not None:
            b = w_post * y / np.sqrt((y ** 2).mean(axis=1, keepdims=True) + eps)
        b = block_scale * b * (1.0 if gate is None else gate)
        h, size = h + b, size + np.abs(b)
    if w_pre is None:
        return (h, None), (size, None)
    r = 1.0 / np.sqrt((h ** 2).mean(axis=1, keepdims=True) + eps)
    # (a change of h moves its norm too)
    moved = size + np.abs(h) * r * r * (np.abs(h) * size).mean(axis=1, keepdims=True)
    return (h, w_pre * h * r), (size, np.abs(w_pre) * moved * r)


def _norm_gradient(x, w, dn, eps, size_dn):
    """dx and dw of w x / rms(x), and the sizes of their terms where those of
    dn are size_dn."""
    r = 1.0 / np.sqrt((x ** 2).mean(axis=1, keepdims=True) + eps)
    g, gs = dn * w, size_dn * np.abs(w)
    dx = r * g - x * r ** 3 * (g * x).mean(axis=1, keepdims=True)
    size = r * gs + np.abs(x) * r ** 3 * (gs * np.abs(x)).mean(axis=1, keepdims=True)
    return dx, (dn * x * r).sum(axis=0), size, (size_dn * np.abs(x) * r).sum(axis=0)


def block_norms_backward(h, y, gate, w_post, w_pre, dh, dn, residual_scale, block_scale, eps):
    """({dx, dy, dgate, dw_post, dw_pre}, the sizes of their terms); the gate
    [width], [tokens, 1], [tokens, width] or None."""
    h, y, gate, w_post, w_pre, dh, dn = (_f64(t) for t in (h, y, gate, w_post, w_pre, dh, dn))
    like = dh if dh is not None else dn
    d, size = np.zeros_like(like), np.zeros_like(like)
    got, sizes = {}, {}
    if dh is not None:
        d, size = d + dh, size + np.abs(dh)
    if dn is not None:
        x, got["dw_pre"], s, sizes["dw_pre"] = _norm_gradient(h, w_pre, dn, eps, np.abs(dn))
        d, size = d + x, size + s
    got["dx"], sizes["dx"] = residual_scale * d, np.abs(residual_scale) * size
    if y is None:
        return got, sizes
    b = y
    if w_post is not None:
        b = w_post * y / np.sqrt((y ** 2).mean(axis=1, keepdims=True) + eps)
    d, size = block_scale * d, np.abs(block_scale) * size
    if gate is not None:
        over = 0 if gate.ndim == 1 else 1 if gate.shape[1] < y.shape[1] else None
        for to, v in ((got, d * b), (sizes, size * np.abs(b))):
            to["dgate"] = v if over is None else v.sum(axis=over, keepdims=over == 1)
        d, size = d * gate, size * np.abs(gate)
    if w_post is None:
        got["dy"], sizes["dy"] = d, size
    else:
        got["dy"], got["dw_post"], sizes["dy"], sizes["dw_post"] = _norm_gradient(y, w_post, d, eps,
                                                                                 size)
    return got, sizes


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after a step."""
    p, g, m, v = (_f64(t) for t in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    root = np.sqrt(v / (1 - beta2 ** step))
    return p - lr * (weight_decay * p + m / (1 - beta1 ** step) / (root + eps)), m, v


def adamw_states_f32(g, m, v, beta1, beta2, grad_scale=None):
    """m, v and the root of v as the formula gives them in float32, one
    rounding to an operation."""
    f = np.float32
    g, m, v = (np.asarray(t, dtype=f) for t in (g, m, v))
    if grad_scale is not None:
        g = g * f(grad_scale)
    m = m * f(beta1) + g * f(1.0 - beta1)
    v = v * f(beta2) + (g * g) * f(1.0 - beta2)
    return m, v, np.sqrt(v)


_E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                  for e in range(16) for m in range(8)])
_E4M3[127] = np.nan


def e4m3_values(codes):
    """The values of e4m3 codes (uint8)."""
    codes = np.asarray(codes)
    return np.where(codes & 128, -1.0, 1.0) * _E4M3[codes & 127]


def e4m3_codes(x):
    """The nearest codes (ties to the even one, beyond 448: 448; NaN: NaN)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_E4M3[:127], a), 1, 126)
    lo = hi - 1
    up, down = _E4M3[hi] - a, a - _E4M3[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def coded(x, least=False):
    """x (float32) in blocks of 256 as (codes, scales), each operation rounded
    to float32 by itself."""
    f = np.float32
    x = np.asarray(x, dtype=f)
    codes, scales = np.zeros(x.size, np.uint8), []
    for a in range(0, x.size, 256):
        b = x[a:a + 256]
        fine = np.isfinite(b)
        top = np.abs(b[fine]).max(initial=f(0))
        scale = top * f(1.0 / 448.0) if top >= f(2.0 ** -100) else f(0)
        inv = f(1) / scale if scale > 0 else f(0)
        c = np.where(fine, b, f(0)) * inv
        if least:
            c = np.where(c > 0, np.maximum(c, f(2.0 ** -9)), c)
        codes[a:a + 256] = np.where(fine, e4m3_codes(c), 127)
        scales.append(scale)
    return codes, np.array(scales, dtype=f)


def _scored(q, k, scale, cap, slope, first, end, causal):
    """Probabilities (0 where nothing is left), log-sum-exps and the cap's
    derivative of one head of one sequence."""
    lq, lk = len(q), len(k)
    s = scale * (q @ k.T)
    chain = np.ones_like(s)
    if cap:
        t = np.tanh(s / cap)
        s, chain = cap * t, 1.0 - t * t
    here = np.arange(lq)[:, None] + (lk - lq)
    key = np.arange(lk)[None]
    s = s - slope * np.abs(here - key)
    seen = np.ones((lq, lk), dtype=bool)
    if causal:
        seen &= key <= here
    if first is not None:
        seen &= key >= np.asarray(first)[:, None]
    if end is not None:
        seen &= key < np.asarray(end)[:, None]
    p, z = np.zeros((lq, lk)), np.full(lq, -np.inf)
    for i in np.flatnonzero(seen.any(axis=1)):
        top = s[i, seen[i]].max()
        e = np.exp(s[i, seen[i]] - top)
        z[i] = top + np.log(e.sum())
        p[i, seen[i]] = e / e.sum()
    return p, z, chain


def _cuts(cu, tokens):
    return [(0, tokens)] if cu is None else [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


def attention_scores(q, k, v, causal, scale, cap=None, slopes=None, first=None, end=None, cu_q=None,
                     cu_k=None):
    """(o, lse, w) with w = sum_j P_ij |v_j|; first and end: [tokens] of q."""
    q, k, v = (_f64(x) for x in (q, k, v))
    group = q.shape[1] // k.shape[1]
    o, w = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((q.shape[1], q.shape[0]), -np.inf)
    for (q0, q1), (k0, k1) in zip(_cuts(cu_q, q.shape[0]), _cuts(cu_k, k.shape[0])):
        for h in range(q.shape[1]):
            cut = [None if x is None else x[q0:q1] for x in (first, end)]
            p, z, _ = _scored(q[q0:q1, h], k[k0:k1, h // group], scale, cap,
                              0.0 if slopes is None else slopes[h], *cut, causal)
            lse[h, q0:q1] = z
            o[q0:q1, h] = p @ v[k0:k1, h // group]
            w[q0:q1, h] = p @ np.abs(v[k0:k1, h // group])
    return o, lse, w


def attention_scores_backward(q, k, v, do, causal, scale, cap=None, slopes=None, first=None,
                              end=None, cu_q=None, cu_k=None):
    """(dq, dk, dv) and, for each, how far it moves when every P, dS and O
    that enters it moves by one part of itself: sums of magnitudes."""
    q, k, v, do = (_f64(x) for x in (q, k, v, do))
    group = q.shape[1] // k.shape[1]
    grads = [np.zeros_like(x) for x in (q, k, v)]
    sizes = [np.zeros_like(x) for x in (q, k, v)]
    for (q0, q1), (k0, k1) in zip(_cuts(cu_q, q.shape[0]), _cuts(cu_k, k.shape[0])):
        for h in range(q.shape[1]):
            g = h // group
            qh, kh, vh, dh = q[q0:q1, h], k[k0:k1, g], v[k0:k1, g], do[q0:q1, h]
            cut = [None if x is None else x[q0:q1] for x in (first, end)]
            p, _, chain = _scored(qh, kh, scale, cap, 0.0 if slopes is None else slopes[h], *cut,
                                  causal)
            o = p @ vh
            delta = (dh * o).sum(axis=1, keepdims=True)
            ds = p * (dh @ vh.T - delta) * chain
            moved = np.abs(ds) + chain * p * (np.abs(dh) * np.abs(o)).sum(axis=1, keepdims=True)
            grads[0][q0:q1, h] = scale * (ds @ kh)
            grads[1][k0:k1, g] += scale * (ds.T @ qh)
            grads[2][k0:k1, g] += p.T @ dh
            sizes[0][q0:q1, h] = scale * (moved @ np.abs(kh))
            sizes[1][k0:k1, g] += scale * (moved.T @ np.abs(qh))
            sizes[2][k0:k1, g] += p.T @ np.abs(dh)
    return grads, sizes
