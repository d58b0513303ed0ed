"""FP64 oracle of linear attention with a fixed decay for each head and of the
norms of queries and keys with the position rotation (TEST INFRASTRUCTURE ONLY).

Everything is written token by token from the definitions, in numpy and 64 bits.
Next to a result stands what bounds its rounding: for the attention the same sum
over absolute values (an upper bound of every partial sum's size), for the norms
the bound itself, in units of U = 2^-24, the relative rounding of one FP32
operation.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
CHUNK = 64


def clamp_alpha(alpha):
    a = np.asarray(alpha, dtype=np.float64)
    return np.clip(np.where(np.isnan(a), 2.0 ** -15, a), 2.0 ** -15, 1.0)


def spans(B, T, cu):
    """(batch row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(lo), int(hi)) for lo, hi in zip(cu[:-1], cu[1:])]


def attn(q, k, v, alpha, initial_state=None, cu=None):
    """o [B, T, H, dv] and the final states [N, H, dk, dv].  S <- a S + k v^T; o = S^T q."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    a = clamp_alpha(alpha)[:, None, None]
    B, T, H, dk = q.shape
    where = spans(B, T, cu)
    last = np.zeros((len(where), H, dk, v.shape[-1])) if initial_state is None else np.array(initial_state, dtype=np.float64)
    o = np.zeros(v.shape)
    for n, (b, lo, hi) in enumerate(where):
        S = last[n]
        for t in range(lo, hi):
            S = a * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = np.einsum("hkv,hk->hv", S, q[b, t])
        last[n] = S
    return o, last


def attn_grads(q, k, v, alpha, d_o, initial_state=None, d_final_state=None, cu=None):
    """Gradients of <d_o, o> + <d_final_state, final_state>: dq_t = S_t d_o_t, and with R the gradient of the
    state, R_t = q_t d_o_t^T + a R_{t+1}: dk_t = R_t v_t, dv_t = R_t^T k_t, d_initial_state = a R_0."""
    q, k, v, d_o = (np.asarray(x, dtype=np.float64) for x in (q, k, v, d_o))
    a = clamp_alpha(alpha)[:, None, None]
    B, T, H, dk = q.shape
    where = spans(B, T, cu)
    shape = (len(where), H, dk, v.shape[-1])
    start = np.zeros(shape) if initial_state is None else np.asarray(initial_state, dtype=np.float64)
    first = np.zeros(shape) if d_final_state is None else np.array(d_final_state, dtype=np.float64)
    dq, dk_, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for n, (b, lo, hi) in enumerate(where):
        S = start[n]
        for t in range(lo, hi):
            S = a * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            dq[b, t] = np.einsum("hkv,hv->hk", S, d_o[b, t])
        R = first[n]
        for t in range(hi - 1, lo - 1, -1):
            R = R + q[b, t][:, :, None] * d_o[b, t][:, None, :]
            dk_[b, t] = np.einsum("hkv,hv->hk", R, v[b, t])
            dv[b, t] = np.einsum("hkv,hk->hv", R, k[b, t])
            R = a * R
        first[n] = R
    return {"dq": dq, "dk": dk_, "dv": dv, "d_initial_state": first}


def pairs(rot, interleaved):
    """Channels of the two members of every pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(n, positions, inv_freq, interleaved, sign):
    """n [B, T, heads, d] turned by sign * position * frequency."""
    y = n.copy()
    if inv_freq is None or not len(inv_freq):
        return y
    one, two = pairs(2 * len(inv_freq), interleaved)
    angle = np.asarray(positions, dtype=np.float64)[..., None, None] * np.asarray(inv_freq, dtype=np.float64) * sign
    c, s = np.cos(angle), np.sin(angle)
    y[..., one] = n[..., one] * c - n[..., two] * s
    y[..., two] = n[..., two] * c + n[..., one] * s
    return y


def _spread(n, inv_freq, interleaved):
    """What rounding can touch of each output channel: its pair's absolute values together."""
    y = np.abs(n)
    if inv_freq is None or not len(inv_freq):
        return y
    one, two = pairs(2 * len(inv_freq), interleaved)
    both = y[..., one] + y[..., two]
    y[..., one] = both
    y[..., two] = both
    return y


# Roundings of a row's norm: a sum of up to 128 squares (8 a lane, four exchanges) halved by the root, the
# root's own two units, the mean's scaling, eps.  A cosine or sine is off by at most 10 units absolutely: two for
# the reduced turn (half a unit of a turn below a half, times 2 pi), eight for the function and its range.
NORM, ANGLE = 16, 10


def norm_rope(x, weight, scale, positions, inv_freq, eps, interleaved):
    """(value, FP32 bound) of scale * rotate(x / rms(x) * weight)."""
    x = np.asarray(x, dtype=np.float64)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, dtype=np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w * scale
    return _turn(n, positions, inv_freq, interleaved, 1.0), (NORM + ANGLE + 8) * U * _spread(n, inv_freq, interleaved)


def norm_rope_grads(x, weight, scale, positions, inv_freq, eps, interleaved, dy):
    """(dx, bound) and (d_weight, bound): xh = x / rms, dn = turned-back scale dy; d_weight = sum dn xh;
    dx = (dn w - xh mean(dn w xh)) / rms."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64) * scale
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, dtype=np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dn = _turn(dy, positions, inv_freq, interleaved, -1.0)
    size = _spread(dy, inv_freq, interleaved)
    t = dn * w
    dx = r * (t - xh * (t * xh).mean(-1, keepdims=True))
    tsize = size * np.abs(w)
    units = 2 * NORM + ANGLE + 30
    b = units * U * r * (tsize + np.abs(xh) * (tsize * np.abs(xh)).mean(-1, keepdims=True))
    rows = dy[..., 0].size
    dw = (dn * xh).reshape(-1, x.shape[-1]).sum(0)
    bw = (units + rows) * U * (size * np.abs(xh)).reshape(-1, x.shape[-1]).sum(0)
    return (dx, b), (dw, bw)
