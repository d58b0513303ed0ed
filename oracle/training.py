"""FP64 oracle of the training operators around the recurrence (TEST INFRASTRUCTURE ONLY).

The step from one block of a layer to the next (norms, gate, residual scale,
dropout) and its gradients, and the gradients of the token mixer's prologue and
epilogue, in numpy and 64 bits.  Next to each result stands a bound on what an
FP32 evaluation of the same formula may be off, carried through the formula
term by term; the tests add the rounding of the output's type to it.

Units: U = 2^-24 is the relative rounding of one FP32 operation.
  * A row's sum of D terms runs over at most 16 terms a lane, six lane
    exchanges and 16 wavefronts: under 40 roundings of its absolute terms.
  * The hardware's exp2, reciprocal and reciprocal square root are within one
    unit in the last place (2 U).  exp(x) multiplies by log2 e first, which adds
    2 |x| U; a sigmoid is therefore within (5 + 2 |x|) U, and with |x| <= 8, as
    in the tests, within 21 U.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


# --- dropout -----------------------------------------------------------------


def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon, Moraes, Dror and Shaw, "Parallel Random Numbers: As
    Easy as 1, 2, 3", 2011): counter [..., 4] and key [2] of 32-bit words ->
    [..., 4] words.  A round multiplies words 0 and 2 by a constant each; the
    high halves, XORed with the other words and the key, go to words 0 and 2
    crosswise and the low halves to words 1 and 3; the key is bumped a round."""
    c = [np.asarray(counter, dtype=np.uint64)[..., i] for i in range(4)]
    mask = np.uint64(0xFFFFFFFF)
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        m0, m1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(m1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), m1 & mask,
             (m0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), m0 & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1).astype(np.uint32)


def threshold(p):
    return int(np.floor(p * 65536 + 0.5))


def kept(rows, D, p, seed, offset, first_row=0):
    """Which elements of [rows, D] (from row first_row on) are kept, one element at a time in meaning:
    block = row * ceil(D / 8) + d / 8, half-word d % 8 of the block's output."""
    g = (D + 7) // 8
    block = (np.arange(first_row, first_row + rows, dtype=np.uint64)[:, None] * np.uint64(g)
             + (np.arange(D, dtype=np.uint64) // np.uint64(8))[None, :])
    ctr = np.stack([block & np.uint64(0xFFFFFFFF), block >> np.uint64(32),
                    np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)], axis=-1)
    words = philox4x32(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    j = np.arange(D) % 8
    word = np.take_along_axis(words, np.broadcast_to((j // 2)[None, :, None], (rows, D, 1)), axis=-1)[..., 0]
    half = np.where(j % 2 == 1, word >> np.uint32(16), word & np.uint32(0xFFFF))
    return half >= threshold(p)


def dropout(x, p, seed, offset, first_row=0):
    """Dropped elements are zero whatever they hold; the others are divided by 1 - p."""
    x = _f64(x)
    t = threshold(p)
    keep = kept(x.shape[0], x.shape[1], p, seed, offset, first_row)
    return np.where(keep, x * (65536.0 / (65536 - t) if t < 65536 else 0.0), 0.0)


# --- the step from one block to the next -------------------------------------


def act(g, kind):
    """Value and derivative of a gate's activation."""
    if kind == "identity":
        return g, np.ones_like(g)
    s = 1.0 / (1.0 + np.exp(-g))
    return (s, s * (1 - s)) if kind == "sigmoid" else (g * s, s * (1 + g * (1 - s)))


def _act_size(g, kind):
    """Sizes that the errors of value and derivative are relative to."""
    if kind == "identity":
        return np.abs(g), np.ones_like(g)
    s = 1.0 / (1.0 + np.exp(-g))
    return (s, s) if kind == "sigmoid" else (np.abs(g) * s, s * (1 + np.abs(g)))


def _rrms(z, eps):
    return 1.0 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)


def _branch(u, gate, layout, gate_act, w_post, eps):
    """n, act(gate), act'(gate), the sizes of the last two, 1 / rms(u)."""
    r = _rrms(u, eps) if w_post is not None else np.ones((u.shape[0], 1))
    n = u * r * w_post if w_post is not None else u
    if layout == "none":
        one = np.ones((1, 1))
        return n, one, 0 * one, one, one, r
    g = gate[:, None] if layout == "token" else gate
    return (n, *act(g, gate_act), *_act_size(g, gate_act), r)


def block_norm_x(x, u, *, gate=None, layout="none", gate_act="sigmoid", w_post=None, eps=1e-5, scale=1.0, p=0.0, seed=0,
                 offset=0):
    """x_out before its rounding, and its FP32 error bound (the last sum's rounding, and 64 U of the branch:
    20 for the norm's root, 21 for the gate, its products, the scale and the dropout factor)."""
    x, u, gate, w_post = _f64(x), _f64(u), _f64(gate), _f64(w_post)
    n, a, _, sa, _, _ = _branch(u, gate, layout, gate_act, w_post, eps)
    m = dropout(np.ones_like(x), p, seed, offset)
    z = np.where(m > 0, scale * m * a * n, 0.0)  # a dropped element is gone, whatever it held
    return x + z, U * np.abs(x + z) + 64 * U * np.where(m > 0, np.abs(scale) * m * sa * np.abs(n), 0.0)


def block_norm_h(x_out, w_pre, eps=1e-5):
    """The norm of the stored stream, and its error bound."""
    x_out, w_pre = _f64(x_out), _f64(w_pre)
    h = x_out * _rrms(x_out, eps) * w_pre
    return h, 32 * U * np.abs(h)


def block_norm_grads(x_out, u, d_x_out, d_h, *, gate=None, layout="none", gate_act="sigmoid", w_post=None, w_pre=None,
                     eps=1e-5, scale=1.0, p=0.0, seed=0, offset=0):
    """Gradients of the step, {name: (value, FP32 error bound)}.

    The stream's gradient t is within 64 U of the sum T of its absolute terms;
    the branch's factors add 40 for the norm, 21 (64 for the derivative) for
    the gate and a few products, so its gradients stay within 320 U of theirs.
    A sum over the rows adds one rounding a row."""
    x_out, u, d_h, gate, w_post, w_pre = (_f64(v) for v in (x_out, u, d_h, gate, w_post, w_pre))
    shape = (x_out if x_out is not None else u).shape
    rows, D = shape
    out = {}
    t = np.zeros(shape) if d_x_out is None else _f64(d_x_out)
    T = np.abs(t)
    if w_pre is not None:
        r = _rrms(x_out, eps)
        wd = w_pre * d_h
        t = t + r * wd - x_out * r ** 3 * (wd * x_out).mean(-1, keepdims=True)
        T = T + r * np.abs(wd) + np.abs(x_out) * r ** 3 * np.abs(wd * x_out).mean(-1, keepdims=True)
        out["d_weight_pre"] = ((d_h * x_out * r).sum(0), (64 + rows) * U * np.abs(d_h * x_out * r).sum(0))
    out["d_x"] = (t, 64 * U * T)
    if u is None:
        return out
    m = dropout(np.ones(shape), p, seed, offset)
    n, a, da, sa, sda, r = _branch(u, gate, layout, gate_act, w_post, eps)
    c, C = np.where(m > 0, scale * m * t, 0.0), np.where(m > 0, np.abs(scale) * m * T, 0.0)
    if layout != "none":
        dg, G = da * c * n, 320 * U * sda * C * np.abs(n)
        if layout == "token":
            dg, G = dg.sum(1), G.sum(1)
        if layout == "channel":
            dg, G = dg.sum(0), G.sum(0) * (320 + rows) / 320
        out["d_gate"] = (dg, G)
    dn, N = c * a, C * sa
    if w_post is None:
        out["d_u"] = (dn, 320 * U * N)
        return out
    out["d_weight_post"] = ((dn * u * r).sum(0), (320 + rows) * U * (N * np.abs(u) * r).sum(0))
    wd, W = w_post * dn, np.abs(w_post) * N
    out["d_u"] = (r * wd - u * r ** 3 * (wd * u).mean(-1, keepdims=True),
                  320 * U * (r * W + np.abs(u) * r ** 3 * (W * np.abs(u)).mean(-1, keepdims=True)))
    return out


# --- the token mixer ---------------------------------------------------------


def epilogue_grads(o, gate, weight, d_y, eps=1e-5, gate_act="sigmoid"):
    """Gradients of the mixer epilogue: the block's branch with scale 1 and no dropout."""
    g = block_norm_grads(None, o, d_y, None, gate=gate, layout="full", gate_act=gate_act, w_post=weight, eps=eps)
    return {"d_o": g["d_u"], "d_gate": g["d_gate"], "d_weight": g["d_weight_post"]}


def _path_grads(x, w, state, dout, d_state_out, kind, scale, eps_l2):
    """One sequence of one convolution path.  x, dout [L, H, d]; w [H d, K]; state, d_state_out [H d, K - 1]
    or None.  Returns dx, dw, dstate, each with its FP32 error bound."""
    L, H, d = x.shape
    C, K = w.shape
    line = np.concatenate([np.zeros((K - 1, C)) if state is None else state.T, x.reshape(L, C)])
    win = np.stack([line[i:i + L] for i in range(K)], axis=-1)                     # [L, C, K]
    y, ey = (win * w).sum(-1), (K + 1) * U * np.abs(win * w).sum(-1)
    s = 1.0 / (1.0 + np.exp(-y))
    v = y * s
    ev = 1.1 * ey + 24 * U * np.abs(v)                                              # |SiLU'| <= 1.1
    g = dout.reshape(L, C)
    if kind == "v":
        dv, edv = g, np.zeros_like(g)
    else:
        V, G, E = (z.reshape(L, H, d) for z in (v, g, ev))
        r = 1.0 / np.sqrt((V * V).sum(-1, keepdims=True) + eps_l2)
        S, Sa = (V * G).sum(-1, keepdims=True), np.abs(V * G).sum(-1, keepdims=True)
        dv = scale * r * (G - V * r * r * S)
        # 64 U of the terms, and what the error of v does to first order: |dv_c| changes by at most
        # s r^2 (|g_c| + 4 r |v_c| |g|) |dv| + s r^2 |g| |dv_c|, as |v| <= 1 / r
        nE, nG = np.sqrt((E * E).sum(-1, keepdims=True)), np.sqrt((G * G).sum(-1, keepdims=True))
        edv = scale * (64 * U * r * (np.abs(G) + np.abs(V) * r * r * Sa)
                       + r * r * ((np.abs(G) + 4 * r * np.abs(V) * nG) * nE + nG * E))
        dv, edv = dv.reshape(L, C), edv.reshape(L, C)
    ds = s * (1 + y * (1 - s))
    dy = dv * ds
    edy = edv * 1.1 + np.abs(dv) * (64 * U * s * (1 + np.abs(y)) + 0.5 * ey) + 2 * U * np.abs(dy)  # |SiLU''| <= 1/2
    dline, eline = np.zeros((L + K - 1, C)), np.zeros((L + K - 1, C))
    for i in range(K):
        dline[i:i + L] += w[:, i] * dy
        eline[i:i + L] += np.abs(w[:, i]) * (edy + (K + 2) * U * np.abs(dy))
    if d_state_out is not None:
        dline[L:] += d_state_out.T
        eline[L:] += 2 * U * np.abs(d_state_out.T)
    dw = (dy[:, :, None] * win).sum(0)
    edw = (np.abs(win) * (edy + (L + 16) * U * np.abs(dy))[:, :, None]).sum(0)
    return (dline[K - 1:].reshape(L, H, d), eline[K - 1:].reshape(L, H, d)), (dw, edw), (dline[:K - 1].T, eline[:K - 1].T)


def prologue_grads(xq, xk, xv, conv_q, conv_k, conv_v, b_logit, w_logit, d_q, d_k, d_v, d_b, d_w, cu_seqlens=None,
                   conv_state=None, d_conv_state_out=None, q_scale=1.0, eps_l2=1e-6):
    """Gradients of the mixer prologue, {name: (value, FP32 error bound)}, d_conv_state included."""
    B, T = np.shape(xq)[:2]
    bounds = [(n, 0, T) for n in range(B)] if cu_seqlens is None else [
        (0, int(a), int(b)) for a, b in zip(cu_seqlens[:-1], cu_seqlens[1:])]
    out, states, chan = {}, [], 0
    for kind, x, w, dout in (("q", xq, conv_q, d_q), ("k", xk, conv_k, d_k), ("v", xv, conv_v, d_v)):
        x, w, dout = _f64(x), _f64(w), _f64(dout)
        C, K = w.shape
        dx, dw = [np.zeros_like(x), np.zeros_like(x)], [np.zeros_like(w), np.zeros_like(w)]
        st = [np.zeros((len(bounds), C, K - 1)), np.zeros((len(bounds), C, K - 1))]
        for n, (row, lo, hi) in enumerate(bounds):
            part = lambda s: None if s is None else _f64(s)[n, chan:chan + C]  # noqa: E731
            got = _path_grads(x[row, lo:hi], w, part(conv_state), dout[row, lo:hi], part(d_conv_state_out), kind,
                              q_scale if kind == "q" else 1.0, eps_l2)
            for i in range(2):
                dx[i][row, lo:hi] = got[0][i]
                dw[i] += got[1][i]
                st[i][n] = got[2][i]
        # the sequences' filter gradients are summed too
        out["d_x" + kind], out["d_conv_" + kind] = tuple(dx), (dw[0], dw[1] + B * T * U * np.abs(dw[0]))
        states.append(st)
        chan += C
    for kind, logit, d in (("b", b_logit, d_b), ("w", w_logit, d_w)):
        s = 1.0 / (1.0 + np.exp(-_f64(logit)))
        out[f"d_{kind}_logit"] = (_f64(d) * s * (1 - s), 64 * U * np.abs(_f64(d)) * s)
    out["d_conv_state"] = tuple(np.concatenate([st[i] for st in states], axis=1) for i in range(2))
    return out
