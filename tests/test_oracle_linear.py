"""Pins of the oracle of linear attention with a fixed decay and of the q, k norm
with rotation (oracle/linear.py), CPU only: the attention against the gated delta
rule's oracle without erase gate and against the closed sum, the rotation against
complex numbers, every gradient against central differences of the forward form."""
import numpy as np
import pytest

import oracle
from oracle import linear as L

CU = np.array([0, 3, 3, 10, 13], dtype=np.int32)


def _inputs(seed, B=1, T=13, H=2, dk=4, dv=3, N=4):
    r = np.random.default_rng(seed)
    return dict(q=r.standard_normal((B, T, H, dk)), k=r.standard_normal((B, T, H, dk)), v=r.standard_normal((B, T, H, dv)),
                alpha=np.array([0.9, 0.3][:H]), initial_state=r.standard_normal((N, H, dk, dv)))


def test_closed_sum():
    x = _inputs(1, B=2, N=2)
    o, S = L.attn(**x)
    a = x["alpha"]
    T = 13
    for h in range(2):
        D = np.tril(a[h] ** (np.arange(T)[:, None] - np.arange(T)))
        for b in range(2):
            q, k, v, S0 = x["q"][b, :, h], x["k"][b, :, h], x["v"][b, :, h], x["initial_state"][b, h]
            ref = (D * (q @ k.T)) @ v + (a[h] ** (np.arange(T) + 1))[:, None] * (q @ S0)
            np.testing.assert_allclose(o[b, :, h], ref, rtol=1e-11, atol=1e-12)
            end = a[h] ** T * S0 + (k * (a[h] ** (T - 1 - np.arange(T)))[:, None]).T @ v
            np.testing.assert_allclose(S[b, h], end, rtol=1e-11, atol=1e-12)


def test_is_the_delta_rule_without_erase():
    r = np.random.default_rng(2)
    B, T, H, d = 2, 40, 3, 32
    q, k, v = (r.standard_normal((B, T, H, d)) for _ in range(3))
    S0 = r.standard_normal((B, H, d, d))
    alpha = np.array([1.0, 0.875, 2.0 ** -15])
    wide = np.broadcast_to(alpha[:, None], (B, T, H, d))
    f = [np.ascontiguousarray(x.astype(np.float32)) for x in (q, k, v, wide, np.zeros_like(q), np.ones_like(v))]
    ro, rs = oracle.recurrent(*f, S0.astype(np.float32))
    o, s = L.attn(f[0], f[1], f[2], alpha, S0.astype(np.float32))
    np.testing.assert_allclose(o, ro, rtol=1e-9, atol=1e-10)
    np.testing.assert_allclose(s, rs, rtol=1e-9, atol=1e-10)


def test_packed_is_each_sequence_alone():
    x = _inputs(3)
    o, S = L.attn(**x, cu=CU)
    for n, (lo, hi) in enumerate(zip(CU[:-1], CU[1:])):
        part, end = L.attn(x["q"][:, lo:hi], x["k"][:, lo:hi], x["v"][:, lo:hi], x["alpha"], x["initial_state"][n:n + 1])
        np.testing.assert_array_equal(o[:, lo:hi], part)
        np.testing.assert_array_equal(S[n:n + 1], end)


def test_alpha_is_clamped():
    np.testing.assert_array_equal(L.clamp_alpha([0.0, 2.0, np.nan, 0.5]), [2.0 ** -15, 1.0, 2.0 ** -15, 0.5])


def _differences(f, x, g):
    """Central differences of f along every element of x against the gradient g."""
    h = 1e-5
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        down = f()
        x[i] = old
        assert abs((up - down) / (2 * h) - g[i]) <= 1e-7 * max(1.0, abs(g[i])), i


@pytest.mark.parametrize("name", ["q", "k", "v", "initial_state"])
@pytest.mark.parametrize("cu", [None, CU])
def test_attention_gradients_by_differences(name, cu):
    x = _inputs(4, N=1 if cu is None else 4)
    r = np.random.default_rng(5)
    d_o, dS = r.standard_normal(x["v"].shape), r.standard_normal(x["initial_state"].shape)

    def loss():
        o, S = L.attn(**x, cu=cu)
        return (o * d_o).sum() + (S * dS).sum()

    g = L.attn_grads(**{k: v for k, v in x.items() if k != "initial_state"}, d_o=d_o, initial_state=x["initial_state"],
                     d_final_state=dS, cu=cu)
    _differences(loss, x[name], g["d_initial_state" if name == "initial_state" else "d" + name])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 8, 16])
def test_rotation_is_complex_multiplication(interleaved, rot):
    r = np.random.default_rng(6)
    x, w = r.standard_normal((2, 5, 3, 16)), r.standard_normal(16)
    pos, freq = r.integers(0, 1 << 20, (2, 5)), r.random(rot // 2).astype(np.float32)
    y, _ = L.norm_rope(x, w, 0.5, pos, freq, 1e-6, interleaved)
    n = 0.5 * w * x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6)
    one, two = L.pairs(rot, interleaved)
    z = (n[..., one] + 1j * n[..., two]) * np.exp(1j * pos[..., None, None] * freq.astype(np.float64))
    np.testing.assert_allclose(y[..., one], z.real, atol=1e-9)
    np.testing.assert_allclose(y[..., two], z.imag, atol=1e-9)
    np.testing.assert_allclose(y[..., rot:], n[..., rot:], rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradients_by_differences(interleaved):
    r = np.random.default_rng(7)
    x, w, dy = r.standard_normal((1, 3, 2, 16)), 1 + 0.3 * r.standard_normal(16), r.standard_normal((1, 3, 2, 16))
    pos, freq = r.integers(0, 50, (1, 3)), r.random(4)

    def loss():
        return (L.norm_rope(x, w, 0.7, pos, freq, 1e-6, interleaved)[0] * dy).sum()

    (dx, _), (dw, _) = L.norm_rope_grads(x, w, 0.7, pos, freq, 1e-6, interleaved, dy)
    _differences(loss, x, dx)
    _differences(loss, w, dw)
