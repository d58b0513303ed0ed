"""Pins of the training operators' oracle (oracle/training.py), CPU only: the
generator against published outputs, the forward formulas against the library
routines of torch, every gradient against central differences of the forward
oracles."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import mixer, training


@pytest.mark.parametrize("counter,key,out", [
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_philox_known_answers(counter, key, out):
    """The known answers that the generator's authors publish for ten rounds."""
    assert training.philox4x32(np.array(counter), key).tolist() == out


def test_mask_is_positional_and_its_share_is_p():
    a = training.kept(64, 21, 0.3, 5, 9)
    np.testing.assert_array_equal(a[10:20], training.kept(10, 21, 0.3, 5, 9, first_row=10))
    assert not np.array_equal(a, training.kept(64, 21, 0.3, 5, 10))
    assert not np.array_equal(a, training.kept(64, 21, 0.3, 6, 9))
    big = training.kept(512, 512, 0.3, 1, 0)
    # share of dropped elements: the standard deviation is sqrt(0.21) / 512 = 9e-4
    assert abs((~big).mean() - 0.3) < 5e-3
    assert training.kept(3, 5, 0.0, 1, 0).all() and not training.kept(3, 5, 1.0, 1, 0).any()


def test_dropout_of_dropped_infinities_is_zero():
    x = np.full((4, 16), np.inf)
    y = training.dropout(x, 0.5, 3, 0)
    assert set(np.unique(y)) == {0.0, np.inf}


def _rng(seed):
    return np.random.default_rng(seed)


def _block(seed, rows=3, D=10, layout="full", post=True, pre=True):
    r = _rng(seed)
    shape = {"none": None, "channel": (D,), "token": (rows,), "full": (rows, D)}[layout]
    return dict(x=r.standard_normal((rows, D)), u=r.standard_normal((rows, D)),
                gate=None if shape is None else r.standard_normal(shape),
                w_post=1 + 0.2 * r.standard_normal(D) if post else None,
                w_pre=1 + 0.2 * r.standard_normal(D) if pre else None)


def test_block_forward_matches_torch():
    b = _block(1)
    x_out, _ = training.block_norm_x(b["x"], b["u"], gate=b["gate"], layout="full", gate_act="silu", w_post=b["w_post"],
                                     scale=0.7)
    t = {k: torch.from_numpy(v) for k, v in b.items()}
    ref = t["x"] + 0.7 * F.silu(t["gate"]) * F.rms_norm(t["u"], (10,), t["w_post"], eps=1e-5)
    np.testing.assert_allclose(x_out, ref.numpy(), rtol=1e-12)
    h, _ = training.block_norm_h(x_out, b["w_pre"])
    np.testing.assert_allclose(h, F.rms_norm(ref, (10,), t["w_pre"], eps=1e-5).numpy(), rtol=1e-12)


def _difference(f, z, step=1e-5):
    """Central differences of the scalar f in every entry of z."""
    d = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        keep = z[i]
        z[i] = keep + step
        hi = f()
        z[i] = keep - step
        lo = f()
        z[i] = keep
        d[i] = (hi - lo) / (2 * step)
    return d


@pytest.mark.parametrize("layout,gate_act", [("none", "identity"), ("channel", "identity"), ("channel", "silu"),
                                             ("token", "sigmoid"), ("full", "sigmoid"), ("full", "silu")])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_block_gradients_match_differences(layout, gate_act, post, pre):
    b = _block(2, layout=layout, post=post, pre=pre)
    how = dict(gate=b["gate"], layout=layout, gate_act=gate_act, w_post=b["w_post"], scale=0.6, p=0.3, seed=11, offset=2)
    r = _rng(3)
    dx_out, dh = r.standard_normal((3, 10)), r.standard_normal((3, 10)) if pre else None

    def loss():
        x_out, _ = training.block_norm_x(b["x"], b["u"], **how)
        return (x_out * dx_out).sum() + ((training.block_norm_h(x_out, b["w_pre"])[0] * dh).sum() if pre else 0.0)

    x_out, _ = training.block_norm_x(b["x"], b["u"], **how)
    g = training.block_norm_grads(x_out, b["u"], dx_out, dh, w_pre=b["w_pre"], **how)
    for name, z in (("d_x", b["x"]), ("d_u", b["u"]), ("d_gate", b["gate"]), ("d_weight_post", b["w_post"]),
                    ("d_weight_pre", b["w_pre"])):
        assert (name in g) == (z is not None)
        if z is not None:
            np.testing.assert_allclose(g[name][0], _difference(loss, z), rtol=1e-6, atol=1e-8, err_msg=name)


def test_norm_alone_gradients_match_differences():
    b = _block(4)
    dx_out, dh = _rng(5).standard_normal((2, 3, 10))
    g = training.block_norm_grads(b["x"], None, dx_out, dh, w_pre=b["w_pre"])
    loss = lambda: (b["x"] * dx_out).sum() + (training.block_norm_h(b["x"], b["w_pre"])[0] * dh).sum()  # noqa: E731
    np.testing.assert_allclose(g["d_x"][0], _difference(loss, b["x"]), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(g["d_weight_pre"][0], _difference(loss, b["w_pre"]), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_epilogue_gradients_match_differences(act):
    r = _rng(6)
    o, gate, dy, w = r.standard_normal((3, 6)), r.standard_normal((3, 6)), r.standard_normal((3, 6)), r.standard_normal(6)
    loss = lambda: (mixer.epilogue(o, gate, w, act=act) * dy).sum()  # noqa: E731
    g = training.epilogue_grads(o, gate, w, dy, gate_act=act)
    for name, z in (("d_o", o), ("d_gate", gate), ("d_weight", w)):
        np.testing.assert_allclose(g[name][0], _difference(loss, z), rtol=1e-6, atol=1e-8, err_msg=name)


@pytest.mark.parametrize("K", [1, 2, 4])
@pytest.mark.parametrize("packed", [False, True])
def test_prologue_gradients_match_differences(K, packed):
    r = _rng(7 + K)
    B, T, H, dk, dv = (1, 7, 2, 3, 2) if packed else (2, 4, 2, 3, 2)
    cu = np.array([0, 1, 1, 3, 7]) if packed else None  # one token, none, two, four
    N = 4 if packed else B
    z = dict(xq=r.standard_normal((B, T, H, dk)), xk=r.standard_normal((B, T, H, dk)), xv=r.standard_normal((B, T, H, dv)),
             conv_q=r.standard_normal((H * dk, K)), conv_k=r.standard_normal((H * dk, K)),
             conv_v=r.standard_normal((H * dv, K)), b_logit=r.standard_normal((B, T, H, dk)),
             w_logit=r.standard_normal((B, T, H, dv)))
    state = r.standard_normal((N, H * (2 * dk + dv), K - 1))
    d = {n: r.standard_normal((B, T, H, w)) for n, w in (("q", dk), ("k", dk), ("v", dv), ("b", dk), ("w", dv))}
    d_state = r.standard_normal(state.shape)

    def loss():
        o = mixer.prologue(*z.values(), cu, state, q_scale=0.4)
        return sum((o[n] * d[n]).sum() for n in d) + (o["conv_state"] * d_state).sum()

    g = training.prologue_grads(*z.values(), d["q"], d["k"], d["v"], d["b"], d["w"], cu, state, d_state, q_scale=0.4)
    for name in ("xq", "xk", "xv", "conv_q", "conv_k", "conv_v", "b_logit", "w_logit"):
        np.testing.assert_allclose(g["d_" + name][0], _difference(loss, z[name]), rtol=1e-6, atol=1e-7, err_msg=name)
    if K > 1:
        np.testing.assert_allclose(g["d_conv_state"][0], _difference(loss, state), rtol=1e-6, atol=1e-7)
