"""Calls of linear attention with a fixed decay for each head, its step, and the q, k norm with rotation at the ends of
what their documentation allows (needs an MI355X)."""
import numpy as np
import pytest

import gpu_util as G
from delta_rule_linear_gdn2_amd import binding
from oracle import linear as L
from test_gpu_linear import BAR, Case, dev, gpu, rnd  # noqa: F401
from test_gpu_qk_rope import EPS, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,dk,dv,cu", [(150, 64, 64, None), (1300, 128, 64, None), (1300, 32, 32, [0, 3, 1100, 1300])])
@pytest.mark.parametrize("into,back,first", [(True, False, False), (True, False, True), (False, True, False),
                                             (False, True, True), (False, False, True), (True, True, False)])
def test_states_given_one_by_one(into, back, first, T, dk, dv, cu, dtype):
    """An initial state, a final state's gradient and a wanted initial state's gradient, each with and without the others."""
    c = Case(1200 + T + dk, 1, T, 2, dk, dv, dtype, cu=cu, alpha=[0.99, 0.9])
    s0, ds = (c.s0 if into else None), (c.ds if back else None)
    args = (c.q, c.k, c.v, c.alpha)
    want = L.attn_grads(*args, c.d_o, s0, ds, c.cu)
    got = binding.gdn2_linear_attn_bwd(**c.t, d_o=c.t_do, initial_state=c.t_s0 if into else None,
                                       d_final_state=c.t_ds if back else None, output_d_initial_state=first, cu_seqlens=c.t_cu)
    assert (got["d_initial_state"] is not None) == first
    for n, x in got.items():
        if x is not None:
            G.assert_rel(G.f64(x), want[n], 1e-6 if n == "d_initial_state" else BAR[dtype], f"{n} {into} {back}")
    for kept in (True, False):
        o, s = binding.gdn2_linear_attn_fwd(**c.t, initial_state=c.t_s0 if into else None, output_final_state=kept, cu_seqlens=c.t_cu)
        ro, rs = L.attn(*args, s0, c.cu)
        G.assert_rel(G.f64(o), ro, BAR[dtype], f"o {into} {kept}")
        assert (s is not None) == kept
        if kept:
            G.assert_rel(G.f64(s), rs, 1e-6, f"final state {into}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_that_are_no_numbers(dtype):
    """Clamped like any other: NaN and what is below 2^-15 to it, what is above 1 to 1."""
    c = Case(1250, 2, 130, 4, 64, 32, dtype, alpha=[float("nan"), float("inf"), -1.0, float("-inf")])
    c.check(f"{dtype} alpha that is no number")
    row = {n: c.t[n][:, 0].contiguous() for n in ("q", "k", "v")}
    state = c.t_s0.clone()
    binding.gdn2_linear_attn_step(**row, alpha=c.t["alpha"], state=state)
    G.assert_rel(G.f64(state), L.attn(c.q[:, :1], c.k[:, :1], c.v[:, :1], c.alpha, c.s0)[1], 1e-6, "step")


@pytest.mark.parametrize("dtype,d", [("f32", 128), ("bf16", 32)])
def test_the_most_heads(dtype, d):
    """2^15 heads: rows 16 MiB apart, a chunk of them 1 GiB."""
    import torch

    H, T = 1 << 15, 70
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    q, k, v, d_o = (torch.randn((1, T, H, d), generator=g, device="cuda").mul_(s).to(dt) for s in (d ** -0.5, 1.0, 1.0, 1.0))
    alpha = torch.full((H,), 0.97, device="cuda")
    o, s = binding.gdn2_linear_attn_fwd(q, k, v, alpha)
    got = binding.gdn2_linear_attn_bwd(q, k, v, alpha, d_o)
    torch.cuda.synchronize()
    for h in (0, 12345, H - 1):
        f = [G.f64(x[:, :, h:h + 1]) for x in (q, k, v, d_o)]
        ro, rs = L.attn(*f[:3], [np.float32(0.97)])
        G.assert_rel(G.f64(o[:, :, h:h + 1]), ro, BAR[dtype], f"o of head {h}")
        G.assert_rel(G.f64(s[:, h:h + 1]), rs, 1e-6, f"state of head {h}")
        want = L.attn_grads(*f[:3], [np.float32(0.97)], f[3])
        for n in ("dq", "dk", "dv"):
            G.assert_rel(G.f64(got[n][:, :, h:h + 1]), want[n], BAR[dtype], f"{n} of head {h}")


def test_step_past_32_bits():
    """States of more than 2^32 elements: the last sequence's."""
    import torch

    N, H, d = 16400, 16, 128
    assert N * H * d * d > 1 << 32
    r = np.random.default_rng(1270)
    q, k, v = (rnd(r, (1, 1, H, d), "f32") for _ in range(3))
    s0, alpha = rnd(r, (1, H, d, d), "f32"), r.uniform(0.5, 1, H).astype(np.float32)
    state = torch.zeros((N, H, d, d), device="cuda")
    state[-1] = dev(s0)[0]
    t = [torch.zeros((N, H, d), device="cuda") for _ in range(3)]
    for x, y in zip(t, (q, k, v)):
        x[-1] = dev(y)[0, 0]
    o = binding.gdn2_linear_attn_step(*t, dev(alpha), state)
    ro, rs = L.attn(q, k, v, alpha, s0)
    G.assert_rel(G.f64(state[-1:]), rs, 1e-6, "state")
    G.assert_rel(G.f64(o[-1]), ro[0, 0], 1e-6, "o")
    assert not o[:-1].any() and not any(state[i:i + 1000].any() for i in range(0, N - 1000, 1000))


def test_norm_of_the_most_heads():
    r = np.random.default_rng(1280)
    B, T, Hq, Hk, d = 1, 3, 1 << 15, 1, 32
    x = {"q": rnd(r, (B, T, Hq, d), "f32", 2.0), "k": rnd(r, (B, T, Hk, d), "f32", 0.5)}
    dy = {n: rnd(r, v.shape, "f32") for n, v in x.items()}
    w = (1 + 0.3 * r.standard_normal(d)).astype(np.float32)
    freq = (1e4 ** (-np.arange(0, d, 2) / d)).astype(np.float32)
    pos = np.array([[5, 1 << 20, -7]], dtype=np.int32)
    how = dict(inv_freq=dev(freq), positions=binding.torch.from_numpy(pos).cuda(), weight_q=dev(w))
    got = dict(zip("qk", binding.gdn2_qk_norm_rope(dev(x["q"]), dev(x["k"]), **how)))
    back = binding.gdn2_qk_norm_rope_bwd(dev(x["q"]), dev(x["k"]), dev(dy["q"]), dev(dy["k"]), **how)
    for n in "qk":
        args = (x[n], w if n == "q" else None, 1.0, pos, freq, EPS, False)
        close(got[n], L.norm_rope(*args), "f32", n)
        dx, dw = L.norm_rope_grads(*args, dy[n])
        close(back["d_" + n], dx, "f32", "d_" + n)
        if n == "q":
            close(back["d_weight_q"], dw, "f32", "d_weight_q")
    assert back["d_weight_k"] is None
