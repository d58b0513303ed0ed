"""Outputs and gradients of linear attention with a fixed decay for each head are those of FP32 arithmetic, rounded
once to their type (needs an MI355X).

Inside, bf16 calls hold what is a factor again in two bf16 terms, the first cut off or rounded and the second rounded:
off by at most 2^-16.  Those are the products inside a chunk, the copy of the state that outputs read, and, where the
caller takes no state, the factor of the state's update (in the walks and in the launch for segments' carries).  An
output's two parts take one or two of them: with A the sum over absolute values, less than 3 x 2^-16 A beside half a
step of the output's own type and the FP32 sums (test_gpu_linear.py).  In relative L2 a rounding is at most
2^-8 / sqrt(3)."""
import numpy as np
import pytest

import gpu_util as G
from delta_rule_linear_gdn2_amd import binding
from delta_rule_linear_gdn2_amd import workloads as W
from oracle import linear as L
from test_gpu_linear import HALF, U, Case, dev, gpu  # noqa: F401

pytestmark = pytest.mark.gpu
ONCE = {"f32": 1e-6, "bf16": 2.0 ** -8 / 3 ** 0.5}


def outputs(c, states, **kw):
    import torch

    how = dict(initial_state=c.t_s0, cu_seqlens=c.t_cu, **kw)
    o, s = binding.gdn2_linear_attn_fwd(**c.t, output_final_state=states, **how)
    g = binding.gdn2_linear_attn_bwd(**c.t, d_o=c.t_do, d_final_state=c.t_ds, output_d_initial_state=states, **how)
    torch.cuda.synchronize()
    assert (s is not None) == states and (g.pop("d_initial_state") is not None) == states
    return {"o": o, **g}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("B,T,dk,dv,cu", [(2, 150, 32, 32, None), (1, 1100, 32, 64, None), (1, 1100, 64, 32, None), (1, 1300, 64, 64, None),
                                          (1, 1100, 128, 64, None), (1, 1100, 64, 128, None), (1, 1300, 128, 128, None),
                                          (1, 1100, 128, 32, None), (1, 1100, 32, 128, None),
                                          (1, 1500, 64, 64, [0, 0, 700, 701, 1500]), (1, 1500, 128, 32, [0, 100, 1490, 1500])])
def test_against_the_oracle(B, T, dk, dv, cu, state, dtype):
    """With and without the states in and out, in segments and in one piece."""
    c = Case(1000 + T + dk, B, T, 2, dk, dv, dtype, cu=cu, state=state, alpha=[0.998, 0.9])
    args, size = (c.q, c.k, c.v, c.alpha), [np.abs(x) for x in (c.q, c.k, c.v)]
    absolute = lambda x: None if x is None else np.abs(x)  # noqa: E731
    want = {"o": L.attn(*args, c.s0, c.cu)[0], **L.attn_grads(*args, c.d_o, c.s0, c.ds, c.cu)}
    most = {"o": L.attn(*size, c.alpha, absolute(c.s0), c.cu)[0],
            **L.attn_grads(*size, c.alpha, np.abs(c.d_o), absolute(c.s0), absolute(c.ds), c.cu)}
    for segmented in (True, False):
        if segmented and T > 1000:
            for query in (binding.gdn2_linear_attn_fwd_workspace_bytes, binding.gdn2_linear_attn_bwd_workspace_bytes):
                assert query(B, T, 2, dk, dv, 0 if cu is None else len(cu) - 1, int(dtype == "bf16")) > 0
        for states in (True, False):
            for name, x in outputs(c, states, segmented=segmented).items():
                x, ref = G.f64(x), want[name]
                inside = 200 * c.chunks * U * most[name] + (3 * 2.0 ** -16 * most[name] if dtype == "bf16" else 0)
                bad = ~(np.abs(x - ref) <= inside + HALF[dtype] * (np.abs(ref) + inside) + 1e-37)
                assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}"
                G.assert_rel(x, ref, ONCE[dtype], f"{dtype} {dk}x{dv} {name}")


@pytest.mark.parametrize("segmented", [True, False])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 64), (64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
def test_single_products(dk, dv, segmented):
    """A state of one product, read by one product: what an output may be off by is half a step of its own type and
    2^-14 for the two-term factors and the products between them.  A factor of one term would be off by half a step
    more, cut off by a whole one."""
    r = np.random.default_rng(1100 + dk + dv)
    B, T, H = 1, 1400, 2
    alpha = np.array([0.9997, 0.9989], dtype=np.float32)

    def full(shape):
        return W.round_bf16((r.uniform(1, 2, shape) * np.exp2(r.integers(-2, 3, shape))).astype(np.float32))

    def lone(shape):  # one channel a row
        x = np.zeros(shape, dtype=np.float32)
        np.put_along_axis(x, r.integers(0, shape[-1], (*shape[:-1], 1)), full((*shape[:-1], 1)), -1)
        return x

    half = 2.0 ** -8 + 2.0 ** -14

    def close(got, ref, what):
        x = G.f64(got)
        off = np.abs(x - ref) - half * np.abs(ref)
        assert (off <= 1e-30).all(), f"{what}: off by {np.nanmax(np.abs(x - ref) / np.abs(ref)) * 256:.3f} half steps"

    # what enters the state enters it at one token, at the front of a chunk or in its middle
    for at in (0, 30, 64, 200):
        k, q, v, d_o = np.zeros((B, T, H, dk), dtype=np.float32), lone((B, T, H, dk)), full((B, T, H, dv)), lone((B, T, H, dv))
        k[:, at] = full((B, H, dk))
        t = [dev(x, "bf16") for x in (q, k, v)] + [dev(alpha)]
        close(binding.gdn2_linear_attn_fwd(*t, output_final_state=False, segmented=segmented)[0], L.attn(q, k, v, alpha)[0], f"o from {at}")
        got = binding.gdn2_linear_attn_bwd(*t, dev(d_o, "bf16"), segmented=segmented)
        close(got["dq"], L.attn_grads(q, k, v, alpha, d_o)["dq"], f"dq from {at}")
        # backwards: one token's q and d_o
        late = T - 1 - at
        q, k, v, d_o = np.zeros((B, T, H, dk), dtype=np.float32), lone((B, T, H, dk)), lone((B, T, H, dv)), np.zeros((B, T, H, dv), dtype=np.float32)
        q[:, late], d_o[:, late] = full((B, H, dk)), full((B, H, dv))
        got = binding.gdn2_linear_attn_bwd(*[dev(x, "bf16") for x in (q, k, v)], dev(alpha), dev(d_o, "bf16"), segmented=segmented)
        ref = L.attn_grads(q, k, v, alpha, d_o)
        close(got["dk"], ref["dk"], f"dk from {late}")
        close(got["dv"], ref["dv"], f"dv from {late}")
