"""Gradients of the norms at the ends of the FP32 range (needs an MI355X): rows far
larger and far smaller than one, and rows of zeros with a small eps.  The cube of
1 / rms leaves FP32 range there although the gradient does not.

Bars: the FP64 oracle's own (oracle/training.py), which are relative to the terms
of each formula and so the same at every scale.  Scales are powers of two, which
bf16 and FP32 inputs take exactly."""
import numpy as np
import pytest

from delta_rule_linear_gdn2_amd import binding
from delta_rule_linear_gdn2_amd import workloads as W
from oracle import training as O
from test_gpu_training import TYPES, Block, Prologue, close, dev, gpu, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


def f32(x):
    return float(np.float32(x))


def block_grads(b, x, u, eps):
    """The block's gradients for the stream x and the block output u, without a gradient of the stream that would
    hide the norm's; and the oracle's."""
    got = binding.gdn2_block_norm_bwd(dev(x, b.res), dev(u, b.dtype), None, b.t["d_h"], **{**b.how, "eps": eps})
    want = O.block_norm_grads(x, u, None, b.d_h, w_pre=b.w_pre, **{**b.oracle, "eps": f32(eps)})
    return got, want


@pytest.mark.parametrize("x_log2,u_log2,eps", [(40, 0, 1e-5), (45, 0, 1e-5), (50, 0, 1e-5), (0, 45, 1e-5), (0, 50, 1e-5),
                                               (25, 55, 1e-5), (-40, 0, 1e-30), (0, -40, 1e-30), (-50, 3, 1e-36)])
@pytest.mark.parametrize("dtype,res", TYPES)
def test_block_gradients_at_any_scale(dtype, res, x_log2, u_log2, eps):
    for D in (7, 96, 333, 1371, 2048):
        b = Block(800 + D, 11, D, dtype, res, "full", "silu", p=0.2)
        got, want = block_grads(b, b.x * np.float32(2.0 ** x_log2), b.u * np.float32(2.0 ** u_log2), eps)
        for name, ref in want.items():
            close(got[name], ref, f"block {dtype}/{res} D={D} x 2^{x_log2} u 2^{u_log2} eps {eps} {name}")


@pytest.mark.parametrize("eps", [1e-5, 1e-20, 1e-30, 1e-36])
@pytest.mark.parametrize("dtype,res", TYPES)
def test_block_gradients_of_rows_of_zeros(dtype, res, eps):
    """rms = sqrt(eps): the gradients are those of a product with 1 / sqrt(eps)."""
    for D in (5, 64, 1001):
        b = Block(810 + D, 6, D, dtype, res, "none", p=0.0)
        for x, u in ((0 * b.x, b.u), (b.x, 0 * b.u)):
            got, want = block_grads(b, x, u, eps)
            for name, ref in want.items():
                close(got[name], ref, f"block {dtype}/{res} D={D} zeros eps {eps} {name}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("log2,eps", [(40, 1e-5), (50, 1e-5), (-45, 1e-30), (None, 1e-30)])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_epilogue_gradients_at_any_scale(dtype, log2, eps, dv):
    """log2 None: rows of zeros."""
    rng = np.random.default_rng(820 + dv)
    o, gate, dy = (rnd(rng, (37, dv), dtype) for _ in range(3))
    o = o * np.float32(0.0 if log2 is None else 2.0 ** log2)
    w = rnd(rng, (dv,), "f32", 0.2, 1.0)
    got = binding.gdn2_mixer_epilogue_bwd(dev(o, dtype), dev(gate, dtype), dev(w), dev(dy, dtype), eps=eps, act="silu")
    for name, ref in O.epilogue_grads(o, gate, w, dy, f32(eps), "silu").items():
        close(got[name], ref, f"epilogue bwd {dtype} dv={dv} 2^{log2} {name}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 4, 7])
def test_prologue_gradients_of_small_heads(dtype, K):
    """eps_l2 = 0 and inputs near 2^-46."""
    p = Prologue(830 + K, 2, 21, 2, 32, 64, K, dtype, state=False)
    p.x = [x * np.float32(2.0 ** -46) for x in p.x]
    p.t[:3] = [dev(x, dtype) for x in p.x]
    got = p.run(eps_l2=0.0)
    want = O.prologue_grads(*p.x, *p.conv, *p.logit, *p.d, None, None, None, 0.125, 0.0)
    for name, ref in want.items():
        close(got[name], ref, f"prologue bwd {dtype} K={K} small {name}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 4, 7])
def test_prologue_gradients_of_large_heads(dtype, K):
    """Positive inputs from 64 on under positive filters: the sigmoid is one in FP32, SiLU the identity, and with
    eps_l2 = 0 q and k do not depend on the inputs' scale.  So 2^44 times the inputs has 2^-44 times the input gradient
    of q and k, and the same gradients of their filters; the oracle gives those at scale one."""
    p = Prologue(840 + K, 2, 21, 2, 32, 64, K, dtype, state=False)
    p.x = [64 + np.minimum(np.abs(x), 4) * np.float32(16) for x in p.x]
    if dtype == "bf16":
        p.x = [W.round_bf16(x) for x in p.x]
    p.conv = [0.5 + np.minimum(np.abs(w), 1) for w in p.conv]
    scale = 2.0 ** 44
    p.t[:6] = [dev(x * np.float32(scale), dtype) for x in p.x] + [dev(w) for w in p.conv]
    got = p.run(eps_l2=0.0)
    want = O.prologue_grads(*p.x, *p.conv, *p.logit, *p.d, None, None, None, 0.125, 0.0)
    for name in ("d_xq", "d_xk"):
        close(got[name].double().mul(scale).float() if dtype == "f32" else got[name] * scale, want[name],
              f"prologue bwd {dtype} K={K} large {name}")
    for name in ("d_conv_q", "d_conv_k"):
        close(got[name], want[name], f"prologue bwd {dtype} K={K} large {name}")
