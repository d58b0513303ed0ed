"""The smallest eps that the norms take (needs an MI355X; the refusal of smaller ones is a
CPU test)."""
import numpy as np
import pytest

from delta_rule_linear_gdn2_amd import binding
from oracle import training as O
from test_gpu_training import TYPES, Block, close, dev, gpu, rnd  # noqa: F401

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -126


@pytest.mark.parametrize("dtype,res", TYPES)
def test_rows_of_zeros(dtype, res):
    """The norm of a row of zeros is zero, and its gradient the product with 1 / sqrt(eps).  Other rows as ever."""
    small = np.float32(2.0 ** -40)  # the gradients are 2^63 and 2^126 times this
    for D in (5, 64, 333, 2048):
        b = Block(850 + D, 5, D, dtype, res, "none", p=0.0, scale=1.0)
        b.x[1] = b.u[1] = b.u[3] = 0
        b.t.update(x=dev(b.x, res), u=dev(b.u, dtype))
        b.oracle["eps"] = LEAST
        x_out, h = b.fwd(eps=LEAST)
        x = x_out.double().cpu().numpy()
        close(x_out, O.block_norm_x(b.x, b.u, **b.oracle), f"x_out {dtype}/{res} D={D}")
        close(h, O.block_norm_h(x, b.w_pre, LEAST), f"h {dtype}/{res} D={D}")
        assert not h[1].any()
        got = binding.gdn2_block_norm_bwd(x_out, b.t["u"], None, b.t["d_h"] * float(small), **{**b.how, "eps": LEAST})
        want = O.block_norm_grads(x, b.u, None, b.d_h * small, w_pre=b.w_pre, **b.oracle)
        for name, ref in want.items():
            close(got[name], ref, f"{name} {dtype}/{res} D={D}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_epilogue_rows_of_zeros(dtype):
    rng = np.random.default_rng(860)
    o, gate, dy = (rnd(rng, (9, 64), dtype) for _ in range(3))
    o[[0, 4]] = 0
    w = rnd(rng, (64,), "f32", 0.2, 1.0)
    got = binding.gdn2_mixer_epilogue_bwd(dev(o, dtype), dev(gate, dtype), dev(w), dev(dy, dtype), eps=LEAST)
    for name, ref in O.epilogue_grads(o, gate, w, dy, LEAST).items():
        close(got[name], ref, f"epilogue bwd {dtype} {name}")
