"""Dropped elements are gone in the backward pass too, whatever they held (needs an MI355X)."""
import numpy as np
import pytest

from delta_rule_linear_gdn2_amd import binding
from oracle import training as O
from test_gpu_training import TYPES, Block, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

BAD = (float("nan"), float("inf"), float("-inf"))


@pytest.mark.parametrize("layout,act", [("none", "identity"), ("channel", "silu"), ("token", "sigmoid"),
                                        ("full", "identity"), ("full", "sigmoid"), ("full", "silu")])
@pytest.mark.parametrize("dtype,res", TYPES)
def test_values_at_dropped_elements_reach_no_gradient(dtype, res, layout, act):
    """Without a norm of the block's output its elements are apart: NaN and infinity where the mask drops them leave
    every output as it is with ordinary values there, bit for bit."""
    import torch

    for D in (5, 96, 333, 1371, 2050):
        b = Block(870 + D, 12, D, dtype, res, layout, act, post=False, p=0.5)
        x_out, h = b.fwd()
        ref = b.bwd(x_out)
        drop = torch.from_numpy(~O.kept(12, D, 0.5, **b.rand)).cuda()
        for bad in BAD:
            b.t["u"][drop] = bad
            y, h2 = b.fwd()
            assert torch.equal(y, x_out) and torch.equal(h2, h)
            for name, v in b.bwd(x_out).items():
                assert v is None or torch.equal(v, ref[name]), f"D={D} u {bad}: {name}"


@pytest.mark.parametrize("act", ["identity", "sigmoid", "silu"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("dtype,res", TYPES)
def test_gates_at_dropped_elements_reach_no_gradient(dtype, res, post, act):
    """A full gate's values at dropped elements, with and without the norm of the block's output."""
    import torch

    for D in (5, 96, 333, 1371, 2050):
        b = Block(880 + D, 12, D, dtype, res, "full", act, post=post, p=0.5)
        x_out, h = b.fwd()
        ref = b.bwd(x_out)
        drop = torch.from_numpy(~O.kept(12, D, 0.5, **b.rand)).cuda()
        assert not ref["d_gate"][drop].any()
        for bad in BAD:
            b.t["gate"][drop] = bad
            y, h2 = b.fwd()
            assert torch.equal(y, x_out) and torch.equal(h2, h)
            for name, v in b.bwd(x_out).items():
                assert v is None or torch.equal(v, ref[name]), f"D={D} gate {bad}: {name}"


def test_everything_dropped():
    """p = 1: the block's output and gate may hold anything."""
    import torch

    b = Block(890, 7, 264, "bf16", "f32", "full", "silu", post=False, p=1.0)
    b.t["u"].fill_(float("nan"))
    b.t["gate"].fill_(float("inf"))
    x_out, _ = b.fwd()
    assert torch.equal(x_out, b.t["x"])
    got = b.bwd(x_out)
    assert not got["d_u"].any() and not got["d_gate"].any() and np.isfinite(got["d_x"].float().cpu().numpy()).all()
