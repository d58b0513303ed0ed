"""A buffer for the gate's gradient that the call would not fill is refused (CPU tensors; the binding's own checks)."""
import pytest
import torch

from delta_rule_linear_gdn2_amd import binding


def _x(*shape):
    return torch.zeros(shape)


@pytest.mark.parametrize("kw", [dict(d_gate=_x(3, 16)),                                                # no gate
                                dict(gate=_x(3, 16), gate_layout="full", d_gate=_x(3, 16), want_d_gate=False)])
def test_block_norm_bwd_refuses_a_gate_gradient_that_it_would_not_write(kw):
    with pytest.raises(ValueError, match="d_gate: there is none"):
        binding.gdn2_block_norm_bwd(_x(3, 16), _x(3, 16), _x(3, 16), None, **kw)
