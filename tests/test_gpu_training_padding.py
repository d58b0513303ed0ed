"""Packed sequences in a longer buffer: gradients of the tokens that no sequence owns, through the Python
call (needs an MI355X)."""
import numpy as np
import pytest

from test_gpu_training import Prologue, dev_int, gpu  # noqa: F401
from delta_rule_linear_gdn2_amd import binding

pytestmark = pytest.mark.gpu


def padded(p, lead, tail):
    """The call's tensors with NaN tokens in front of and behind the packed sequences."""
    import torch

    out = []
    for z in p.t:
        if z.dim() == 4:
            nan = lambda n: torch.full((1, n, *z.shape[2:]), float("nan"), dtype=z.dtype, device="cuda")  # noqa: E731
            z = torch.cat([nan(lead), z, nan(tail)], 1)
        out.append(z)
    return out


@pytest.mark.parametrize("lead,tail", [(0, 77), (9, 0), (200, 1), (1, 500)])
@pytest.mark.parametrize("K", [1, 4, 7])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_padding_are_zero(dtype, K, lead, tail):
    """Whatever the allocator hands out (here blocks that held NaN), tokens without a sequence have a zero gradient,
    and the others' are those of the sequences alone."""
    import torch

    lens = [5, 0, 130, 33]
    p = Prologue(900 + K, 1, 0, 3, 64, 32, K, dtype, lens=lens)
    ref, T = p.run(), sum(lens)
    t = padded(p, lead, tail)
    held = [torch.full_like(z, float("nan")) for z in t for _ in range(2)]
    torch.cuda.synchronize()
    del held
    how = {**p.how, "cu_seqlens": dev_int(p.cu + np.int32(lead))}
    got = binding.gdn2_mixer_prologue_bwd(*t, **how)
    for name in ("d_xq", "d_xk", "d_xv", "d_b_logit", "d_w_logit"):
        assert torch.equal(got[name][:, lead:lead + T], ref[name]), name
        assert not got[name][:, :lead].any() and not got[name][:, lead + T:].any(), name
    assert torch.equal(got["d_conv_state"], ref["d_conv_state"])


def test_gradients_without_any_sequence():
    """Only padding, in an even number of ways: every gradient is zero, the carried state's passes through."""
    import torch

    p = Prologue(910, 1, 0, 2, 32, 32, 4, "bf16", lens=[60])
    t = padded(p, 0, 0)
    for cu in ([0, 0, 0], [60, 60, 60], [17, 17, 17]):
        st = torch.randn((2, 2 * 96, 3), device="cuda")
        held = [torch.full_like(z, float("nan")) for z in t for _ in range(2)]
        torch.cuda.synchronize()
        del held
        got = binding.gdn2_mixer_prologue_bwd(*t, conv_state=st, d_conv_state_out=st, output_d_conv_state=True,
                                              cu_seqlens=dev_int(np.array(cu, dtype=np.int32)))
        assert torch.equal(got.pop("d_conv_state"), st)
        for name, v in got.items():
            assert not v.any(), (cu, name)
