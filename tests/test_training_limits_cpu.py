"""Limits that the training operators' C ABI checks, on a machine without a GPU."""
import pytest

from test_abi_cpu import SHAPE, lib  # noqa: F401
from test_training_cpu import BWD, EPI, FWD, call


@pytest.mark.parametrize("eps", [2.0 ** -127, 1e-40, 1e-45, -1.0])
def test_rejects_an_eps_below_the_normal_numbers(lib, eps):  # noqa: F811
    """The reciprocal square root of a subnormal number is infinity on the device: a row of zeros would be NaN."""
    for f, args in ((lib.gdn2_block_norm_fwd, FWD), (lib.gdn2_block_norm_bwd, BWD), (lib.gdn2_mixer_epilogue_bwd, EPI)):
        assert call(f, list(args), args, dict(eps=eps)) == SHAPE
