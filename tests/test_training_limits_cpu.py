"""Limits that the training operators' C ABI checks, on a machine without a GPU."""
import pytest

import test_training_cpu
from test_abi_cpu import SHAPE, fake, lib  # noqa: F401
from test_training_cpu import BWD, EPI, FWD, PRO, call


@pytest.mark.parametrize("eps", [2.0 ** -127, 1e-40, 1e-45, -1.0])
def test_rejects_an_eps_below_the_normal_numbers(lib, eps):  # noqa: F811
    """The reciprocal square root of a subnormal number is infinity on the device: a row of zeros would be NaN."""
    for f, args in ((lib.gdn2_block_norm_fwd, FWD), (lib.gdn2_block_norm_bwd, BWD), (lib.gdn2_mixer_epilogue_bwd, EPI)):
        assert call(f, list(args), args, dict(eps=eps)) == SHAPE


@pytest.mark.parametrize("rows", [1, 1000, 1 << 20, 1 << 30])
def test_block_workspace_stays_under_its_documented_bound(lib, rows):  # noqa: F811
    """At most 1024 partial rows of 3 x D sums at every width (rounded up to 256 bytes), as the header says."""
    most = 0
    for D in range(1, 16385):
        n = lib.gdn2_block_norm_bwd_workspace_bytes(rows, D)
        assert 0 < n <= (1024 * 3 * D * 4 + 255) // 256 * 256, D
        most = max(most, n / (3 * D * 4))
    assert most >= min(1000, rows)  # the bound is no larger than it has to be


def test_rejects_prologues_past_64_bits(lib):  # noqa: F811
    """Sizes whose products overflow: refused, and a workspace of none."""
    big = (1 << 31) - 1
    for B, T, H in ((big, big, 1 << 20), (big, big, 1), (1 << 20, 1 << 20, 2), (1 << 20, big, 1 << 20)):
        assert call(lib.gdn2_mixer_prologue_bwd, list(PRO), PRO, dict(B=B, T=T, H=H, ws=None, ws_bytes=0)) == SHAPE
        assert lib.gdn2_mixer_prologue_bwd_workspace_bytes(B, T, H, 64, 64, 4) == 0
    packed = dict(B=1, cu=fake(40), num_seqs=big, H=1 << 20)
    assert call(lib.gdn2_mixer_prologue_bwd, list(PRO), PRO, packed) == SHAPE
    n = lib.gdn2_mixer_prologue_bwd_workspace_bytes(1 << 10, 1 << 20, 1 << 10, 64, 64, 4)  # the most tokens times heads
    assert n > 1 << 40


@pytest.mark.parametrize("kw,expected", test_training_cpu.test_mixer_prologue_bwd_rejects.pytestmark[0].args[1])
def test_mixer_prologue_bwd_zeroed_rejects(lib, kw, expected):  # noqa: F811
    """The checks of gdn2_mixer_prologue_bwd."""
    assert call(lib.gdn2_mixer_prologue_bwd_zeroed, list(PRO), PRO, kw) == expected
