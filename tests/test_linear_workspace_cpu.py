"""Workspaces of linear attention with a fixed decay for each head, on a machine without a GPU (plans for 256 compute
units): their size goes by the segments whose carries are kept."""
import pytest

from delta_rule_linear_gdn2_amd import binding
from test_abi_cpu import lib  # noqa: F401


@pytest.mark.parametrize("dtype,least", [(1, 4 * 64), (0, 2 * 64)])  # a segment's least length
@pytest.mark.parametrize("T,H,dk,dv", [(32768, 16, 128, 128), (4096, 2, 64, 32), (700, 1, 32, 32)])
def test_packed_goes_by_the_segments(lib, T, H, dk, dv, dtype, least):  # noqa: F811
    """Of sequences, segments and a carry each, only sequences longer than a segment have any."""
    state = 4 * H * dk * dv
    for N in (1, 3, 100, 1000, 5000, 1 << 20):
        fwd = binding.gdn2_linear_attn_fwd_workspace_bytes(1, T, H, dk, dv, N, dtype)
        bwd = binding.gdn2_linear_attn_bwd_workspace_bytes(1, T, H, dk, dv, N, dtype)
        assert fwd <= 2 * (T // least) * state and bwd <= 4 * (T // least) * state, N
        assert fwd % 256 == 0 and bwd % 512 == 0
    many, few = (binding.gdn2_linear_attn_fwd_workspace_bytes(1, 32768, 16, 128, 128, n, 1) for n in (5000, 7))
    assert many == few > 0


def test_smaller_calls_may_need_more(lib):  # noqa: F811
    """Each call's own query counts: a workspace of the larger call's size is refused where the smaller one needs more."""
    from test_linear_cpu import BWD, FWD, call
    from test_abi_cpu import WS

    fwd, bwd = binding.gdn2_linear_attn_fwd_workspace_bytes, binding.gdn2_linear_attn_bwd_workspace_bytes
    assert fwd(64, 4096, 4, 64, 64, 0, 1) == bwd(64, 4096, 4, 64, 64, 0, 1) == 0
    for query, name, sizes in ((fwd, "gdn2_linear_attn_fwd", FWD), (bwd, "gdn2_linear_attn_bwd", BWD)):
        need = query(1, 4096, 4, 64, 64, 0, 1)
        assert need > 0
        assert call(getattr(lib, name), list(sizes), sizes, dict(ws_bytes=need - 1)) == WS
