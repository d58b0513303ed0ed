"""The row loops of every cover and the long column sums, against the FP64 oracle (needs an MI355X).

A launch has as many workgroups as are resident at once; with more rows than they take
together each walks several, with the next row's loads in the registers that the current
one frees and two LDS buffers in turn.  The row counts here are over two such rounds of
each cover (512 workgroups of two rows up to 2048 channels, 768 up to 4096, 256 above),
and no row is zero."""
import pytest

from delta_rule_linear_gdn2_amd import binding
from test_gpu_training import TYPES, Block, Prologue, gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [33, 41, 63, 129, 203, 255])
@pytest.mark.parametrize("dtype,res", TYPES)
def test_ragged_rows_of_eight_and_thirty_two_lanes(D, dtype, res):
    Block(920 + D, 37, D, dtype, res, p=0.2).check(f"block {dtype}/{res} D={D}")


@pytest.mark.parametrize("rows,D", [(70003, 41), (18001, 203), (17001, 200), (2201, 2048), (1601, 2050), (1600, 4096),
                                    (541, 4104), (541, 5461), (540, 8192), (531, 9001), (530, 16384)])
@pytest.mark.parametrize("layout,act", [("full", "silu"), ("channel", "sigmoid")])
def test_many_rows_of_every_cover(rows, D, layout, act):
    dtype, res = TYPES[(rows + D + len(layout)) % 3]
    Block(930 + D, rows, D, dtype, res, layout, act, p=0.2).check(f"block {dtype}/{res} {rows} x {D} gate {layout}")


@pytest.mark.parametrize("rows,D", [(2201, 1371), (2200, 1376)])
def test_many_rows_of_three_wavefronts(rows, D):
    """The backward pass's own cover: 1024 workgroups."""
    for dtype, res in TYPES:
        Block(940 + D, rows, D, dtype, res, "token", "sigmoid", p=0.1).check(f"block {dtype}/{res} {rows} x {D}")


@pytest.mark.parametrize("lens", [None, [900, 0, 3, 1500, 97]])
def test_filter_gradients_over_many_runs_of_wide_calls(lens):
    """9216 columns of filter gradients over some 150 runs of tokens: the wide column sum and its loop of four."""
    p = Prologue(950, 1, 2000, 12, 32, 128, 4, "bf16", lens=lens)
    H, dk, dv, K, T = 12, 32, 128, 4, p.x[0].shape[1]
    width = H * (2 * dk + dv) * K
    partials = binding.gdn2_mixer_prologue_bwd_workspace_bytes(1, T, H, dk, dv, K) // (4 * width)
    assert width >= 8192 and partials > 100
    p.check(f"prologue bwd {partials} runs")


def test_two_streams_side_by_side_pass_by_pass():
    """Two streams run the same backward calls at once: every pass gives what the call alone gives."""
    import torch

    blocks = [Block(960 + k, 2000, 264, "bf16", "f32", "channel", "silu", p=0.3) for k in range(2)]
    outs = [b.fwd()[0] for b in blocks]
    refs = [b.bwd(x) for b, x in zip(blocks, outs)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = [[binding.gdn2_block_norm_bwd(x, b.t["u"], b.t["d_x_out"], b.t["d_h"], stream=s, **b.how)
            for b, x, s in zip(blocks, outs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for n, one in enumerate(got):
        for g, ref in zip(one, refs):
            for name, v in ref.items():
                assert torch.equal(g[name], v), f"pass {n}: {name}"


def test_every_call_by_keyword_on_a_stream():
    """The first argument by keyword, with a stream of its own: what the positional call gives."""
    import torch

    b = Block(970, 300, 264, "bf16", "f32", "full", "silu", p=0.3)
    x_out, h = b.fwd()
    ref = b.bwd(x_out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, h2 = binding.gdn2_block_norm_fwd(x=b.t["x"], u=b.t["u"], stream=s, **b.how)
    got = binding.gdn2_block_norm_bwd(x_out=y, u=b.t["u"], d_x_out=b.t["d_x_out"], d_h=b.t["d_h"], stream=s, **b.how)
    d = binding.gdn2_dropout(x=b.t["x"], p=0.3, seed=5, stream=s)
    s.synchronize()
    assert torch.equal(y, x_out) and torch.equal(h2, h) and torch.equal(d, binding.gdn2_dropout(b.t["x"], 0.3, 5))
    for name, v in ref.items():
        assert torch.equal(got[name], v), name
