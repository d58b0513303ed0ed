"""The mixer's backward in a captured graph (needs an MI355X)."""
import numpy as np
import pytest

from delta_rule_linear_gdn2_amd import binding
from test_gpu_training import Prologue, dev, gpu, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [None, [33, 0, 70, 5]])
def test_mixer_backward_in_a_replayed_graph(lens):
    """Epilogue and prologue captured once; every replay is the eager call on what the inputs hold by then, with eager
    calls between the replays."""
    import torch

    rng = np.random.default_rng(980)
    p = Prologue(981, 2, 90, 3, 64, 64, 4, "bf16", lens=lens)
    o, gate, dy = (dev(rnd(rng, (700, 64), "bf16"), "bf16") for _ in range(3))
    w = dev(rnd(rng, (64,), "f32", 0.2, 1.0))

    def both():
        return {**binding.gdn2_mixer_prologue_bwd(*p.t, **p.how), **binding.gdn2_mixer_epilogue_bwd(o, gate, w, dy, act="silu")}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        for name, v in both().items():
            assert torch.equal(got[name], v), f"replay {k}: {name}"
        for z in (o, dy, p.t[0], p.t[8]):  # other inputs for the next one
            z.mul_(-0.5)
