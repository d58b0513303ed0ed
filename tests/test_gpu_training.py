"""GPU parity of the training operators (gdn2_block_norm_fwd/_bwd, gdn2_dropout,
gdn2_mixer_epilogue_bwd, gdn2_mixer_prologue_bwd) against the FP64 oracle in
oracle/training.py (needs an MI355X).

Bar, element by element: the FP32 error bound that the oracle derives for the
formula, and half a step of the output's type (2^-8 of the value for bf16,
2^-24 for FP32).  The oracle sees exactly the values the kernels see."""
import numpy as np
import pytest

import gpu_util as G
from delta_rule_linear_gdn2_amd import binding
from delta_rule_linear_gdn2_amd import workloads as W
from oracle import training as O

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    yield


def close(got, want, what):
    """got: device tensor; want: (value, FP32 error bound)."""
    import torch

    ref, bound = want
    half = HALF_STEP["bf16" if got.dtype == torch.bfloat16 else "f32"]
    assert tuple(got.shape) == ref.shape, f"{what}: shape {tuple(got.shape)} != {ref.shape}"
    off = np.abs(G.f64(got) - ref)
    room = bound + half * (np.abs(ref) + bound) + 1e-37  # the last: flushed denormals
    bad = ~(off <= room)
    worst = float((off / room).max()) if off.size else 0.0
    G.log(f"{what}: worst error {worst:.3f} of its bound")
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}, {worst:.2f}x"


def rnd(rng, shape, dtype, scale=1.0, mean=0.0):
    x = (mean + scale * rng.standard_normal(shape)).astype(np.float32)
    return W.round_bf16(x) if dtype == "bf16" else x


def dev(x, dtype="f32"):
    return None if x is None else W.to_torch(x, dtype, "cuda")


class Block:
    """Inputs of one block step and its calls."""

    def __init__(self, seed, rows, D, dtype, res, layout="full", act="sigmoid", post=True, pre=True, p=0.0, scale=0.7):
        import torch

        rng = np.random.default_rng(seed)
        gd = "f32" if layout == "channel" else dtype
        gate = {"none": None, "channel": (D,), "token": (rows,), "full": (rows, D)}[layout]
        self.x, self.u = rnd(rng, (rows, D), res, 2.0), rnd(rng, (rows, D), dtype)
        self.gate = None if gate is None else rnd(rng, gate, gd)
        self.w_post = rnd(rng, (D,), "f32", 0.2, 1.0) if post else None
        self.w_pre = rnd(rng, (D,), "f32", 0.2, 1.0) if pre else None
        self.d_x_out, self.d_h = rnd(rng, (rows, D), res), rnd(rng, (rows, D), dtype) if pre else None
        self.dtype, self.res = dtype, res
        self.t = dict(x=dev(self.x, res), u=dev(self.u, dtype), gate=dev(self.gate, gd), w_post=dev(self.w_post),
                      w_pre=dev(self.w_pre), d_x_out=dev(self.d_x_out, res), d_h=dev(self.d_h, dtype))
        self.rand = dict(seed=0x123456789ABCDEF0 + seed, offset=(1 << 33) + 5)
        self.how = dict(gate=self.t["gate"], gate_layout=layout, gate_act=act, weight_post=self.t["w_post"],
                        weight_pre=self.t["w_pre"], residual_scale=scale, dropout_p=p, **self.rand)
        self.oracle = dict(gate=self.gate, layout=layout, gate_act=act, w_post=self.w_post, scale=float(np.float32(scale)),
                           p=p, eps=float(np.float32(1e-5)), **self.rand)
        self.torch = torch

    def fwd(self, **kw):
        out = binding.gdn2_block_norm_fwd(self.t["x"], self.t["u"], **{**self.how, **kw})
        self.torch.cuda.synchronize()
        return out

    def bwd(self, x_out, **kw):
        out = binding.gdn2_block_norm_bwd(x_out, self.t["u"], self.t["d_x_out"], self.t["d_h"], **{**self.how, **kw})
        self.torch.cuda.synchronize()
        return out

    def check(self, what):
        x_out, h = self.fwd()
        close(x_out, O.block_norm_x(self.x, self.u, **self.oracle), f"{what} x_out")
        if self.w_pre is not None:
            close(h, O.block_norm_h(G.f64(x_out), self.w_pre, self.oracle["eps"]), f"{what} h")
        else:
            assert h is None
        got = self.bwd(x_out)
        want = O.block_norm_grads(G.f64(x_out), self.u, self.d_x_out, self.d_h, w_pre=self.w_pre, **self.oracle)
        assert {k for k, v in got.items() if v is not None} == set(want)
        for name, w in want.items():
            close(got[name], w, f"{what} {name}")


TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


# every cover of a row (lane group, wavefront, several), whole groups of eight and ragged ones, a group more than a cover holds
@pytest.mark.parametrize("D", [1, 7, 8, 9, 16, 31, 32, 64, 65, 96, 200, 256, 333, 512, 1000, 1001, 1024, 1200, 1371, 1536, 2047,
                               2048, 2050, 4096, 4104, 5461, 6000, 8192, 9001, 16384])
@pytest.mark.parametrize("dtype,res", TYPES)
def test_block_widths(D, dtype, res):
    rows = 37 if D <= 2048 else 5
    Block(400 + D, rows, D, dtype, res, p=0.2).check(f"block {dtype}/{res} D={D}")


@pytest.mark.parametrize("layout,act", [("none", "identity"), ("channel", "identity"), ("channel", "silu"),
                                        ("token", "sigmoid"), ("token", "silu"), ("full", "identity"), ("full", "silu")])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_block_gates_and_norms(layout, act, post, pre):
    for n, (dtype, res) in enumerate(TYPES):
        Block(440 + n, 21, 136 if n else 91, dtype, res, layout, act, post, pre, p=0.4 * (n != 1)).check(
            f"block {dtype}/{res} gate {layout} {act} post={post} pre={pre}")


@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 1024, 3001])
def test_block_rows(rows):
    """One token, a decode batch, more rows than workgroups walk at once (32 rows of 64 channels a workgroup)."""
    Block(460 + rows, rows, 64, "bf16", "f32", "channel", "identity", p=0.1).check(f"block rows={rows} D=64")
    Block(470 + rows, rows, 520, "bf16", "bf16", "token", "silu").check(f"block rows={rows} D=520")


def test_block_many_rows_walk():
    """More rows than one round of workgroups takes: each workgroup walks several."""
    Block(480, 40003, 24, "f32", "f32", "full", p=0.5).check("block 40003 x 24")
    Block(481, 2500, 1100, "bf16", "f32", "channel", "silu", p=0.1).check("block 2500 x 1100")


@pytest.mark.parametrize("D", [96, 101])
def test_norm_alone(D):
    """Without a block's output the call is a norm of the stream; its backward adds the stream's own gradient."""
    import torch

    b = Block(490 + D, 19, D, "bf16", "f32", "none")
    x_out, h = binding.gdn2_block_norm_fwd(b.t["x"], weight_pre=b.t["w_pre"], dtype=torch.bfloat16)
    assert x_out is b.t["x"] and h.dtype == torch.bfloat16
    close(h, O.block_norm_h(b.x, b.w_pre, b.oracle["eps"]), "norm alone h")
    for d in (b.d_x_out, None):
        got = binding.gdn2_block_norm_bwd(b.t["x"], None, dev(d, "f32"), b.t["d_h"], weight_pre=b.t["w_pre"])
        want = O.block_norm_grads(b.x, None, d, b.d_h, w_pre=b.w_pre, eps=b.oracle["eps"])
        for name in ("d_x", "d_weight_pre"):
            close(got[name], want[name], f"norm alone {name}")
        assert got["d_u"] is None and got["d_gate"] is None


def test_block_in_place_and_unwanted_gradients():
    import torch

    b = Block(500, 50, 264, "bf16", "f32", "channel", "silu", p=0.3)
    x_out, h = b.fwd()
    x = b.t["x"].clone()
    y, h2 = binding.gdn2_block_norm_fwd(x, b.t["u"], x_out=x, **b.how)
    assert y is x and torch.equal(x, x_out) and torch.equal(h, h2)
    full = b.bwd(x_out)
    d = b.t["d_x_out"].clone()
    got = binding.gdn2_block_norm_bwd(x_out, b.t["u"], d, b.t["d_h"], d_x=d, want_d_gate=False, want_d_weights=False,
                                      **b.how)
    assert got["d_x"] is d and torch.equal(d, full["d_x"]) and torch.equal(got["d_u"], full["d_u"])
    assert got["d_gate"] is None and got["d_weight_post"] is None and got["d_weight_pre"] is None
    # no dx from later blocks is a zero one
    zero = b.bwd(x_out, d_x=torch.empty_like(d))
    b.t["d_x_out"] = None
    none = b.bwd(x_out)
    b.t["d_x_out"] = torch.zeros_like(d)
    assert torch.equal(none["d_u"], b.bwd(x_out)["d_u"]) and not torch.equal(none["d_u"], zero["d_u"])


def test_block_keeps_what_lies_around_its_outputs():
    """Outputs inside larger buffers: rows before and behind them stay as they were (odd width: unaligned row ends)."""
    import torch

    b = Block(505, 13, 75, "bf16", "bf16", "token", p=0.2)
    pad = 16  # elements in front: keeps the 16-byte alignment
    def inside(t):
        n = t.numel()
        big = torch.full((n + 2 * pad,), 7.0, dtype=t.dtype, device="cuda")
        return big, big[pad:pad + n].view(t.shape)
    x_out, h = b.fwd()
    bx, vx = inside(x_out)
    bh, vh = inside(h)
    b.fwd(x_out=vx, h=vh)
    want = b.bwd(x_out)
    bufs = {n: inside(want[n]) for n in ("d_x", "d_u", "d_gate")}
    b.bwd(x_out, **{n: v for n, (_, v) in bufs.items()})
    for big, view, ref in [(bx, vx, x_out), (bh, vh, h)] + [(*bufs[n], want[n]) for n in bufs]:
        assert torch.equal(view, ref)
        assert (big[:pad] == 7).all() and (big[pad + ref.numel():] == 7).all()


def test_block_nonfinite_rows_stay_apart():
    """A row with NaN or infinity does not reach another one; a dropped NaN leaves the stream alone; a row of zeros
    has a finite norm."""
    import torch

    b = Block(510, 6, 40, "f32", "f32", "full", p=0.0)
    ref_x, ref_h = b.fwd()
    b.t["u"][1, 3] = float("nan")
    b.t["u"][3, 5] = float("inf")
    b.t["x"][4] = 0
    b.t["u"][4] = 0
    x_out, h = b.fwd()
    for r in (0, 2, 5):
        assert torch.equal(x_out[r], ref_x[r]) and torch.equal(h[r], ref_h[r])
    assert torch.isnan(x_out[1]).all() and torch.isnan(h[1]).all()
    assert torch.isnan(x_out[3, 5]) and torch.isnan(h[3]).all()
    assert (x_out[4] == 0).all() and (h[4] == 0).all()
    got = b.bwd(ref_x)
    for r in (0, 2, 4, 5):
        assert torch.isfinite(got["d_u"][r]).all() and torch.isfinite(got["d_x"][r]).all()
    # everything dropped: the stream passes, NaN or not, and the block's gradients are zero
    one = dict(dropout_p=1.0)
    x_out, _ = b.fwd(**one)
    assert torch.equal(x_out, b.t["x"])
    got = b.bwd(ref_x, **one)
    assert (got["d_u"][[0, 2, 4, 5]] == 0).all() and (got["d_gate"][[0, 2, 4, 5]] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 8), (1, 100003), (257, 333), (1000, 2048), (4, 5461)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(dtype, rows, D, p):
    import torch

    x = rnd(np.random.default_rng(520 + D), (rows, D), dtype)
    seed, offset = 0xFEDCBA9876543210, 77 + (1 << 40)
    y = binding.gdn2_dropout(dev(x, dtype), p, seed, offset)
    ref = O.dropout(x, p, seed, offset)
    close(y, (ref, 2 * O.U * np.abs(ref)), f"dropout {dtype} {rows}x{D} p={p}")
    z = dev(x, dtype)
    assert binding.gdn2_dropout(z, p, seed, offset, out=z) is z and torch.equal(z, y)


def test_dropout_drops_nonfinite_values():
    import torch

    x = torch.full((8, 333), float("nan"), device="cuda")
    y = binding.gdn2_dropout(x, 0.5, 9)
    keep = torch.from_numpy(O.kept(8, 333, 0.5, 9, 0)).cuda()
    assert torch.isnan(y[keep]).all() and (y[~keep] == 0).all()


def test_dropout_is_the_mask_of_the_block():
    """x = 0, u = 1 without norms and gate: the block step is dropout alone, with the same mask at any width."""
    import torch

    for D in (16, 77, 1000, 5000):
        u = torch.ones((9, D), device="cuda")
        x_out, _ = binding.gdn2_block_norm_fwd(torch.zeros_like(u), u, dropout_p=0.3, seed=4, offset=6)
        assert torch.equal(x_out, binding.gdn2_dropout(u, 0.3, 4, 6))


def test_dropout_past_two_to_the_32_elements():
    """Rows on both sides of element 2^32 of one call (bf16, 8.6 GB each way)."""
    import torch

    D = 4096
    rows = (1 << 20) + 40
    x = torch.ones((rows, D), dtype=torch.bfloat16, device="cuda")
    y = binding.gdn2_dropout(x, 0.25, 3, 1, out=x)
    for first in (0, (1 << 19) - 3, (1 << 20) - 8, rows - 8):
        keep = O.kept(8, D, 0.25, 3, 1, first_row=first)
        np.testing.assert_array_equal(G.f64(y[first:first + 8]) > 0, keep)
    del x, y
    torch.cuda.empty_cache()


def test_block_past_two_to_the_32_elements():
    """x_out in place over 2^32 elements; the last rows against the same rows alone, with the dropout mask off."""
    import torch

    D, rows = 2048, (1 << 21) + 17
    g = torch.Generator(device="cuda").manual_seed(5)
    tail_u = torch.randn((17, D), generator=g, device="cuda").to(torch.bfloat16)
    tail_x = torch.randn((17, D), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(D, device="cuda")
    u = torch.zeros((rows, D), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((rows, D), dtype=torch.bfloat16, device="cuda")
    u[-17:], x[-17:] = tail_u, tail_x
    ref, href = binding.gdn2_block_norm_fwd(tail_x, tail_u, weight_post=w, weight_pre=w)
    x_out, h = binding.gdn2_block_norm_fwd(x, u, weight_post=w, weight_pre=w, x_out=x)
    assert torch.equal(x_out[-17:], ref) and torch.equal(h[-17:], href) and not x_out[:-17].any()
    got = binding.gdn2_block_norm_bwd(x_out, u, h, h, weight_post=w, weight_pre=w, d_x=h.clone())
    alone = binding.gdn2_block_norm_bwd(ref, tail_u, href, href, weight_post=w, weight_pre=w)
    assert torch.equal(got["d_x"][-17:], alone["d_x"]) and torch.equal(got["d_u"][-17:], alone["d_u"])
    for name in ("d_weight_post", "d_weight_pre"):  # 17 terms in another order: 34 roundings of the largest partial sum
        assert (got[name] - alone[name]).abs().max() <= 64 * O.U * 17 * alone[name].abs().max()
    del u, x, x_out, h, got
    torch.cuda.empty_cache()


def test_block_step_in_a_replayed_graph():
    """Forward and backward captured with a device offset: every replay draws the mask of the offset at that time,
    and equals the eager calls, with eager work between the replays."""
    import torch

    b = Block(540, 70, 520, "bf16", "f32", "channel", "silu", p=0.3)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        x_out, h = binding.gdn2_block_norm_fwd(b.t["x"], b.t["u"], offset_device=counter, **b.how)
        return x_out, h, binding.gdn2_block_norm_bwd(x_out, b.t["u"], b.t["d_x_out"], b.t["d_h"], offset_device=counter,
                                                     **b.how)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x_out, h, got = step()
        counter.add_(1)
    counter.zero_()
    masks = []
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert int(counter) == k + 1
        how = {**b.how, "offset": b.rand["offset"] + k}
        ex, eh = binding.gdn2_block_norm_fwd(b.t["x"], b.t["u"], **how)
        eager = binding.gdn2_block_norm_bwd(ex, b.t["u"], b.t["d_x_out"], b.t["d_h"], **how)
        assert torch.equal(x_out, ex) and torch.equal(h, eh), f"replay {k}"
        for name, v in eager.items():
            assert torch.equal(got[name], v), f"replay {k}: {name}"
        masks.append(x_out.clone())
    assert not torch.equal(masks[0], masks[1])


def test_calls_without_rows():
    """Nothing to read, and the gradients of shared inputs are zero."""
    import torch

    for D in (64, 75):
        e = torch.empty((0, D), dtype=torch.bfloat16, device="cuda")
        w, g = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        how = dict(gate=g, gate_layout="channel", weight_post=w, weight_pre=w, dropout_p=0.1, seed=1)
        x_out, h = binding.gdn2_block_norm_fwd(e, e.clone(), **how)
        assert x_out.shape == h.shape == (0, D)
        got = binding.gdn2_block_norm_bwd(e, e.clone(), e.clone(), e.clone(), **how)
        for n in ("d_gate", "d_weight_post", "d_weight_pre"):
            assert got[n].shape == (D,) and not got[n].any()
        assert binding.gdn2_dropout(e, 0.1, 1).shape == (0, D)
    e = torch.empty((0, 64), device="cuda")
    assert not binding.gdn2_mixer_epilogue_bwd(e, e.clone(), torch.ones(64, device="cuda"), e.clone())["d_weight"].any()


def test_calls_at_once_on_two_streams():
    """Two streams run the same backward calls side by side, many times over: each result is that of the call alone."""
    import torch

    blocks = [Block(548 + k, 2000, 264, "bf16", "f32", "channel", "silu", p=0.3) for k in range(2)]
    outs = [b.fwd()[0] for b in blocks]
    refs = [b.bwd(x) for b, x in zip(blocks, outs)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [binding.gdn2_block_norm_bwd(x, b.t["u"], b.t["d_x_out"], b.t["d_h"], stream=s, **b.how)
               for b, x, s in zip(blocks, outs, streams)]
    torch.cuda.synchronize()
    for g, ref in zip(got, refs):
        for name, v in ref.items():
            assert torch.equal(g[name], v), name


@pytest.mark.parametrize("dtype,res", TYPES)
def test_fused_step_is_the_step_and_then_the_norm(dtype, res):
    """The norm of the stored stream alone gives the fused call's h, bit for bit, and so do its gradients in turn."""
    import torch

    for D in (75, 96, 1371, 2048):
        b = Block(549 + D, 40, D, dtype, res, "full", "silu", p=0.2)
        x_out, h = b.fwd()
        t = b.t["u"].dtype
        assert torch.equal(binding.gdn2_block_norm_fwd(x_out, weight_pre=b.t["w_pre"], dtype=t)[1], h)
        alone, _ = b.fwd(weight_pre=None)
        assert torch.equal(alone, x_out)
        fused = b.bwd(x_out)
        norm = binding.gdn2_block_norm_bwd(x_out, None, b.t["d_x_out"], b.t["d_h"], weight_pre=b.t["w_pre"])
        assert torch.equal(norm["d_x"], fused["d_x"])


def test_one_leading_axis_or_several():
    """A call over [B, T, D] is the call over its rows."""
    import torch

    b = Block(546, 24, 96, "bf16", "f32", "token", "silu", p=0.2)
    x_out, h = b.fwd()
    cut = lambda t: t.view(4, 6, *t.shape[1:])  # noqa: E731
    how = {**b.how, "gate": cut(b.t["gate"])}
    y, h3 = binding.gdn2_block_norm_fwd(cut(b.t["x"]), cut(b.t["u"]), **how)
    assert torch.equal(y, cut(x_out)) and torch.equal(h3, cut(h))
    one = binding.gdn2_dropout(b.t["x"], 0.2, 3)
    assert torch.equal(binding.gdn2_dropout(cut(b.t["x"]), 0.2, 3), cut(one))


def test_calls_on_another_stream_and_repeated():
    """On a stream of its own, twice: bit for bit what the current stream gives."""
    import torch

    b = Block(545, 3000, 264, "bf16", "f32", "channel", "silu", p=0.3)
    x_out, h = b.fwd()
    ref = b.bwd(x_out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        y, h2 = binding.gdn2_block_norm_fwd(b.t["x"], b.t["u"], stream=s, **b.how)
        got = binding.gdn2_block_norm_bwd(y, b.t["u"], b.t["d_x_out"], b.t["d_h"], stream=s, **b.how)
        s.synchronize()
        assert torch.equal(y, x_out) and torch.equal(h2, h)
        for name, v in ref.items():
            assert torch.equal(got[name], v), name


# --- mixer backward ----------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dv", [32, 64, 128])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("rows", [1, 15, 1027])
def test_epilogue_bwd(dtype, dv, act, rows):
    rng = np.random.default_rng(560 + dv + rows)
    o, gate, dy = (rnd(rng, (rows, dv), dtype) for _ in range(3))
    w = rnd(rng, (dv,), "f32", 0.2, 1.0)
    got = binding.gdn2_mixer_epilogue_bwd(dev(o, dtype), dev(gate, dtype), dev(w), dev(dy, dtype), act=act)
    want = O.epilogue_grads(o, gate, w, dy, float(np.float32(1e-5)), act)
    for name, ref in want.items():
        close(got[name], ref, f"epilogue bwd {dtype} {act} {rows}x{dv} {name}")


def test_epilogue_bwd_many_rows():
    """More rows than the workgroups take at once; the weight's gradient not wanted leaves the others alone."""
    import torch

    rng = np.random.default_rng(570)
    o, gate, dy = (rnd(rng, (3, 50, 333, 32), "bf16") for _ in range(3))
    w = rnd(rng, (32,), "f32", 0.2, 1.0)
    a = [dev(o, "bf16"), dev(gate, "bf16"), dev(w), dev(dy, "bf16")]
    got = binding.gdn2_mixer_epilogue_bwd(*a)
    flat = lambda z: z.reshape(-1, 32)  # noqa: E731
    want = O.epilogue_grads(flat(o), flat(gate), w, flat(dy), float(np.float32(1e-5)))
    close(flat(got["d_o"]), want["d_o"], "epilogue bwd d_o")
    close(flat(got["d_gate"]), want["d_gate"], "epilogue bwd d_gate")
    close(got["d_weight"], want["d_weight"], "epilogue bwd d_weight")
    less = binding.gdn2_mixer_epilogue_bwd(*a, want_d_weight=False)
    assert less["d_weight"] is None and torch.equal(less["d_o"], got["d_o"]) and torch.equal(less["d_gate"], got["d_gate"])


class Prologue:
    def __init__(self, seed, B, T, H, dk, dv, K, dtype, lens=None, state=True):
        rng = np.random.default_rng(seed)
        self.cu = None if lens is None else W.cu_from_lengths(lens)
        N = B if lens is None else len(lens)
        if lens is not None:
            B, T = 1, int(self.cu[-1])
        wide = {"q": dk, "k": dk, "v": dv, "b": dk, "w": dv}
        self.x = [rnd(rng, (B, T, H, d), dtype) for d in (dk, dk, dv)]
        self.conv = [rnd(rng, (H * d, K), "f32", 0.5) for d in (dk, dk, dv)]
        self.logit = [rnd(rng, (B, T, H, d), dtype) for d in (dk, dv)]
        self.d = [rnd(rng, (B, T, H, d), dtype) for d in wide.values()]
        st = (N, H * (2 * dk + dv), K - 1)
        self.state, self.d_state = (rnd(rng, st, "f32") for _ in range(2)) if state else (None, None)
        self.dtype = dtype
        self.t = [dev(z, dtype) for z in self.x] + [dev(z) for z in self.conv] + [dev(z, dtype) for z in self.logit + self.d]
        self.how = dict(conv_state=dev(self.state), d_conv_state_out=dev(self.d_state), output_d_conv_state=True,
                        cu_seqlens=None if self.cu is None else dev_int(self.cu), q_scale=0.125)

    def run(self, **kw):
        import torch

        got = binding.gdn2_mixer_prologue_bwd(*self.t, **{**self.how, **kw})
        torch.cuda.synchronize()
        return got

    def check(self, what):
        got = self.run()
        want = O.prologue_grads(*self.x, *self.conv, *self.logit, *self.d, self.cu, self.state, self.d_state, 0.125,
                                float(np.float32(1e-6)))
        for name, ref in want.items():
            close(got[name], ref, f"{what} {name}")
        return got


def dev_int(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,K", [(32, 32, 4), (64, 128, 4), (128, 64, 2), (128, 128, 4), (64, 64, 1), (64, 32, 3),
                                     (32, 64, 7), (128, 32, 16), (32, 128, 5), (64, 64, 8), (128, 128, 11), (32, 32, 13)])
def test_prologue_bwd(dtype, dk, dv, K):
    Prologue(600 + dk + dv + K, 2, 37, 3, dk, dv, K, dtype).check(f"prologue bwd {dtype} dk={dk} dv={dv} K={K}")


@pytest.mark.parametrize("K", [1, 2, 4, 6, 16])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 64, 65, 130])
def test_prologue_bwd_lengths(K, T):
    """Rows shorter than the filter, and one run of tokens and a little more."""
    Prologue(640 + T + K, 3, T, 2, 64, 32, K, "f32").check(f"prologue bwd T={T} K={K}")
    Prologue(650 + T + K, 1, T, 9, 32, 32, K, "bf16", state=False).check(f"prologue bwd no state T={T} K={K}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 4, 8, 16])
def test_prologue_bwd_packed(dtype, K):
    """Packed sequences: empty ones (first, last and in a row), ones shorter than the filter, ones that end on, just
    before and just after a wavefront's run of tokens."""
    lens = [0, 1, 2, 9, 0, 0, 40, 3, 8, 1, 64, 1, 1, 62, 2, 130, 0]
    Prologue(680 + K, 1, 0, 2, 64, 64, K, dtype, lens=lens).check(f"prologue bwd packed {dtype} K={K}")


def test_prologue_bwd_long_rows():
    """Many runs a row: the filters' gradients are summed over them."""
    Prologue(700, 2, 1500, 2, 32, 32, 4, "bf16").check("prologue bwd T=1500")
    Prologue(701, 1, 0, 1, 64, 32, 3, "f32", lens=[700, 11, 1301]).check("prologue bwd packed long")


def test_prologue_bwd_without_tokens():
    """T = 0: the state's gradient passes through, the filters' gradients are zero."""
    import torch

    p = Prologue(710, 3, 0, 2, 32, 32, 4, "f32")
    got = p.run()
    assert torch.equal(got["d_conv_state"], p.how["d_conv_state_out"])
    for n in ("d_conv_q", "d_conv_k", "d_conv_v"):
        assert not got[n].any()


def test_prologue_bwd_unwanted_and_repeated():
    import torch

    p = Prologue(711, 2, 200, 4, 128, 128, 4, "bf16")
    a, b, c = p.run(), p.run(), p.run(want_d_conv=False, output_d_conv_state=False)
    for n in a:
        assert torch.equal(a[n], b[n]), n
        assert c[n] is None if "conv" in n else torch.equal(a[n], c[n]), n


@pytest.mark.parametrize("K", [1, 4, 7])
def test_prologue_bwd_padding_is_left_alone(K):
    """Packed sequences in a longer buffer with NaN behind them: the gradients are those of the sequences alone, and the
    gradient buffers keep what they held there."""
    import torch

    lens, pad = [5, 0, 130, 33], 77
    p = Prologue(713, 1, 0, 3, 64, 32, K, "bf16", lens=lens)
    ref = p.run()
    T, padded = sum(lens), []
    for z in p.t:
        if z.dim() == 4:
            z = torch.cat([z, torch.full((1, pad, *z.shape[2:]), float("nan"), dtype=z.dtype, device="cuda")], 1)
        padded.append(z)
    out = {n: torch.full((1, T + pad, *ref[n].shape[2:]), 7.0, dtype=torch.bfloat16, device="cuda") if ref[n].dim() == 4
           else torch.empty_like(ref[n]) for n in ref}
    ws = torch.empty(binding.gdn2_mixer_prologue_bwd_workspace_bytes(1, T + pad, 3, 64, 32, K), dtype=torch.uint8, device="cuda")
    at = lambda z: z.data_ptr()  # noqa: E731
    rc = binding.load().gdn2_mixer_prologue_bwd(
        *map(at, padded[:8]), at(p.how["conv_state"]), *map(at, padded[8:]), at(p.how["d_conv_state_out"]),
        *map(at, out.values()), at(p.how["cu_seqlens"]), 1, T + pad, 3, 64, 32, K, len(lens), 0.125, 1e-6, 1, at(ws),
        ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    for n, want in ref.items():
        if want.dim() == 4:
            assert torch.equal(out[n][:, :T], want), n
            assert (out[n][:, T:] == 7).all(), n
        elif "state" in n:
            assert torch.equal(out[n], want), n
        else:  # summed over another partition of the tokens
            assert torch.isfinite(out[n]).all() and (out[n] - want).norm() <= T * O.U * want.abs().max() * want.numel() ** 0.5, n


def test_prologue_bwd_malformed_offsets_stay_inside():
    """Offsets out of order or out of range are clamped like the forward call's: the call ends without a fault and the
    inputs are as they were (the results mean nothing); a well-formed call after it is right."""
    import torch

    p = Prologue(712, 1, 0, 2, 32, 32, 4, "f32", lens=[30, 40, 20])
    before = [z.clone() for z in p.t]
    for cu in ([-5, 40, 30, 90], [0, 1000, -3, 90], [10, 20, 30, 40]):
        p.run(cu_seqlens=dev_int(np.array(cu, dtype=np.int32)))
    assert all(torch.equal(a, b) for a, b in zip(before, p.t))
    p.check("prologue bwd after malformed offsets")


def test_prologue_bwd_headline_shape_sampled():
    """B=8, T=4096, H=16, d=128, K=4, bf16: two (row, head) chains over all their tokens."""
    import torch

    p = Prologue(720, 8, 4096, 16, 128, 128, 4, "bf16")
    got = p.run()
    torch.cuda.synchronize()
    for n, h in ((0, 0), (6, 11)):
        cut = lambda z: np.ascontiguousarray(z[n:n + 1, :, h:h + 1])  # noqa: E731
        st = lambda z: np.concatenate([z[n:n + 1, i * 2048 + h * 128:i * 2048 + (h + 1) * 128] for i in range(3)], axis=1)  # noqa: E731
        want = O.prologue_grads(*(cut(z) for z in p.x), *(z[h * 128:(h + 1) * 128] for z in p.conv),
                                *(cut(z) for z in p.logit + p.d), None, st(p.state), st(p.d_state), 0.125,
                                float(np.float32(1e-6)))
        for name, ref in want.items():
            if "conv" in name and "state" not in name:
                continue  # summed over the batch rows
            g = got[name]
            g = torch.cat([g[n:n + 1, i * 2048 + h * 128:i * 2048 + (h + 1) * 128] for i in range(3)], 1) if "state" in name \
                else g[n:n + 1, :, h:h + 1]
            close(g, ref, f"headline prologue bwd ({n}, {h}) {name}")


# --- a layer, forward and backward -------------------------------------------


def test_layer_forward_and_backward():
    """A layer as a training step runs it, through every operator: norm, projections, mixer prologue, recurrence,
    epilogue, output projection, block step; and back.  Its gradients against the same layer in 64 bits on the CPU.

    FP32, so errors are those of the chain of FP32 operators: the bar is the suite's 1e-4 in relative L2."""
    import torch

    gen = torch.Generator().manual_seed(8)
    B, T, H, d, K, p = 2, 70, 2, 32, 4, 0.2
    D = H * d
    seed, offset = 99, 5
    new = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=gen, dtype=torch.float64)).float().double()  # noqa: E731
    leaf = {"x": new(B, T, D), "w_in": 1 + new(D, scale=0.1), "w_q": new(D, D, scale=0.2), "w_k": new(D, D, scale=0.2),
            "w_v": new(D, D, scale=0.2), "w_b": new(D, D, scale=0.2), "w_w": new(D, D, scale=0.2),
            "w_g": new(D, D, scale=0.2), "w_o": new(D, D, scale=0.2), "conv_q": new(D, K, scale=0.5),
            "conv_k": new(D, K, scale=0.5), "conv_v": new(D, K, scale=0.5), "w_norm": 1 + new(d, scale=0.1),
            "w_post": 1 + new(D, scale=0.1), "w_pre": 1 + new(D, scale=0.1), "gate": new(D, scale=0.5)}
    alpha = (0.9 + 0.1 * torch.rand(B, T, H, d, generator=gen, dtype=torch.float64)).float().double()
    d_x_out, d_h = new(B, T, D), new(B, T, D)
    eps, eps_l2 = float(np.float32(1e-5)), float(np.float32(1e-6))

    # 64 bits, by reverse mode through the definition
    ref = {k: v.clone().requires_grad_(True) for k, v in leaf.items()}
    rms = lambda z, w: z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps) * w  # noqa: E731
    hin = rms(ref["x"], ref["w_in"])
    def conv(name):
        z = hin @ ref["w_" + name]
        z = torch.cat([torch.zeros(B, K - 1, D, dtype=torch.float64), z], 1)
        y = sum(ref["conv_" + name][:, i] * z[:, i:i + T] for i in range(K))
        y = (y * torch.sigmoid(y)).reshape(B, T, H, d)
        return y if name == "v" else y / torch.sqrt((y * y).sum(-1, keepdim=True) + eps_l2)
    q, k, v = conv("q"), conv("k"), conv("v")
    b, w = (torch.sigmoid((hin @ ref["w_" + n]).reshape(B, T, H, d)) for n in "bw")
    S, o = torch.zeros(B, H, d, d, dtype=torch.float64), []
    for t in range(T):
        S = alpha[:, t, :, :, None] * S
        read = ((b[:, t] * k[:, t])[..., None] * S).sum(-2)
        S = S + k[:, t, :, :, None] * (w[:, t] * v[:, t] - read)[..., None, :]
        o.append((q[:, t, :, :, None] * S).sum(-2))
    o = torch.stack(o, 1)
    y = rms(o, ref["w_norm"]) * torch.sigmoid((hin @ ref["w_g"]).reshape(B, T, H, d))
    u = y.reshape(B, T, D) @ ref["w_o"]
    m = torch.from_numpy(O.dropout(np.ones((B * T, D)), p, seed, offset)).reshape(B, T, D)
    g = ref["gate"] * torch.sigmoid(ref["gate"])
    x_out = ref["x"] + 0.5 * m * g * rms(u, ref["w_post"])
    loss = (x_out * d_x_out).sum() + (rms(x_out, ref["w_pre"]) * d_h).sum()
    grads = dict(zip(ref, torch.autograd.grad(loss, list(ref.values()))))

    # the library, FP32
    L = {k: z.float().cuda() for k, z in leaf.items()}
    A, DX, DH = alpha.float().cuda(), d_x_out.float().cuda(), d_h.float().cuda()
    heads = lambda z: z.reshape(B, T, H, d)  # noqa: E731
    flat = lambda z: z.reshape(B * T, D)  # noqa: E731
    x, hin = binding.gdn2_block_norm_fwd(L["x"], weight_pre=L["w_in"])
    proj = {n: heads(hin @ L["w_" + n]) for n in "qkvbwg"}
    mix = binding.gdn2_mixer_prologue(proj["q"], proj["k"], proj["v"], L["conv_q"], L["conv_k"], L["conv_v"], proj["b"],
                                      proj["w"])
    o, _ = binding.gdn2_chunk_fwd(mix["q"], mix["k"], mix["v"], A, mix["b"], mix["w"])
    y = binding.gdn2_mixer_epilogue(o, proj["g"], L["w_norm"])
    u = y.reshape(B, T, D) @ L["w_o"]
    step = dict(gate=L["gate"], gate_layout="channel", gate_act="silu", weight_post=L["w_post"], weight_pre=L["w_pre"],
                residual_scale=0.5, dropout_p=p, seed=seed, offset=offset)
    x_out, h = binding.gdn2_block_norm_fwd(x, u, **step)
    bs = binding.gdn2_block_norm_bwd(x_out, u, DX, DH, **step)
    got = {"w_post": bs["d_weight_post"], "w_pre": bs["d_weight_pre"], "gate": bs["d_gate"],
           "w_o": flat(y).T @ flat(bs["d_u"])}
    e = binding.gdn2_mixer_epilogue_bwd(o, proj["g"], L["w_norm"], heads(bs["d_u"] @ L["w_o"].T))
    r = binding.gdn2_chunk_bwd(mix["q"], mix["k"], mix["v"], A, mix["b"], mix["w"], e["d_o"])
    pb = binding.gdn2_mixer_prologue_bwd(proj["q"], proj["k"], proj["v"], L["conv_q"], L["conv_k"], L["conv_v"], proj["b"],
                                         proj["w"], r["dq"], r["dk"], r["dv"], r["db"], r["dw"])
    got.update({n: pb["d_" + n] for n in ("conv_q", "conv_k", "conv_v")}, w_norm=e["d_weight"])
    d_proj = {"q": pb["d_xq"], "k": pb["d_xk"], "v": pb["d_xv"], "b": pb["d_b_logit"], "w": pb["d_w_logit"],
              "g": e["d_gate"]}
    for n, dz in d_proj.items():
        got["w_" + n] = flat(hin).T @ flat(dz)
    d_hin = sum(flat(dz) @ L["w_" + n].T for n, dz in d_proj.items()).reshape(B, T, D)
    first = binding.gdn2_block_norm_bwd(x, None, bs["d_x"], d_hin, weight_pre=L["w_in"])
    got.update(x=first["d_x"], w_in=first["d_weight_pre"])
    assert set(got) == set(grads)
    for n in got:
        G.assert_rel(G.f64(got[n]), grads[n].numpy(), G.TOL["f32"], f"layer gradient of {n}")
