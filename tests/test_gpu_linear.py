"""GPU parity of linear attention with a fixed decay for each head (gdn2_linear_attn_fwd, _bwd, _step)
against the FP64 oracle in oracle/linear.py (needs an MI355X).

Bars.  Element by element, with A the oracle's sum over absolute values:
  * a state: FP32 sums.  A chunk adds 64 products in three bf16 parts, at most 3 x 64 additions, and multiplies
    the carry once: at most 200 roundings of U = 2^-24 a chunk, of terms below A.
  * an output: half a step of its type of its own value, of A where the carry's copy is rounded to bf16 (2^-8; FP32
    inputs: none), 2^-16 of A for products inside the chunk that go in as two bf16 terms, and a state's roundings.
Whole tensors: the parts of an output are sums of independent terms of both signs, so the two roundings to bf16 add as
squares: each at most 2^-8 / sqrt(3) rms, together 2^-8 sqrt(2 / 3), in relative L2 (a quarter more for small
samples).  FP32 results: 1e-6 (17 U rms)."""
import numpy as np
import pytest

import gpu_util as G
import oracle
from delta_rule_linear_gdn2_amd import binding
from delta_rule_linear_gdn2_amd import workloads as W
from oracle import linear as L

pytestmark = pytest.mark.gpu

U = L.U
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
BAR = {"f32": 1e-6, "bf16": 1.25 * 2.0 ** -8 * (2 / 3) ** 0.5}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    yield


def rnd(rng, shape, dtype, scale=1.0):
    x = (scale * rng.standard_normal(shape)).astype(np.float32)
    return W.round_bf16(x) if dtype == "bf16" else x


def dev(x, dtype="f32"):
    return None if x is None else W.to_torch(np.ascontiguousarray(x), dtype, "cuda")


def alphas(H):
    """From heads that forget at once to heads that never do."""
    return np.array([0.996, 0.5, 1.0, 0.9, 0.0, 0.98, 0.1, 0.999], dtype=np.float32)[np.arange(H) % 8]


class Case:
    def __init__(self, seed, B, T, H, dk, dv, dtype, cu=None, state=True, alpha=None):
        r = np.random.default_rng(seed)
        N = B if cu is None else len(cu) - 1
        self.dtype, self.cu = dtype, None if cu is None else np.asarray(cu, dtype=np.int32)
        self.q, self.k = rnd(r, (B, T, H, dk), dtype, dk ** -0.5), rnd(r, (B, T, H, dk), dtype)
        self.v, self.d_o = rnd(r, (B, T, H, dv), dtype), rnd(r, (B, T, H, dv), dtype)
        self.alpha = alphas(H) if alpha is None else np.asarray(alpha, dtype=np.float32)
        self.s0 = rnd(r, (N, H, dk, dv), "f32") if state else None
        self.ds = rnd(r, (N, H, dk, dv), "f32") if state else None
        self.t = dict(q=dev(self.q, dtype), k=dev(self.k, dtype), v=dev(self.v, dtype), alpha=dev(self.alpha))
        self.t_s0, self.t_ds, self.t_do = dev(self.s0), dev(self.ds), dev(self.d_o, dtype)
        self.t_cu = None
        if cu is not None:
            import torch

            self.t_cu = torch.from_numpy(self.cu).cuda()
        lengths = [T] if cu is None else np.diff(self.cu).tolist()
        self.chunks = max(1, -(-max(lengths) // L.CHUNK))

    def fwd(self, **kw):
        import torch

        out = binding.gdn2_linear_attn_fwd(**self.t, initial_state=self.t_s0, cu_seqlens=self.t_cu, **kw)
        torch.cuda.synchronize()
        return out

    def bwd(self, **kw):
        import torch

        out = binding.gdn2_linear_attn_bwd(**self.t, d_o=self.t_do, initial_state=self.t_s0, d_final_state=self.t_ds,
                                           output_d_initial_state=True, cu_seqlens=self.t_cu, **kw)
        torch.cuda.synchronize()
        return out

    def close(self, got, ref, size, what, state=False):
        x, half = G.f64(got), HALF["f32" if state else self.dtype]
        assert x.shape == ref.shape, f"{what}: {x.shape} != {ref.shape}"
        room = 200 * self.chunks * U * size + half * np.abs(ref) + 1e-37
        if self.dtype == "bf16" and not state:
            room = room + (HALF["bf16"] + 2.0 ** -16) * size
        bad = ~(np.abs(x - ref) <= room)
        assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}"
        if ref.size:
            G.assert_rel(x, ref, BAR["f32" if state else self.dtype], what)

    def check(self, what, **kw):
        """Both directions against the oracle."""
        args, size = (self.q, self.k, self.v, self.alpha), [np.abs(x) for x in (self.q, self.k, self.v)]
        ab = None if self.s0 is None else np.abs(self.s0)
        o, s = self.fwd(**kw)
        (ro, rs), (ao, as_) = L.attn(*args, self.s0, self.cu), L.attn(*size, self.alpha, ab, self.cu)
        self.close(o, ro, ao, f"{what} o")
        self.close(s, rs, as_, f"{what} final state", state=True)
        got = self.bwd(**kw)
        want = L.attn_grads(*args, self.d_o, self.s0, self.ds, self.cu)
        bound = L.attn_grads(*size, self.alpha, np.abs(self.d_o), ab, None if self.ds is None else np.abs(self.ds), self.cu)
        for name in want:
            self.close(got[name], want[name], bound[name], f"{what} {name}", state=name == "d_initial_state")
        return o, s, got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_head_sizes(dk, dv, dtype):
    Case(dk + dv, 2, 150, 3, dk, dv, dtype).check(f"{dtype} dk={dk} dv={dv}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 31, 32, 33, 63, 64, 65, 95, 96, 127, 128, 129, 191, 257])
def test_lengths(T, dtype):
    """Either side of a chunk's and of a tile's border."""
    Case(300 + T, 1, T, 2, 64, 64, dtype, state=T % 2 == 1, alpha=[0.97, 0.4]).check(f"{dtype} T={T}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 1], [0, 0, 5], [0, 64, 64, 64, 128], [0, 1, 2, 3, 70, 200], [0, 63, 128, 193, 193],
                                [0] + [7] * 70 + [20]])
def test_packed(cu, dtype):
    Case(400 + len(cu), 1, cu[-1], 2, 32, 64, dtype, cu=cu, alpha=[0.95, 1.0]).check(f"{dtype} packed {cu[:6]}")


@pytest.mark.parametrize("alpha", [[1.0] * 4, [0.0] * 4, [1e-30, 3.0, 2.0 ** -15, 0.9999]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_at_the_ends(alpha, dtype):
    """No decay, everything forgotten within a token (clamped to 2^-15), and values outside [0, 1]."""
    Case(450, 2, 200, 4, 64, 32, dtype, alpha=alpha).check(f"{dtype} alpha {alpha}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv,T", [(128, 128, 2050), (64, 32, 1500), (128, 64, 1024)])
def test_segments(dk, dv, T, dtype):
    """Few heads: several segments a row.  The walk in one piece gives the same up to rounding, the final state in
    place gives it bit for bit."""
    import torch

    c = Case(500 + T, 1, T, 2, dk, dv, dtype, alpha=[0.999, 0.9])
    assert binding.gdn2_linear_attn_fwd_workspace_bytes(1, T, 2, dk, dv, 0, int(dtype == "bf16")) > 0
    o, s, got = c.check(f"{dtype} segments T={T} {dk}x{dv}")
    c.check(f"{dtype} one piece T={T} {dk}x{dv}", segmented=False)
    state = c.t_s0.clone()
    o2, s2 = binding.gdn2_linear_attn_fwd(**c.t, initial_state=state, final_state=state)
    assert s2 is state and torch.equal(o2, o) and torch.equal(s2, s)
    again = c.bwd()
    assert all(torch.equal(again[n], got[n]) for n in got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_segments(dtype):
    """Sequences longer than a segment beside short and empty ones, with segment borders that fall anywhere."""
    cu = [0, 0, 700, 701, 701, 2100, 2163, 2500]
    c = Case(520, 1, 2500, 2, 64, 128, dtype, cu=cu, alpha=[0.998, 0.8])
    assert binding.gdn2_linear_attn_fwd_workspace_bytes(1, 2500, 2, 64, 128, len(cu) - 1, 1) > 0
    o, s, _ = c.check(f"{dtype} packed segments")
    state = c.t_s0.clone()
    binding.gdn2_linear_attn_fwd(**c.t, initial_state=state, final_state=state, cu_seqlens=c.t_cu)
    import torch

    assert torch.equal(state, s)
    c.check(f"{dtype} packed, one piece", segmented=False)
    d = Case(521, 1, 2500, 2, 64, 128, dtype, cu=[0] * 100 + cu[1:], alpha=[0.998, 0.8])  # more than 64 sequences
    d.check(f"{dtype} packed segments behind empty sequences")


def test_thousands_of_sequences():
    """Most of them empty or of a token, two of them longer than a segment."""
    r = np.random.default_rng(523)
    cu = np.sort(np.concatenate([[0, 0], r.integers(0, 900, 4996), [900, 1700, 2600]]))
    c = Case(524, 1, 2600, 1, 32, 32, "bf16", cu=cu, alpha=[0.99])
    assert binding.gdn2_linear_attn_fwd_workspace_bytes(1, 2600, 1, 32, 32, len(cu) - 1, 1) > 0
    c.check("5000 sequences")


@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 128), (128, 128)])
def test_a_lone_token_is_rounded_once(dk, dv):
    """Without a state, o = (q . k) v: half a step of bf16, and 2^-16 of the product's size."""
    c = Case(580 + dk, 5, 1, 3, dk, dv, "bf16", state=False)
    ref, _ = L.attn(c.q, c.k, c.v, c.alpha)
    size, _ = L.attn(np.abs(c.q), np.abs(c.k), np.abs(c.v), c.alpha)
    assert (np.abs(G.f64(c.fwd()[0]) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -16 + 200 * U) * size).all()


def test_nothing_to_walk():
    """T = 0 and empty sequences hand the state on, in both directions."""
    import torch

    for cu in (None, [0, 0, 0]):
        c = Case(530, 1 if cu else 2, 0, 2, 32, 64, "bf16", cu=cu)
        o, s = c.fwd()
        assert o.numel() == 0 and torch.equal(s, c.t_s0)
        assert torch.equal(c.bwd()["d_initial_state"], c.t_ds)
    c = Case(531, 2, 0, 2, 32, 64, "f32", state=False)
    assert not c.fwd()[1].any()


def test_padding_around_packed_sequences():
    """Tokens that no sequence owns are not read; their rows are zero in new tensors and untouched in given ones."""
    import torch

    c = Case(540, 1, 300, 2, 64, 64, "bf16", cu=[10, 100, 250])
    for x in ("q", "k", "v"):
        c.t[x][:, :10] = float("nan")
        c.t[x][:, 250:] = float("nan")
    c.t_do[:, :10] = float("nan")
    c.t_do[:, 250:] = float("nan")
    inner = Case(540, 1, 300, 2, 64, 64, "bf16")
    sl = slice(10, 250)
    ro, rs = L.attn(inner.q[:, sl], inner.k[:, sl], inner.v[:, sl], c.alpha, c.s0, [0, 90, 240])
    o, s = c.fwd()
    G.assert_rel(G.f64(o[:, sl]), ro, BAR["bf16"], "padded o")
    G.assert_rel(G.f64(s), rs, 1e-6, "padded state")
    got = c.bwd()
    for x in (o, got["dq"], got["dk"], got["dv"]):
        assert not x[:, :10].any() and not x[:, 250:].any() and torch.isfinite(x).all()
    mine = torch.full_like(o, 7.0)
    c.fwd(out=mine)
    assert (mine[:, :10] == 7).all() and (mine[:, 250:] == 7).all() and torch.equal(mine[:, sl], o[:, sl])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 100, 1300])
def test_surroundings_stay(T, dtype):
    """What lies before and behind every output is left as it was."""
    import torch

    c = Case(550, 1, T, 2, 64, 128, dtype)

    def room(like):
        n, pad = like.numel(), 64
        flat = torch.full((n + 2 * pad,), 3.0, dtype=like.dtype, device="cuda")
        return flat, flat[pad:pad + n].view(like.shape)

    fo, o = room(c.t["v"])
    fs, s = room(c.t_s0)
    c.fwd(out=o, final_state=s)
    ro, rs = c.fwd()
    assert torch.equal(o, ro) and torch.equal(s, rs)
    for flat in (fo, fs):
        assert (flat[:64] == 3).all() and (flat[-64:] == 3).all()


def test_malformed_offsets_stay_inside():
    """Offsets out of range or falling give results without meaning, inside the tensors."""
    import torch

    c = Case(560, 1, 700, 2, 64, 64, "bf16", cu=[0, 300, 700])
    for cu in ([-5, 900, 700], [0, 650, 100], [700, 0, 700], [0, 1 << 30, -(1 << 30)]):
        c.t_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        flat = torch.full((700 * 2 * 64 + 128,), 3.0, dtype=torch.bfloat16, device="cuda")
        c.fwd(out=flat[64:-64].view(c.t["v"].shape))
        c.bwd()
        assert (flat[:64] == 3).all() and (flat[-64:] == 3).all()


def test_non_finite_values_stay_in_their_sequence_and_behind():
    """A NaN reaches its own sequence and head from its chunk on, and nothing else."""
    import torch

    c = Case(570, 1, 400, 2, 64, 64, "bf16", cu=[0, 200, 400], alpha=[0.9, 0.9])
    ref, sref = c.fwd()
    for name in ("q", "k", "v"):
        t = c.t[name].clone()
        c.t[name][0, 150, 1, 3] = float("nan")
        o, s = c.fwd()
        same = o == ref
        assert same[:, :, 0].all() and same[:, 200:].all() and same[:, :128].all()
        if name == "q":
            bad = ~same[0, :, 1].all(-1)
            assert bad.nonzero().flatten().tolist() == [150] and torch.equal(s, sref)
        else:
            assert torch.isnan(o[0, 150:200, 1]).any(-1).all() and torch.isnan(s[0, 1]).any()
            assert torch.equal(s[1], sref[1]) and torch.equal(s[0, 0], sref[0, 0])
        c.t[name] = t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,dk,dv", [(1, 1, 128, 128), (3, 5, 64, 32), (7, 3, 32, 64), (2, 4, 128, 32), (33, 2, 32, 128),
                                       (5, 1, 64, 128), (2, 3, 32, 32), (4, 2, 64, 64), (3, 3, 128, 64)])
def test_step(N, H, dk, dv, dtype):
    """One token: the recurrence itself.  A state element takes two roundings, an output at most dk + 4."""
    import torch

    c = Case(600 + N, N, 1, H, dk, dv, dtype)
    state = c.t_s0.clone()
    o = binding.gdn2_linear_attn_step(c.t["q"][:, 0].contiguous(), c.t["k"][:, 0].contiguous(), c.t["v"][:, 0].contiguous(),
                                      c.t["alpha"], state)
    torch.cuda.synchronize()
    ro, rs = L.attn(c.q, c.k, c.v, c.alpha, c.s0)
    ao, as_ = L.attn(np.abs(c.q), np.abs(c.k), np.abs(c.v), c.alpha, np.abs(c.s0))
    assert (np.abs(G.f64(state) - rs) <= 3 * U * as_).all()
    off = np.abs(G.f64(o) - ro[:, 0])
    assert (off <= HALF[dtype] * np.abs(ro[:, 0]) + (dk + 6) * U * ao[:, 0]).all()
    assert binding.gdn2_linear_attn_step(c.t["q"][:0, 0], c.t["k"][:0, 0], c.t["v"][:0, 0], c.t["alpha"], state[:0]).numel() == 0


def test_prompt_then_steps():
    """The state of a prompt continues token by token as the whole sequence would."""
    import torch

    c = Case(620, 2, 140, 3, 64, 64, "bf16", alpha=[0.99, 0.8, 1.0])
    P = 100
    cut = {n: c.t[n][:, :P].contiguous() for n in ("q", "k", "v")}
    o, state = binding.gdn2_linear_attn_fwd(**cut, alpha=c.t["alpha"], initial_state=c.t_s0)
    rest = [binding.gdn2_linear_attn_step(*(c.t[n][:, t].contiguous() for n in ("q", "k", "v")), c.t["alpha"], state)
            for t in range(P, 140)]
    ro, rs = L.attn(c.q, c.k, c.v, c.alpha, c.s0)
    G.assert_rel(G.f64(torch.cat([o, torch.stack(rest, 1)], 1)), ro, BAR["bf16"], "prompt and steps")
    G.assert_rel(G.f64(state), rs, 1e-6, "state behind them")


def test_equals_the_delta_rule_without_erase():
    """gdn2_chunk_fwd with b = 0, w = 1 and the decay in every channel is the same layer."""
    import torch

    c = Case(630, 2, 300, 4, 128, 128, "bf16", alpha=[0.99, 0.9, 1.0, 0.97])
    o, s = c.fwd()
    one = torch.ones_like(c.t["v"])
    wide = c.t["alpha"][:, None].expand(2, 300, 4, 128).contiguous()
    o2, s2 = binding.gdn2_chunk_fwd(c.t["q"], c.t["k"], c.t["v"], wide, torch.zeros_like(c.t["k"]), one, c.t_s0)
    torch.cuda.synchronize()
    G.assert_rel(G.f64(o), G.f64(o2), 1e-2, "linear attention against the delta rule")
    G.assert_rel(G.f64(s), G.f64(s2), 1e-2, "its states")


def test_training_shape_sampled_heads():
    """The training shape, whole chains of some (sequence, head)s; the same call gives the same bits."""
    import torch

    B, T, H, d = 8, 4096, 16, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    q, k, v, d_o = (torch.randn((B, T, H, d), generator=g, device="cuda").mul_(s).to(torch.bfloat16)
                    for s in (d ** -0.5, 1.0, 1.0, 1.0))
    alpha = torch.exp(-(2.0 ** (-8.0 * (torch.arange(H, device="cuda") + 1) / H)))
    o, s = binding.gdn2_linear_attn_fwd(q, k, v, alpha)
    got = binding.gdn2_linear_attn_bwd(q, k, v, alpha, d_o)
    again = binding.gdn2_linear_attn_bwd(q, k, v, alpha, d_o)
    assert torch.equal(o, binding.gdn2_linear_attn_fwd(q, k, v, alpha)[0])
    assert all(torch.equal(got[n], again[n]) for n in ("dq", "dk", "dv"))
    for b, h in ((0, 0), (3, 7), (7, 15)):
        f = [G.f64(x[b:b + 1, :, h:h + 1]) for x in (q, k, v)]
        a = G.f64(alpha[h:h + 1])
        ro, rs = L.attn(*f, a)
        G.assert_rel(G.f64(o[b:b + 1, :, h:h + 1]), ro, BAR["bf16"], f"training o ({b}, {h})")
        G.assert_rel(G.f64(s[b:b + 1, h:h + 1]), rs, 1e-6, f"training state ({b}, {h})")
        want = L.attn_grads(*f, a, G.f64(d_o[b:b + 1, :, h:h + 1]))
        for n in ("dq", "dk", "dv"):
            G.assert_rel(G.f64(got[n][b:b + 1, :, h:h + 1]), want[n], BAR["bf16"], f"training {n} ({b}, {h})")


def test_offsets_past_32_bits():
    """More than 2^32 elements a tensor.  With a decay of 1/2 nothing older than 200 tokens counts, so the ends of
    the last head are checked alone."""
    import torch

    T, H, d = 264000, 128, 128
    assert T * H * d > 1 << 32
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def make():
        x = torch.empty((1, T, H, d), dtype=torch.bfloat16, device="cuda")
        for i in range(0, T, 33000):
            x[:, i:i + 33000] = torch.randn((1, 33000, H, d), generator=g, device="cuda")
        return x

    q, k, v = make(), make(), make()
    alpha = torch.full((H,), 0.5, device="cuda")
    o, s = binding.gdn2_linear_attn_fwd(q, k, v, alpha)
    got = binding.gdn2_linear_attn_bwd(q, k, v, alpha, v)
    torch.cuda.synchronize()
    for lo, keep in ((0, slice(0, 300)), (T - 700, slice(300, 700))):
        f = [G.f64(x[:, lo:lo + 700, -1:]) for x in (q, k, v)]
        ro, rs = L.attn(*f, [0.5])
        G.assert_rel(G.f64(o[:, lo:lo + 700, -1:])[:, keep], ro[:, keep], BAR["bf16"], f"o from {lo}")
        want = L.attn_grads(*f, [0.5], f[2])
        for n in ("dq", "dk", "dv"):
            G.assert_rel(G.f64(got[n][:, lo:lo + 700, -1:])[:, keep], want[n][:, keep], BAR["bf16"], f"{n} from {lo}")
        if lo:
            G.assert_rel(G.f64(s[:, -1:]), rs, 1e-6, "final state")


def test_captured_and_replayed():
    """Both directions and the step in one graph, replayed with new inputs between eager work."""
    import torch

    c = Case(640, 1, 1100, 2, 64, 64, "bf16", cu=[0, 400, 1100], alpha=[0.99, 0.9])
    state = c.t_s0.clone()
    tok = {n: torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda") for n in "qkv"}

    def work():
        o, s = binding.gdn2_linear_attn_fwd(**c.t, initial_state=c.t_s0, cu_seqlens=c.t_cu)
        g = binding.gdn2_linear_attn_bwd(**c.t, d_o=c.t_do, initial_state=c.t_s0, d_final_state=c.t_ds, cu_seqlens=c.t_cu,
                                         output_d_initial_state=True)
        y = binding.gdn2_linear_attn_step(**tok, alpha=c.t["alpha"], state=state)
        return [o, s, *g.values(), y]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for turn in range(4):
        r = Case(650 + turn, 1, 1100, 2, 64, 64, "bf16", cu=[0, 100 + 200 * turn, 1100], alpha=[0.99, 0.9])
        for n in ("q", "k", "v"):
            c.t[n].copy_(r.t[n])
            tok[n].copy_(r.t[n][0, :2])
        c.t_do.copy_(r.t_do)
        c.t_cu.copy_(r.t_cu)
        c.t_s0.copy_(r.t_s0)
        c.t_ds.copy_(r.t_ds)
        start = r.t_s0.clone()
        state.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        got, after = [x.clone() for x in outs], state.clone()
        state.copy_(start)
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(after, state)


def test_two_streams():
    """Calls side by side on two streams, each with its own workspace, give what they give alone."""
    import torch

    cases = [Case(660 + i, 1, 1500, 2, 128, 128, "bf16") for i in range(2)]
    want = [(c.fwd(), c.bwd()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            a = binding.gdn2_linear_attn_fwd(**c.t, initial_state=c.t_s0, stream=s)
            b = binding.gdn2_linear_attn_bwd(**c.t, d_o=c.t_do, initial_state=c.t_s0, d_final_state=c.t_ds,
                                             output_d_initial_state=True, stream=s)
            got.append((a, b))
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(got, want):
            assert all(torch.equal(p, r) for p, r in zip(a, x)) and all(torch.equal(b[n], y[n]) for n in y)


def test_layer_forward_and_backward():
    """A layer's run as it is used: norm and rotation of q and k, attention, and back to the projections, against the
    same in 64 bits.  The bar adds the roundings of the bf16 tensors in between: q, k and o, then dq, dk and the
    results, each at most 2^-8 rms of what passes through it."""
    import torch

    r = np.random.default_rng(700)
    B, T, H, d = 2, 200, 3, 64
    xq, xk, v, d_o = (rnd(r, (B, T, H, d), "bf16") for _ in range(4))
    wq, wk = (1 + 0.2 * r.standard_normal(d)).astype(np.float32), (1 + 0.2 * r.standard_normal(d)).astype(np.float32)
    freq = (1e4 ** (-np.arange(0, d, 2) / d)).astype(np.float32)
    alpha = np.array([0.99, 0.9, 0.5], dtype=np.float32)
    t = {n: dev(x, "bf16") for n, x in dict(xq=xq, xk=xk, v=v, d_o=d_o).items()}
    how = dict(inv_freq=dev(freq), weight_q=dev(wq), weight_k=dev(wk), q_scale=d ** -0.5)
    q, k = binding.gdn2_qk_norm_rope(t["xq"], t["xk"], **how)
    o, _ = binding.gdn2_linear_attn_fwd(q, k, t["v"], dev(alpha))
    g = binding.gdn2_linear_attn_bwd(q, k, t["v"], dev(alpha), t["d_o"])
    back = binding.gdn2_qk_norm_rope_bwd(t["xq"], t["xk"], g["dq"], g["dk"], **how)
    torch.cuda.synchronize()
    pos = np.broadcast_to(np.arange(T), (B, T))
    rq, rk = (L.norm_rope(x, w, s, pos, freq, 1e-6, False)[0] for x, w, s in ((xq, wq, d ** -0.5), (xk, wk, 1.0)))
    ro, _ = L.attn(rq, rk, v, alpha)
    rg = L.attn_grads(rq, rk, v, alpha, d_o)
    bar = 2 * 2.0 ** -8
    G.assert_rel(G.f64(o), ro, bar, "layer o")
    G.assert_rel(G.f64(g["dv"]), rg["dv"], bar, "layer dv")
    for n, x, w, s in (("q", xq, wq, d ** -0.5), ("k", xk, wk, 1.0)):
        (dx, _), (dw, _) = L.norm_rope_grads(x, w, s, pos, freq, 1e-6, False, rg["d" + n])
        G.assert_rel(G.f64(back["d_" + n]), dx, bar, f"layer d_{n}")
        G.assert_rel(G.f64(back["d_weight_" + n]), dw, bar, f"layer d_weight_{n}")
