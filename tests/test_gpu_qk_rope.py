"""GPU parity of the norms of queries and keys with the position rotation (gdn2_qk_norm_rope, _bwd) against the FP64
oracle in oracle/linear.py, element by element: its FP32 bound and half a step of the output's type."""
import numpy as np
import pytest

import gpu_util as G
from delta_rule_linear_gdn2_amd import binding
from oracle import linear as L
from test_gpu_linear import HALF, dev, rnd

pytestmark = pytest.mark.gpu
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    yield


def close(got, want, dtype, what):
    ref, bound = want
    x = G.f64(got)
    assert x.shape == ref.shape, f"{what}: {x.shape} != {ref.shape}"
    room = bound + HALF[dtype] * (np.abs(ref) + bound) + 1e-37
    bad = ~(np.abs(x - ref) <= room)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}"


class Case:
    def __init__(self, seed, B, T, Hq, Hk, d, rot, dtype, interleaved=False, weights=True, positions="far", scale=0.125):
        import torch

        r = np.random.default_rng(seed)
        self.dtype, self.eps = dtype, EPS
        self.x = {"q": rnd(r, (B, T, Hq, d), dtype, 2.0), "k": rnd(r, (B, T, Hk, d), dtype, 0.5)}
        self.dy = {"q": rnd(r, (B, T, Hq, d), dtype), "k": rnd(r, (B, T, Hk, d), dtype)}
        self.w = {n: (1 + 0.3 * r.standard_normal(d)).astype(np.float32) if weights else None for n in "qk"}
        self.freq = (1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32) if rot else None
        self.scale = {"q": float(np.float32(scale)), "k": 1.0}
        self.interleaved = interleaved
        at = {"far": lambda: r.integers(-(1 << 20), 1 << 20, (B, T)), "index": lambda: np.broadcast_to(np.arange(T), (B, T)),
              "ends": lambda: r.choice([0, -1, (1 << 31) - 1, -(1 << 31), 1 << 24], (B, T))}[positions]()
        self.pos = np.ascontiguousarray(at).astype(np.int32)
        self.t = {n: dev(x, dtype) for n, x in self.x.items()}
        self.how = dict(inv_freq=dev(self.freq), weight_q=dev(self.w["q"]), weight_k=dev(self.w["k"]), q_scale=scale,
                        interleaved=interleaved,
                        positions=None if positions == "index" else torch.from_numpy(self.pos).cuda())
        self.t_dy = [dev(self.dy[n], dtype) for n in "qk"]

    def fwd(self, **kw):
        import torch

        out = binding.gdn2_qk_norm_rope(self.t["q"], self.t["k"], **self.how, **kw)
        torch.cuda.synchronize()
        return out

    def bwd(self, **kw):
        import torch

        out = binding.gdn2_qk_norm_rope_bwd(self.t["q"], self.t["k"], *self.t_dy, **self.how, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, what):
        got = dict(zip("qk", self.fwd()))
        back = self.bwd()
        for n in "qk":
            how = (self.x[n], self.w[n], self.scale[n], self.pos, self.freq, EPS, self.interleaved)
            close(got[n], L.norm_rope(*how), self.dtype, f"{what} {n}")
            dx, dw = L.norm_rope_grads(*how, self.dy[n])
            close(back["d_" + n], dx, self.dtype, f"{what} d_{n}")
            if self.w[n] is None:
                assert back["d_weight_" + n] is None
            else:
                close(back["d_weight_" + n], dw, "f32", f"{what} d_weight_{n}")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,rot", [(d, r) for d in (32, 64, 128) for r in (0, 8, 24, d // 2, d - 8, d)])
def test_sizes(d, rot, dtype, interleaved):
    Case(d + rot, 2, 9, 5, 3, d, rot, dtype, interleaved).check(f"{dtype} d={d} rot={rot} {interleaved}")


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 4), (16, 2), (7, 1), (33, 5), (1, 9)])
@pytest.mark.parametrize("d", [32, 128])
def test_heads(Hq, Hk, d):
    """Head counts that fill a wavefront's rows and that do not."""
    Case(100 + Hq, 1, 11, Hq, Hk, d, d, "bf16").check(f"heads {Hq}, {Hk} d={d}")


@pytest.mark.parametrize("B,T", [(1, 1), (3, 1), (1, 2), (5, 7), (2, 513), (1, 4100)])
def test_tokens(B, T):
    """One token; fewer tokens than wavefronts; more than one round of them (4096 wavefronts)."""
    Case(200 + T, B, T, 3, 2, 64, 32, "bf16", positions="index").check(f"tokens {B} x {T}")
    Case(210 + T, B, T, 6, 2, 32, 32, "f32", weights=False, positions="index", scale=1.0).check(f"tokens {B} x {T} f32")


@pytest.mark.parametrize("d", [32, 64, 128])
def test_positions_at_the_ends(d):
    Case(300 + d, 2, 40, 2, 2, d, d, "f32", positions="ends").check(f"positions at the ends d={d}")


def test_ends_of_the_range():
    """Rows of zeros, of tiny and of huge values: 1 / rms is never raised to a power."""
    import torch

    c = Case(320, 1, 6, 2, 2, 64, 64, "f32", positions="index")
    for n in "qk":
        for i, s in enumerate((0.0, 1e-20, 1e-4, 1.0, 1e12, 1e17)):
            c.x[n][:, i] *= np.float32(s)
        c.t[n] = dev(c.x[n])
    c.check("ends of the range")
    c.how["q_scale"], c.scale["q"] = 0.0, 0.0
    assert not c.fwd()[0].any()
    assert torch.isfinite(c.bwd()["d_q"]).all()


def test_non_finite_rows_stay_alone():
    import torch

    c = Case(330, 1, 20, 4, 2, 64, 32, "bf16")
    ref = c.fwd()
    c.t["q"][0, 7, 2, 5] = float("inf")
    c.t["k"][0, 9, 1, 60] = float("nan")
    q, k = c.fwd()
    same_q, same_k = (q == ref[0]).all(-1), (k == ref[1]).all(-1)
    assert (~same_q).nonzero().tolist() == [[0, 7, 2]] and (~same_k).nonzero().tolist() == [[0, 9, 1]]
    assert torch.isnan(k[0, 9, 1]).all()
    # a row's infinity is divided by itself; the others by it
    assert torch.isnan(q[0, 7, 2]).sum() <= 2 and (q[0, 7, 2][~torch.isnan(q[0, 7, 2])] == 0).all()


def test_in_place_and_given_outputs():
    import torch

    for dtype in ("bf16", "f32"):
        c = Case(340, 2, 50, 6, 2, 64, 48, dtype)
        q, k = c.fwd()
        mine = torch.empty_like(q), torch.empty_like(k)
        got = c.fwd(q_out=mine[0], k_out=mine[1])
        assert got[0] is mine[0] and got[1] is mine[1] and torch.equal(got[0], q) and torch.equal(got[1], k)
        xq, xk = c.t["q"], c.t["k"]
        a, b = c.fwd(q_out=xq, k_out=xk)
        assert a is xq and b is xk and torch.equal(a, q) and torch.equal(b, k)


def test_wanted_gradients_only():
    import torch

    c = Case(350, 2, 300, 6, 2, 128, 128, "bf16")
    full = c.bwd()
    part = c.bwd(want_d_weights=False)
    assert part["d_weight_q"] is None and part["d_weight_k"] is None
    assert torch.equal(part["d_q"], full["d_q"]) and torch.equal(part["d_k"], full["d_k"])
    c.how["weight_k"] = None
    one = c.bwd()
    assert one["d_weight_k"] is None and torch.equal(one["d_weight_q"], full["d_weight_q"])
    again = c.bwd()
    assert torch.equal(one["d_weight_q"], again["d_weight_q"])


def test_no_tokens():
    import torch

    c = Case(360, 2, 0, 3, 2, 64, 64, "bf16", positions="index")
    q, k = c.fwd()
    assert q.numel() == 0 and k.numel() == 0
    got = c.bwd()
    torch.cuda.synchronize()
    assert not got["d_weight_q"].any() and not got["d_weight_k"].any()


def test_offsets_past_32_bits():
    """More than 2^32 elements of q: the last token against the same row alone."""
    import torch

    T, H, d = 262200, 128, 128
    assert T * H * d > 1 << 32
    q = torch.empty((1, T, H, d), dtype=torch.bfloat16, device="cuda").normal_()
    k = torch.empty((1, T, 1, d), dtype=torch.bfloat16, device="cuda").normal_()
    freq = torch.full((64,), 0.01, device="cuda")
    qo, ko = binding.gdn2_qk_norm_rope(q, k, freq)
    got = binding.gdn2_qk_norm_rope_bwd(q, k, qo, ko, freq)
    at = torch.tensor([[T - 1]], dtype=torch.int32, device="cuda")
    one = [x[:, -1:].contiguous() for x in (q, k, qo, ko)]
    a, b = binding.gdn2_qk_norm_rope(one[0], one[1], freq, positions=at)
    g = binding.gdn2_qk_norm_rope_bwd(*one, freq, positions=at)
    torch.cuda.synchronize()
    assert torch.equal(qo[:, -1:], a) and torch.equal(ko[:, -1:], b)
    assert torch.equal(got["d_q"][:, -1:], g["d_q"]) and torch.equal(got["d_k"][:, -1:], g["d_k"])


def test_captured_and_replayed():
    import torch

    c = Case(370, 2, 300, 6, 2, 64, 64, "bf16")

    def work():
        q, k = binding.gdn2_qk_norm_rope(c.t["q"], c.t["k"], **c.how)
        return [q, k, *binding.gdn2_qk_norm_rope_bwd(c.t["q"], c.t["k"], *c.t_dy, **c.how).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for turn in range(4):
        r = Case(380 + turn, 2, 300, 6, 2, 64, 64, "bf16")
        for n in "qk":
            c.t[n].copy_(r.t[n])
        for a, b in zip(c.t_dy, r.t_dy):
            a.copy_(b)
        c.how["positions"].copy_(r.how["positions"])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_another_stream():
    import torch

    c = Case(390, 4, 500, 8, 8, 128, 128, "bf16")
    want, wb = c.fwd(), c.bwd()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, k = binding.gdn2_qk_norm_rope(c.t["q"], c.t["k"], **c.how, stream=s)
    g = binding.gdn2_qk_norm_rope_bwd(c.t["q"], c.t["k"], *c.t_dy, **c.how, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and all(torch.equal(g[n], wb[n]) for n in wb)
