"""What lies around the outputs and workspaces of linear attention and of the q, k norm with rotation stays as it was,
what a workspace holds on entry does not matter, and its queried size is enough (needs an MI355X).  Outputs and
workspaces stand between guard bands, full of NaN; the results are those of the default calls, bit for bit."""
import numpy as np
import pytest

from delta_rule_linear_gdn2_amd import binding
from test_gpu_linear import Case, dev, gpu  # noqa: F401
from test_gpu_qk_rope import Case as RopeCase

pytestmark = pytest.mark.gpu
BAND, MARK = 4096, 0xA5  # bytes; a mark that no output is made of


class Guarded:
    """Tensors between bands of bytes, filled with NaN."""

    def __init__(self):
        self.flats = []

    def bytes(self, n):
        import torch

        flat = torch.full((n + 2 * BAND,), MARK, dtype=torch.uint8, device="cuda")
        flat[BAND:BAND + n] = 0xFF
        self.flats.append((flat, n))
        return flat[BAND:BAND + n]

    def like(self, shape, dtype):
        import torch

        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        return self.bytes(n).view(dtype).view(shape)

    def check(self, what):
        for i, (flat, n) in enumerate(self.flats):
            for side, band in (("before", flat[:BAND]), ("behind", flat[BAND + n:])):
                assert (band == MARK).all(), f"{what}: buffer {i} written {side} it"


def addr(t):
    return None if t is None else t.data_ptr()


def run(name, *args):
    import torch

    rc = getattr(binding.load(), name)(*args, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == binding.GDN2_OK, f"{name}: {rc}"


def sizes(c):
    B, T, H, dk = c.t["q"].shape
    return B, T, H, dk, c.t["v"].shape[3], 0 if c.cu is None else len(c.cu) - 1


def fwd(g, c, code, in_place, wanted=True, segmented=True, zero=1):
    import torch

    B, T, H, dk, dv, packed = sizes(c)
    o = g.like(c.t["v"].shape, c.t["v"].dtype)
    s0, s = c.t_s0, None
    if in_place:
        s = g.like(s0.shape, torch.float32)
        s.copy_(s0)
        s0 = s
    elif wanted:
        s = g.like((packed or B, H, dk, dv), torch.float32)
    need = binding.gdn2_linear_attn_fwd_workspace_bytes(B, T, H, dk, dv, packed, code) if segmented else 0
    ws = g.bytes(need) if need else None
    run("gdn2_linear_attn_fwd", *[addr(c.t[n]) for n in ("q", "k", "v", "alpha")], addr(s0), addr(s), addr(o), addr(c.t_cu),
        B, T, H, dk, dv, packed, zero, code, addr(ws), need)
    return o, s, need


def bwd(g, c, code, wanted=True, segmented=True, zero=1):
    import torch

    B, T, H, dk, dv, packed = sizes(c)
    out = [g.like(c.t[n].shape, c.t[n].dtype) for n in ("q", "k", "v")]
    out.append(g.like((packed or B, H, dk, dv), torch.float32) if wanted else None)
    need = binding.gdn2_linear_attn_bwd_workspace_bytes(B, T, H, dk, dv, packed, code) if segmented else 0
    ws = g.bytes(need) if need else None
    run("gdn2_linear_attn_bwd", *[addr(c.t[n]) for n in ("q", "k", "v", "alpha")], addr(c.t_s0), addr(c.t_do), addr(c.t_ds),
        *map(addr, out), addr(c.t_cu), B, T, H, dk, dv, packed, zero, code, addr(ws), need)
    return dict(zip(("dq", "dk", "dv", "d_initial_state"), out)), need


def equal(a, b, what):
    import torch

    assert torch.equal(a, b), f"{what} differs"


SHAPES = [(1, 1, 1, 32, 32, None), (2, 5, 3, 64, 128, None), (1, 100, 2, 128, 64, None), (3, 191, 1, 32, 64, None),
          (1, 1300, 2, 128, 128, None), (2, 1111, 1, 64, 32, None), (1, 1500, 1, 32, 128, None),
          (1, 2500, 2, 64, 128, [0, 0, 700, 701, 701, 2100, 2163, 2500]), (1, 2501, 1, 128, 64, [0, 1300, 1301, 2501]),
          (1, 1900, 1, 32, 32, [0] * 90 + [1, 700, 900, 1900]), (1, 1700, 2, 128, 32, [30, 400, 1600, 1650])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv,cu", SHAPES)
def test_attention(B, T, H, dk, dv, cu, dtype):
    c, code = Case(900 + T, B, T, H, dk, dv, dtype, cu=cu, alpha=[0.97, 0.8, 1.0][:H]), int(dtype == "bf16")
    what = f"{dtype} {B}x{T}x{H} {dk}x{dv} {'packed' if cu else ''}"
    for segmented in (True, False):
        ro, rs = c.fwd(segmented=segmented)
        ref = c.bwd(segmented=segmented)
        for in_place in (False, True):
            g = Guarded()
            o, s, need = fwd(g, c, code, in_place, segmented=segmented)
            assert not segmented or T < 1000 or need > 0
            g.check(f"{what} forward, in place {in_place}")
            equal(o, ro, f"{what} o")
            equal(s, rs, f"{what} final state")
        g = Guarded()
        got, _ = bwd(g, c, code, segmented=segmented)
        g.check(f"{what} backward")
        for n in ref:
            equal(got[n], ref[n], f"{what} {n}")
        # without the states, whose walks take fewer terms
        o = c.fwd(segmented=segmented, output_final_state=False)[0]
        g = Guarded()
        equal(fwd(g, c, code, False, wanted=False, segmented=segmented)[0], o, f"{what} o without a state")
        g.check(f"{what} forward without a state")
        g = Guarded()
        got, _ = bwd(g, c, code, wanted=False, segmented=segmented)
        g.check(f"{what} backward without a state")
        equal(got["dv"], binding.gdn2_linear_attn_bwd(**c.t, d_o=c.t_do, initial_state=c.t_s0, d_final_state=c.t_ds,
                                                      cu_seqlens=c.t_cu, segmented=segmented)["dv"], f"{what} dv without a state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_no_sequence_stay(dtype):
    """Without zero_padding the rows around packed sequences are left as they were, in every output."""
    c, code = Case(930, 1, 300, 2, 64, 32, dtype, cu=[11, 100, 250]), int(dtype == "bf16")
    g = Guarded()
    o, _, _ = fwd(g, c, code, False, zero=0)
    got, _ = bwd(g, c, code, zero=0)
    g.check(f"{dtype} rows of no sequence")
    import torch

    for x in (o, got["dq"], got["dk"], got["dv"]):
        rows = x[0].flatten(1).view(torch.uint8)
        assert (rows[:11] == 0xFF).all() and (rows[250:] == 0xFF).all() and torch.isfinite(x[:, 11:250]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 32), (32, 128)])
def test_malformed_offsets(dk, dv, dtype):
    """Offsets out of range or falling: results without meaning, inside the tensors and the workspace."""
    import torch

    c, code = Case(940, 1, 1400, 2, dk, dv, dtype, cu=[0, 300, 900, 1400]), int(dtype == "bf16")
    for cu in ([-5, 900, 5000, 1400], [0, 1250, 100, 1400], [1400, 0, 1400, 0], [0, 1 << 30, -(1 << 30), 1400],
               [1399, 1400, 1401, -1], [700, 700, 0, 0], [(1 << 31) - 1, -(1 << 31), (1 << 31) - 1, -(1 << 31)]):
        c.t_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for segmented in (True, False):
            for in_place in (False, True):
                g = Guarded()
                need = fwd(g, c, code, in_place, segmented=segmented)[2]
                assert (need > 0) == segmented
                g.check(f"forward {cu}")
            g = Guarded()
            bwd(g, c, code, segmented=segmented)
            bwd(g, c, code, wanted=False, segmented=segmented, zero=0)
            g.check(f"backward {cu}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,dk,dv", [(1, 1, 32, 32), (3, 5, 64, 32), (7, 3, 128, 64), (9, 1, 32, 128), (2, 4, 128, 128)])
def test_step(N, H, dk, dv, dtype):
    import torch

    c, code = Case(950 + N, N, 1, H, dk, dv, dtype), int(dtype == "bf16")
    row = {n: c.t[n][:, 0].contiguous() for n in ("q", "k", "v")}
    want_s = c.t_s0.clone()
    want_o = binding.gdn2_linear_attn_step(**row, alpha=c.t["alpha"], state=want_s)
    g = Guarded()
    s, o = g.like(c.t_s0.shape, torch.float32), g.like(row["v"].shape, row["v"].dtype)
    s.copy_(c.t_s0)
    run("gdn2_linear_attn_step", *[addr(row[n]) for n in ("q", "k", "v")], addr(c.t["alpha"]), addr(s), addr(o), N, H, dk, dv, code)
    g.check(f"{dtype} step {N}x{H} {dk}x{dv}")
    equal(o, want_o, "o")
    equal(s, want_s, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", [(1, 1, 1, 1, 32, 32), (2, 9, 5, 3, 64, 24), (1, 501, 11, 3, 64, 48), (3, 7, 33, 1, 128, 128),
                                             (1, 4100, 1, 2, 32, 8), (2, 3, 2, 9, 128, 0)])
def test_norm_and_rotation(B, T, Hq, Hk, d, rot, dtype):
    import torch

    c, code = RopeCase(960 + T, B, T, Hq, Hk, d, rot, dtype), int(dtype == "bf16")
    q, k = c.fwd()
    want = c.bwd()
    ins = [addr(c.t["q"]), addr(c.t["k"]), addr(c.how["weight_q"]), addr(c.how["weight_k"]), addr(c.how["inv_freq"]),
           addr(c.how["positions"])]
    tail = [B, T, Hq, Hk, d, rot, 0, 0.125, 1e-6, code]
    g = Guarded()
    out = [g.like(x.shape, x.dtype) for x in (q, k)]
    run("gdn2_qk_norm_rope", *ins, *map(addr, out), *tail)
    g.check(f"{dtype} norm and rotation")
    equal(out[0], q, "q")
    equal(out[1], k, "k")
    need = binding.gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d)
    for weights in (True, False):
        g = Guarded()
        out = [g.like(x.shape, x.dtype) for x in (q, k)]
        dw = [g.like((d,), torch.float32) if weights else None for _ in range(2)]
        ws = g.bytes(need) if weights else None
        run("gdn2_qk_norm_rope_bwd", *ins, *map(addr, c.t_dy), *map(addr, out), *map(addr, dw), *tail, addr(ws), need if weights else 0)
        g.check(f"{dtype} norm and rotation backward")
        equal(out[0], want["d_q"], "d_q")
        equal(out[1], want["d_k"], "d_k")
        if weights:
            equal(dw[0], want["d_weight_q"], "d_weight_q")
            equal(dw[1], want["d_weight_k"], "d_weight_k")
