"""What a NaN or an infinity in linear attention with a fixed decay reaches (needs an MI355X): what the recurrence
lets it reach, and nothing else, bit for bit.  A token's value reaches its own output and the later ones (in the
gradients of k and v the earlier ones), also where it stands in the same chunk, tile or operand as tokens that come
before it."""
import numpy as np
import pytest

from test_gpu_linear import Case, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

CU = [0, 150, 310]  # the poisoned sequence is the second, its length no multiple of a tile
PLACES = [0, 1, 14, 15, 16, 31, 33, 47, 48, 62, 63, 64, 80, 127, 128, 130, 159]


def same(a, b):
    return (a == b).cpu().numpy()


def reach_fwd(name, n, lo, hi, at, h, c, o, s):
    """Masks of what may differ: o [B, T, H, dv], states [N, H, dk, dv]."""
    mo, ms = np.zeros(o, dtype=bool), np.zeros(s, dtype=bool)
    if name == "q":
        mo[0, lo + at, h] = True
    elif name == "k":
        mo[0, lo + at:hi, h] = ms[n, h, c] = True
    else:
        mo[0, lo + at:hi, h, c] = ms[n, h, :, c] = True
    return {"o": mo, "s": ms}


def reach_bwd(name, n, lo, hi, at, h, c, dk, dv, s):
    """Masks over dq, dk, dv and d_initial_state."""
    m = {"dq": np.zeros(dk, dtype=bool), "dk": np.zeros(dk, dtype=bool), "dv": np.zeros(dv, dtype=bool),
         "d_initial_state": np.zeros(s, dtype=bool)}
    here, on, back = (0, lo + at, h), (0, slice(lo + at, hi), h), (0, slice(lo, lo + at + 1), h)
    if name == "q":     # dk = sum of R's rows q, dv = (R^T k): q from the token on back
        m["dk"][(*back, c)] = m["dv"][back] = m["d_initial_state"][n, h, c] = True
    elif name == "k":
        m["dq"][(*on, c)] = m["dv"][here] = True
    elif name == "v":
        m["dq"][on] = m["dk"][here] = True
    else:
        m["dq"][here] = m["dk"][back] = m["dv"][(*back, c)] = m["d_initial_state"][n, h, :, c] = True
    return m


def compare(got, want, masks, what):
    for k, mask in masks.items():
        eq = same(got[k], want[k])
        stray = ~eq & ~mask
        assert not stray.any(), f"{what}: {k} differs at {np.argwhere(stray)[:3].tolist()} ({stray.sum()} places)"
        finite = np.isfinite(got[k].float().cpu().numpy()) & mask
        assert not finite.any(), f"{what}: {k} finite at {np.argwhere(finite)[:3].tolist()} ({finite.sum()} places)"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 64), (64, 32), (128, 32)])
@pytest.mark.parametrize("segmented", [True, False])
def test_reach(dk, dv, dtype, segmented):
    import torch

    c = Case(800 + dk + dv, 1, CU[-1], 2, dk, dv, dtype, cu=CU, alpha=[0.9, 0.98])
    # the recurrence multiplies by every value, a zero times a NaN included: no factor hides one
    clean_o, clean_s = c.fwd(segmented=segmented)
    clean_g = c.bwd(segmented=segmented)
    n, lo, hi, h = 1, CU[1], CU[2], 1
    inputs = {"q": c.t["q"], "k": c.t["k"], "v": c.t["v"], "d_o": c.t_do}
    for name, t in inputs.items():
        for i, at in enumerate(PLACES):
            value = [float("nan"), float("inf"), float("-inf")][i % 3]
            col = (7 * at + 3) % t.shape[-1]
            old = t[0, lo + at, h, col].clone()
            t[0, lo + at, h, col] = value
            what = f"{dtype} {dk}x{dv} {name} = {value} at {at}"
            if name != "d_o":
                o, s = c.fwd(segmented=segmented)
                compare({"o": o, "s": s}, {"o": clean_o, "s": clean_s},
                        reach_fwd(name, n, lo, hi, at, h, col, o.shape, s.shape), what)
            g = c.bwd(segmented=segmented)
            compare(g, clean_g, reach_bwd(name, n, lo, hi, at, h, col, g["dq"].shape, g["dv"].shape,
                                          g["d_initial_state"].shape), what + " backward")
            t[0, lo + at, h, col] = old
    o, s = c.fwd(segmented=segmented)
    assert torch.equal(o, clean_o) and torch.equal(s, clean_s)


def test_padded_batch():
    """Rows behind a prompt's end that hold anything leave the prompt's own outputs as they are."""
    import torch

    c = Case(850, 3, 100, 2, 64, 64, "bf16", state=False)
    lengths = [37, 64, 99]
    want = []
    for b, n in enumerate(lengths):
        d = Case(850, 3, 100, 2, 64, 64, "bf16", state=False)
        for x in d.t.values():
            if x.dim() == 4:
                x[b, n:] = 0
        want.append(d.fwd()[0][b, :n].clone())
        for x in ("q", "k", "v"):
            c.t[x][b, n:] = float("nan")
    o, _ = c.fwd()
    for b, n in enumerate(lengths):
        assert torch.equal(o[b, :n], want[b])
        assert torch.isnan(o[b, n:]).all()
