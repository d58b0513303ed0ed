"""Rounding of linear attention with a fixed decay for each head, where single products can be told apart
(needs an MI355X).

FP32 operands are three bf16 terms x0 + x1 + x2 and a product six of the nine.  Rounded to nearest, x1 is at most
2^-8 and x2 at most 2^-17 of a value in [1, 2), so the three products left out are below 2 x 2^-25 + 2^-34.  The
six are added in FP32: the last addition is off by at most 2 U (U = 2^-24; half that if rounded to nearest), the
others, of terms 2^-7 of the product, by 4 x 2^-7 x 2 U.  Together less than 3.1 U of a product."""
import numpy as np
import pytest

from delta_rule_linear_gdn2_amd import binding
from oracle import linear as L
from test_gpu_linear import dev, gpu  # noqa: F401

pytestmark = pytest.mark.gpu
U = L.U
PRODUCT = 3.1 * U


def full_mantissas(r, shape):
    """FP32 values with all of their low bits in use: half of them drawn evenly, half right below where a bf16
    ends, so that cut off terms leave as much as they can."""
    even = 1 + r.integers(0, 1 << 23, shape) * 2.0 ** -23
    below = 1 + (r.integers(1, 128, shape) * 2.0 ** -7 - r.integers(1, 4, shape) * 2.0 ** -23)
    x = np.where(r.random(shape) < 0.5, even, below) * np.exp2(r.integers(-3, 4, shape)) * r.choice([-1.0, 1.0], shape)
    return x.astype(np.float32)


@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 32)])
def test_fp32_products(dk, dv):
    """One token whose query has one channel: o = (q_c k_c) v, two products behind one another, and the state k v^T,
    one."""
    r = np.random.default_rng(dk + dv)
    B, H = 48, 3
    q, k, v = np.zeros((B, 1, H, dk), dtype=np.float32), full_mantissas(r, (B, 1, H, dk)), full_mantissas(r, (B, 1, H, dv))
    at = r.integers(0, dk, (B, 1, H, 1))
    np.put_along_axis(q, at, full_mantissas(r, (B, 1, H, 1)), -1)
    o, s = binding.gdn2_linear_attn_fwd(dev(q), dev(k), dev(v), dev(np.ones(H)))
    ro, rs = L.attn(q, k, v, np.ones(H))
    o, s = o.double().cpu().numpy(), s.double().cpu().numpy()
    assert (np.abs(s - rs) <= PRODUCT * np.abs(rs)).all(), f"state off by {(np.abs(s / rs - 1)).max() / U:.1f} U"
    assert (np.abs(o - ro) <= 2 * PRODUCT * np.abs(ro)).all(), f"o off by {(np.abs(o / ro - 1)).max() / U:.1f} U"
