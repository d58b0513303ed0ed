"""Refusals of linear attention with a fixed decay and of the q, k norm with rotation
on a machine without a GPU: the C ABI rejects bad arguments before any HIP call, the
binding before the C call."""
import inspect

import pytest
import torch

from delta_rule_linear_gdn2_amd import binding
from test_abi_cpu import ALIAS, DTYPE, MISAL, NULLP, OK, SHAPE, UNSUP, WS, fake, lib  # noqa: F401
from test_training_cpu import call

# B=1, T=4096, H=4, d=64, bf16: [B, T, H, d] is 2 MiB, the states 64 KiB; 256 compute units: 16 segments of 256 tokens
FWD = dict(q=fake(0), k=fake(1), v=fake(2), alpha=fake(3), s0=fake(4), sf=fake(5), o=fake(6), cu=None, B=1, T=4096, H=4,
           dk=64, dv=64, num_seqs=0, zero=0, dtype=1, ws=fake(7), ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=2), DTYPE),
    (dict(dtype=-1), DTYPE),
    (dict(B=0), SHAPE),
    (dict(T=-1), SHAPE),
    (dict(H=0), SHAPE),
    (dict(H=(1 << 15) + 1), SHAPE),
    (dict(B=1 << 30, T=1 << 30), SHAPE),
    (dict(cu=fake(8), num_seqs=0), SHAPE),
    (dict(cu=fake(8), B=2, num_seqs=3), SHAPE),
    (dict(dk=48), UNSUP),
    (dict(dv=256), UNSUP),
    (dict(q=None), NULLP),
    (dict(k=None), NULLP),
    (dict(v=None), NULLP),
    (dict(o=None), NULLP),
    (dict(alpha=None), NULLP),
    (dict(T=0, alpha=None), NULLP),
    (dict(q=fake(0, 8)), MISAL),
    (dict(sf=fake(5, 4)), MISAL),
    (dict(alpha=fake(3, 2)), MISAL),
    (dict(cu=fake(8, 2), num_seqs=2), MISAL),
    (dict(ws=fake(7, 8)), MISAL),
    (dict(ws_bytes=16), WS),
    (dict(o=fake(2)), ALIAS),
    (dict(o=fake(0, 16)), ALIAS),
    (dict(o=fake(3)), ALIAS),
    (dict(sf=fake(4, 16)), ALIAS),                # the final state inside the initial one, not it itself
    (dict(sf=fake(1)), ALIAS),
    (dict(sf=fake(6, 1 << 20)), ALIAS),
    (dict(ws=fake(6)), ALIAS),
    (dict(ws=fake(4)), ALIAS),
    (dict(cu=fake(6, 64), num_seqs=2), ALIAS),
])
def test_linear_attn_fwd_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_linear_attn_fwd, list(FWD), FWD, kw) == expected


BWD = dict(q=fake(0), k=fake(1), v=fake(2), alpha=fake(3), s0=fake(4), d_o=fake(5), dsf=fake(6), dq=fake(7), dk_=fake(8),
           dv_=fake(9), ds0=fake(10), cu=None, B=1, T=4096, H=4, dk=64, dv=64, num_seqs=0, zero=0, dtype=1, ws=fake(11),
           ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=3), DTYPE),
    (dict(B=-1), SHAPE),
    (dict(H=1 << 16), SHAPE),
    (dict(cu=fake(12), num_seqs=-1), SHAPE),
    (dict(dv=16), UNSUP),
    (dict(d_o=None), NULLP),
    (dict(dq=None), NULLP),
    (dict(dv_=None), NULLP),
    (dict(alpha=None), NULLP),
    (dict(d_o=fake(5, 2)), MISAL),
    (dict(ds0=fake(10, 8)), MISAL),
    (dict(ws_bytes=1024), WS),
    (dict(dq=fake(0)), ALIAS),
    (dict(dk_=fake(7)), ALIAS),
    (dict(dv_=fake(5)), ALIAS),
    (dict(ds0=fake(6)), ALIAS),                   # one walk reads d_final_state while another writes
    (dict(ds0=fake(4)), ALIAS),
    (dict(ws=fake(9, 256)), ALIAS),
    (dict(ws=fake(2)), ALIAS),
])
def test_linear_attn_bwd_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_linear_attn_bwd, list(BWD), BWD, kw) == expected


STEP = dict(q=fake(0), k=fake(1), v=fake(2), alpha=fake(3), state=fake(4), o=fake(5), N=8, H=4, dk=64, dv=64, dtype=1)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=2), DTYPE),
    (dict(N=-1), SHAPE),
    (dict(H=0), SHAPE),
    (dict(N=(1 << 31) - 1, H=1 << 20), SHAPE),
    (dict(dk=96), UNSUP),
    (dict(state=None), NULLP),
    (dict(alpha=None), NULLP),
    (dict(state=fake(4, 4)), MISAL),
    (dict(alpha=fake(3, 1)), MISAL),
    (dict(o=fake(2)), ALIAS),
    (dict(o=fake(4, 256)), ALIAS),
    (dict(state=fake(3)), ALIAS),
    (dict(N=0, q=None, k=None, v=None, alpha=None, state=None, o=None), OK),
])
def test_linear_attn_step_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_linear_attn_step, list(STEP), STEP, kw) == expected


QK = dict(q=fake(0), k=fake(1), wq=fake(2), wk=fake(3), freq=fake(4), pos=fake(5), qo=fake(6), ko=fake(7), B=2, T=100, Hq=8,
          Hk=2, d=64, rot=64, inter=0, scale=1.0, eps=1e-6, dtype=1)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=2), DTYPE),
    (dict(B=0), SHAPE),
    (dict(T=-1), SHAPE),
    (dict(Hq=0), SHAPE),
    (dict(Hk=(1 << 15) + 1), SHAPE),
    (dict(rot=66), SHAPE),
    (dict(rot=72), SHAPE),
    (dict(rot=-8), SHAPE),
    (dict(rot=12), SHAPE),
    (dict(rot=0), SHAPE),                         # frequencies without a rotation
    (dict(eps=0.0), SHAPE),
    (dict(eps=1e-39), SHAPE),
    (dict(eps=float("nan")), SHAPE),
    (dict(d=256), UNSUP),
    (dict(freq=None), NULLP),
    (dict(q=None), NULLP),
    (dict(ko=None), NULLP),
    (dict(q=fake(0, 8)), MISAL),
    (dict(wq=fake(2, 4)), MISAL),
    (dict(pos=fake(5, 2)), MISAL),
    (dict(qo=fake(0, 16)), ALIAS),                # inside q, not q itself
    (dict(qo=fake(1)), ALIAS),
    (dict(ko=fake(0)), ALIAS),
    (dict(ko=fake(6, 1024)), ALIAS),
    (dict(qo=fake(5)), ALIAS),
    (dict(ko=fake(2)), ALIAS),
    (dict(T=0, q=None, k=None, qo=None, ko=None), OK),
])
def test_qk_norm_rope_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_qk_norm_rope, list(QK), QK, kw) == expected


QKB = dict(q=fake(0), k=fake(1), wq=fake(2), wk=fake(3), freq=fake(4), pos=fake(5), dqo=fake(6), dko=fake(7), dq=fake(8),
           dk=fake(9), dwq=fake(10), dwk=fake(11), B=2, T=100, Hq=8, Hk=2, d=64, rot=64, inter=0, scale=1.0, eps=1e-6, dtype=1,
           ws=fake(12), ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=5), DTYPE),
    (dict(rot=20), SHAPE),
    (dict(wq=None), SHAPE),                       # the gradient of a weight that is not there
    (dict(wk=None), SHAPE),
    (dict(d=96), UNSUP),
    (dict(dqo=None), NULLP),
    (dict(dk=None), NULLP),
    (dict(ws=None), WS),
    (dict(ws_bytes=8), WS),
    (dict(dwk=fake(11, 4)), MISAL),
    (dict(ws=fake(12, 8)), MISAL),
    (dict(dq=fake(6)), ALIAS),
    (dict(dk=fake(8, 4096)), ALIAS),
    (dict(dwq=fake(2)), ALIAS),
    (dict(dwk=fake(10)), ALIAS),
    (dict(ws=fake(9)), ALIAS),
])
def test_qk_norm_rope_bwd_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_qk_norm_rope_bwd, list(QKB), QKB, kw) == expected


def test_workspace_queries(lib):  # noqa: F811
    """Plans for 256 compute units, as there is no device here."""
    fwd, bwd = binding.gdn2_linear_attn_fwd_workspace_bytes, binding.gdn2_linear_attn_bwd_workspace_bytes
    assert fwd(8, 4096, 16, 128, 128, 0, 1) == 0                  # enough sequences and heads
    one = fwd(1, 4096, 16, 128, 128, 0, 1)
    assert one > 0 and one % (16 * 128 * 128 * 4) == 0            # whole states of every head
    assert bwd(1, 4096, 16, 128, 128, 0, 1) > 0
    assert fwd(1, 64, 16, 128, 128, 0, 1) == 0                    # one chunk
    assert fwd(1, 0, 16, 128, 128, 0, 1) == fwd(1, 0, 16, 128, 128, 3, 1) == 0
    for bad in ((0, 64, 4, 64, 64, 0), (1, -1, 4, 64, 64, 0), (1, 64, 4, 48, 64, 0), (1, 64, 4, 64, 64, -2),
                (1, 4096, (1 << 15) + 1, 64, 64, 0), (1 << 30, 1 << 30, 1, 64, 64, 0)):
        assert fwd(*bad, 1) == bwd(*bad, 1) == 0
    rope = binding.gdn2_qk_norm_rope_bwd_workspace_bytes
    assert rope(8, 4096, 16, 16, 128) == 1024 * 2 * 128 * 4
    assert rope(1, 1, 4, 4, 128) >= 2 * 128 * 4
    assert rope(1, 0, 4, 4, 128) == rope(1, 5, 0, 4, 128) == rope(1, 5, 4, 4, 96) == 0


def _x(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _attn():
    return dict(q=_x(1, 3, 2, 32), k=_x(1, 3, 2, 32), v=_x(1, 3, 2, 64), alpha=_x(2))


def _qk():
    return dict(q=_x(1, 3, 4, 32), k=_x(1, 3, 2, 32))


CALLS = {"gdn2_linear_attn_fwd": _attn,
         "gdn2_linear_attn_bwd": lambda: dict(_attn(), d_o=_x(1, 3, 2, 64)),
         "gdn2_linear_attn_step": lambda: dict(q=_x(3, 2, 32), k=_x(3, 2, 32), v=_x(3, 2, 64), alpha=_x(2),
                                               state=_x(3, 2, 32, 64)),
         "gdn2_qk_norm_rope": lambda: dict(_qk(), inv_freq=_x(16)),
         "gdn2_qk_norm_rope_bwd": lambda: dict(_qk(), d_q_out=_x(1, 3, 4, 32), d_k_out=_x(1, 3, 2, 32), inv_freq=_x(16))}


@pytest.mark.parametrize("name", CALLS)
def test_calls_by_keyword_need_a_gpu(name):
    with pytest.raises(ValueError, match="must be on a GPU"):
        getattr(binding, name)(**CALLS[name]())


@pytest.mark.parametrize("name", CALLS)
def test_the_signature_has_the_stream(name):
    assert inspect.signature(getattr(binding, name)).parameters["stream"].default is None


@pytest.mark.parametrize("name,kw,error", [
    ("gdn2_linear_attn_fwd", dict(k=_x(1, 3, 2, 64)), ValueError),
    ("gdn2_linear_attn_fwd", dict(v=_x(1, 4, 2, 64)), ValueError),
    ("gdn2_linear_attn_fwd", dict(q=_x(3, 2, 32)), ValueError),
    ("gdn2_linear_attn_fwd", dict(v=_x(3, 64)), ValueError),
    ("gdn2_linear_attn_fwd", dict(alpha=_x(3)), ValueError),
    ("gdn2_linear_attn_fwd", dict(alpha=_x(2, dtype=torch.float64)), TypeError),
    ("gdn2_linear_attn_fwd", dict(k=_x(1, 3, 2, 32, dtype=torch.bfloat16)), TypeError),
    ("gdn2_linear_attn_fwd", dict(q=_x(1, 3, 2, 32, dtype=torch.float16)), TypeError),
    ("gdn2_linear_attn_fwd", dict(q=_x(1, 2, 3, 32).transpose(1, 2)), ValueError),
    ("gdn2_linear_attn_fwd", dict(initial_state=_x(1, 2, 64, 32)), ValueError),
    ("gdn2_linear_attn_fwd", dict(final_state=_x(2, 2, 32, 64)), ValueError),
    ("gdn2_linear_attn_fwd", dict(cu_seqlens=_x(3, dtype=torch.int64)), TypeError),
    ("gdn2_linear_attn_fwd", dict(out=_x(1, 3, 2, 32)), ValueError),
    ("gdn2_linear_attn_bwd", dict(d_o=_x(1, 3, 2, 32)), ValueError),
    ("gdn2_linear_attn_bwd", dict(d_final_state=_x(1, 2, 32, 32)), ValueError),
    ("gdn2_linear_attn_step", dict(q=_x(1, 3, 2, 32)), ValueError),
    ("gdn2_linear_attn_step", dict(state=_x(3, 2, 32, 64, dtype=torch.bfloat16)), TypeError),
    ("gdn2_linear_attn_step", dict(out=_x(3, 2, 32)), ValueError),
    ("gdn2_qk_norm_rope", dict(k=_x(1, 4, 2, 32)), ValueError),
    ("gdn2_qk_norm_rope", dict(k=_x(1, 3, 2, 64)), ValueError),
    ("gdn2_qk_norm_rope", dict(inv_freq=_x(2, 8)), ValueError),
    ("gdn2_qk_norm_rope", dict(positions=_x(3, dtype=torch.int32)), ValueError),
    ("gdn2_qk_norm_rope", dict(positions=_x(1, 3, dtype=torch.int64)), TypeError),
    ("gdn2_qk_norm_rope", dict(weight_k=_x(64)), ValueError),
    ("gdn2_qk_norm_rope", dict(q_out=_x(1, 3, 2, 32)), ValueError),
    ("gdn2_qk_norm_rope_bwd", dict(d_q_out=_x(1, 3, 2, 32)), ValueError),
    ("gdn2_qk_norm_rope_bwd", dict(d_k_out=_x(1, 3, 2, 32, dtype=torch.bfloat16)), TypeError),
])
def test_the_binding_refuses(name, kw, error):
    with pytest.raises(error):
        getattr(binding, name)(**{**CALLS[name](), **kw})
