"""Refusals of the training operators on a machine without a GPU: the C ABI
rejects bad arguments before any HIP call, the binding before the C call."""
import ctypes

import pytest
import torch

from delta_rule_linear_gdn2_amd import binding
from test_abi_cpu import ALIAS, DTYPE, MISAL, NULLP, SHAPE, UNSUP, WS, fake, lib  # noqa: F401


def call(f, order, args, kw):
    args = {**args, **kw}
    return f(*(args[n] for n in order), None)


# rows=100, D=96: [rows, D] is 19200 bytes of bf16, 38400 of FP32
FWD = dict(x=fake(0), u=fake(1), gate=fake(2), w_post=fake(3), w_pre=fake(4), x_out=fake(5), h=fake(6), rows=100, D=96,
           eps=1e-5, scale=1.0, layout=3, act=0, p=0.1, seed=1, offset=2, offset_device=None, dtype=1, rdtype=0)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=2), DTYPE),
    (dict(dtype=0, rdtype=1), DTYPE),             # a bf16 stream of FP32 blocks
    (dict(rdtype=-1), DTYPE),
    (dict(rows=-1), SHAPE),
    (dict(rows=(1 << 40) + 1), SHAPE),
    (dict(D=0), SHAPE),
    (dict(D=16385), UNSUP),
    (dict(eps=0.0), SHAPE),
    (dict(eps=float("nan")), SHAPE),
    (dict(layout=4), SHAPE),
    (dict(layout=-1), SHAPE),
    (dict(act=3), SHAPE),
    (dict(p=-0.01), SHAPE),
    (dict(p=1.01), SHAPE),
    (dict(p=float("nan")), SHAPE),
    (dict(layout=0), SHAPE),                      # a gate without a layout
    (dict(gate=None), NULLP),
    (dict(x=None), NULLP),
    (dict(x_out=None), NULLP),
    (dict(h=None), NULLP),
    (dict(w_pre=None), NULLP),
    (dict(u=None), SHAPE),                        # gate, norm and dropout of nothing
    (dict(u=None, gate=None, layout=0, w_post=None, p=0.0), SHAPE),               # a stream out without a block
    (dict(u=None, gate=None, layout=0, w_post=None, p=0.0, x_out=None, h=None, w_pre=None), NULLP),
    (dict(u=fake(1, 8)), MISAL),
    (dict(w_pre=fake(4, 4)), MISAL),
    (dict(offset_device=fake(7, 4)), MISAL),
    (dict(x_out=fake(0, 16)), ALIAS),             # x_out inside x, not x itself
    (dict(x_out=fake(1)), ALIAS),                 # x_out over u
    (dict(h=fake(1)), ALIAS),
    (dict(h=fake(0, 38384)), ALIAS),              # h from the last bytes of x on
    (dict(h=fake(5, 1024)), ALIAS),               # h inside x_out
    (dict(h=fake(4)), ALIAS),                     # h over a weight
    (dict(offset_device=fake(5, 8)), ALIAS),      # the dropout offset inside x_out
])
def test_block_norm_fwd_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_block_norm_fwd, list(FWD), FWD, kw) == expected


BWD = dict(x_out=fake(0), u=fake(1), gate=fake(2), w_post=fake(3), w_pre=fake(4), d_x_out=fake(5), d_h=fake(6), d_x=fake(7),
           d_u=fake(8), d_gate=fake(9), d_w_post=fake(10), d_w_pre=fake(11), rows=100, D=96, eps=1e-5, scale=1.0, layout=3,
           act=0, p=0.1, seed=1, offset=2, offset_device=None, dtype=1, rdtype=0, ws=fake(12), ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=9), DTYPE),
    (dict(dtype=0, rdtype=1), DTYPE),
    (dict(D=20000), UNSUP),
    (dict(p=2.0), SHAPE),
    (dict(u=None, gate=None, layout=0, w_post=None, p=0.0, d_gate=None, d_w_post=None), SHAPE),  # d_u without u
    (dict(gate=None, layout=0), SHAPE),                   # d_gate without a gate
    (dict(w_post=None), SHAPE),                           # d_w_post without its weight
    (dict(w_pre=None, d_h=None), SHAPE),                  # d_w_pre without its weight
    (dict(d_h=None), NULLP),
    (dict(w_pre=None, d_w_pre=None), NULLP),              # d_h without its weight
    (dict(w_pre=None, d_w_pre=None, d_h=None, d_x_out=None), NULLP),
    (dict(x_out=None), NULLP),
    (dict(d_x=None), NULLP),
    (dict(d_u=None), NULLP),
    (dict(ws=None), WS),
    (dict(ws_bytes=100), WS),
    (dict(d_h=fake(6, 2)), MISAL),
    (dict(ws=fake(12, 8)), MISAL),
    (dict(d_x=fake(0)), ALIAS),                           # d_x over the stream
    (dict(d_x=fake(5, 16)), ALIAS),                       # d_x inside d_x_out, not d_x_out itself
    (dict(d_u=fake(1)), ALIAS),
    (dict(d_gate=fake(8, 64)), ALIAS),
    (dict(d_w_pre=fake(10, 16)), ALIAS),
    (dict(ws=fake(6, 256)), ALIAS),                       # workspace inside an input
    (dict(ws=fake(11)), ALIAS),                           # workspace over an output
])
def test_block_norm_bwd_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_block_norm_bwd, list(BWD), BWD, kw) == expected


DROP = dict(x=fake(0), y=fake(1), rows=100, D=96, p=0.1, seed=1, offset=2, offset_device=None, dtype=1)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=2), DTYPE),
    (dict(rows=-1), SHAPE),
    (dict(D=0), SHAPE),
    (dict(rows=1 << 50, D=1 << 40), SHAPE),
    (dict(D=(1 << 56) + 1, rows=1), SHAPE),
    (dict(p=1.5), SHAPE),
    (dict(x=None), NULLP),
    (dict(y=None), NULLP),
    (dict(y=fake(1, 2)), MISAL),
    (dict(offset_device=fake(3, 4)), MISAL),
    (dict(y=fake(0, 16)), ALIAS),
    (dict(offset_device=fake(1, 16)), ALIAS),
])
def test_dropout_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_dropout, list(DROP), DROP, kw) == expected


EPI = dict(o=fake(0), gate=fake(1), weight=fake(2), d_y=fake(3), d_o=fake(4), d_gate=fake(5), d_weight=fake(6), rows=100,
           dv=64, eps=1e-5, act=0, dtype=1, ws=fake(7), ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=3), DTYPE),
    (dict(act=2), SHAPE),
    (dict(eps=0.0), SHAPE),
    (dict(rows=-1), SHAPE),
    (dict(dv=80), UNSUP),
    (dict(d_y=None), NULLP),
    (dict(d_o=None), NULLP),
    (dict(ws=None), WS),
    (dict(ws_bytes=1), WS),
    (dict(weight=fake(2, 4)), MISAL),
    (dict(d_o=fake(3)), ALIAS),
    (dict(d_gate=fake(4, 256)), ALIAS),
    (dict(d_weight=fake(2)), ALIAS),
    (dict(ws=fake(6)), ALIAS),
])
def test_mixer_epilogue_bwd_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_mixer_epilogue_bwd, list(EPI), EPI, kw) == expected


# B=2, T=64, H=4, dk=dv=64, K=4 bf16
PRO_NAMES = ("xq xk xv cq ck cv bl wl si dq dk_ dv_ db dw dso dxq dxk dxv dcq dck dcv dbl dwl dsi").split()
PRO = dict({n: fake(i) for i, n in enumerate(PRO_NAMES)}, cu=None, B=2, T=64, H=4, dk=64, dv=64, K=4, num_seqs=0, scale=1.0,
           eps=1e-6, dtype=1, ws=fake(30), ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=7), DTYPE),
    (dict(K=0), SHAPE),
    (dict(K=17), SHAPE),
    (dict(eps=-1.0), SHAPE),
    (dict(T=-1), SHAPE),
    (dict(cu=fake(40), num_seqs=3), SHAPE),               # packed with B = 2
    (dict(cu=fake(40), B=1, num_seqs=0), SHAPE),
    (dict(H=(1 << 20) + 1), SHAPE),
    (dict(dk=96), UNSUP),
    (dict(cq=None), NULLP),
    (dict(dw=None), NULLP),
    (dict(dxv=None), NULLP),
    (dict(dwl=None), NULLP),
    (dict(ws=None), WS),
    (dict(ws_bytes=1000), WS),
    (dict(xv=fake(2, 8)), MISAL),
    (dict(cu=fake(40, 2), B=1, num_seqs=2), MISAL),
    (dict(dxq=fake(0)), ALIAS),
    (dict(dxk=fake(15, 512)), ALIAS),                     # inside d_xq
    (dict(dcv=fake(5)), ALIAS),                           # over its filters
    (dict(dsi=fake(8)), ALIAS),
    (dict(dsi=fake(14)), ALIAS),                          # no in-place state gradient
    (dict(ws=fake(22)), ALIAS),
])
def test_mixer_prologue_bwd_rejects(lib, kw, expected):  # noqa: F811
    assert call(lib.gdn2_mixer_prologue_bwd, list(PRO), PRO, kw) == expected


def test_workspace_queries(lib):  # noqa: F811
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    f = binding.gdn2_block_norm_bwd_workspace_bytes
    assert f(0, 64) == f(-1, 64) == f(10, 0) == f(10, 16385) == 0
    assert 0 < f(1, 2048) <= f(32768, 2048) <= up(1024 * 3 * 2048 * 4)
    f = binding.gdn2_mixer_epilogue_bwd_workspace_bytes
    assert f(0, 64) == f(10, 80) == 0
    assert 0 < f(1, 128) <= f(1 << 30, 128) <= up(1024 * 128 * 4)
    f = binding.gdn2_mixer_prologue_bwd_workspace_bytes
    assert f(1, 0, 4, 64, 64, 4) == f(1, 10, 4, 64, 64, 17) == f(1, 10, 4, 48, 64, 4) == f(0, 10, 4, 64, 64, 4) == 0
    assert f(2, 1, 4, 64, 32, 4) == up(2 * 4 * 160 * 4 * 4)


# --- the binding's own checks, on CPU tensors --------------------------------


def _x(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_cpu_tensors():
    x = _x(3, 16)
    for f in (lambda: binding.gdn2_dropout(x, 0.1, 1), lambda: binding.gdn2_block_norm_fwd(x, x),
              lambda: binding.gdn2_block_norm_fwd(x, weight_pre=_x(16)),
              lambda: binding.gdn2_block_norm_bwd(x, x, x, None),
              lambda: binding.gdn2_mixer_epilogue_bwd(_x(3, 32), _x(3, 32), _x(32), _x(3, 32))):
        with pytest.raises(ValueError, match="must be on a GPU"):
            f()


@pytest.mark.parametrize("error,kw", [
    (ValueError, dict(u=_x(3, 15))),                                          # another shape
    (ValueError, dict(u=_x(16, 3).T)),                                        # strided
    (ValueError, dict(gate=_x(3, 16))),                                       # a gate without a layout
    (ValueError, dict(gate_layout="full")),                                   # a layout without a gate
    (ValueError, dict(gate=_x(3, 16), gate_layout="rows")),
    (ValueError, dict(gate=_x(3), gate_layout="channel")),
    (ValueError, dict(gate=_x(16), gate_layout="token")),
    (TypeError, dict(gate=_x(16, dtype=torch.bfloat16), gate_layout="channel")),
    (ValueError, dict(gate_act="tanh")),
    (TypeError, dict(weight_post=_x(16, dtype=torch.bfloat16))),
    (ValueError, dict(weight_pre=_x(15))),
    (ValueError, dict(h=_x(3, 16))),                                          # h without its weight
    (ValueError, dict(x_out=_x(3, 17))),
    (ValueError, dict(seed=-1)),
    (ValueError, dict(offset=1 << 64)),
    (TypeError, dict(offset_device=_x(1))),
    (TypeError, dict(u=_x(3, 16, dtype=torch.float16))),
    (TypeError, dict(dtype=torch.bfloat16)),                                  # h has u's type
])
def test_block_norm_fwd_binding_rejects(error, kw):
    with pytest.raises(error, match="^(?!.*must be on a GPU)"):
        binding.gdn2_block_norm_fwd(_x(3, 16), **{"u": _x(3, 16), **kw})


@pytest.mark.parametrize("error,kw", [
    (ValueError, dict(d_h=_x(3, 16))),                                        # d_h without weight_pre
    (ValueError, dict(weight_pre=_x(16))),                                    # weight_pre without d_h
    (ValueError, dict(d_x_out=_x(3, 15))),
    (TypeError, dict(d_x_out=_x(3, 16, dtype=torch.bfloat16))),
    (ValueError, dict(d_u=_x(2, 16))),
])
def test_block_norm_bwd_binding_rejects(error, kw):
    args = {"d_x_out": _x(3, 16), "d_h": None, **kw}
    with pytest.raises(error, match="^(?!.*must be on a GPU)"):
        binding.gdn2_block_norm_bwd(_x(3, 16), _x(3, 16), args.pop("d_x_out"), args.pop("d_h"), **args)


def test_binding_refuses_rows_without_elements():
    for x in (torch.tensor(1.0), _x(3, 0)):
        with pytest.raises(ValueError, match="last axis"):
            binding.gdn2_dropout(x, 0.1, 1)


def test_public_names():
    import delta_rule_linear_gdn2_amd as pkg

    for name in ("gdn2_block_norm_fwd", "gdn2_block_norm_bwd", "gdn2_dropout", "gdn2_mixer_epilogue_bwd",
                 "gdn2_mixer_prologue_bwd"):
        assert name in pkg.__all__ and getattr(pkg, name) is getattr(binding, name)
        assert isinstance(getattr(binding.load(), name), ctypes._CFuncPtr)


def _prologue(**kw):
    B, T, H, dk, dv, K = 2, 3, 2, 32, 64, 4
    z = dict(xq=_x(B, T, H, dk), xk=_x(B, T, H, dk), xv=_x(B, T, H, dv), conv_q=_x(H * dk, K), conv_k=_x(H * dk, K),
             conv_v=_x(H * dv, K), b_logit=_x(B, T, H, dk), w_logit=_x(B, T, H, dv), d_q=_x(B, T, H, dk),
             d_k=_x(B, T, H, dk), d_v=_x(B, T, H, dv), d_b=_x(B, T, H, dk), d_w=_x(B, T, H, dv))
    named = {n: kw.pop(n) for n in list(kw) if n not in z}
    return binding.gdn2_mixer_prologue_bwd(*{**z, **kw}.values(), **named)


@pytest.mark.parametrize("error,match,kw", [
    (ValueError, "d_k: shape", dict(d_k=_x(2, 3, 2, 31))),
    (ValueError, "w_logit: shape", dict(w_logit=_x(2, 3, 2, 32))),
    (TypeError, "xv: dtype", dict(xv=_x(2, 3, 2, 64, dtype=torch.bfloat16))),
    (ValueError, "d_b: must be contiguous", dict(d_b=_x(2, 3, 32, 2).transpose(2, 3))),
    (ValueError, "conv_v: shape", dict(conv_v=_x(64, 4))),
    (TypeError, "conv_q: dtype", dict(conv_q=_x(64, 4, dtype=torch.bfloat16))),
    (ValueError, "conv_state: shape", dict(conv_state=_x(2, 256, 4))),
    (TypeError, "cu_seqlens: dtype", dict(cu_seqlens=torch.zeros(3, dtype=torch.int64))),
    (ValueError, r"\[B, T, H, d\]", dict(xv=_x(2, 3, 128))),
    (ValueError, "must be on a GPU", dict()),
])
def test_mixer_prologue_bwd_binding_rejects(error, match, kw):
    with pytest.raises(error, match=match):
        _prologue(**kw)
