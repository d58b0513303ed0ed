"""The training operators called by keyword, as their documentation names the arguments (CPU tensors: a
whole call ends at the check for a GPU)."""
import inspect

import pytest
import torch

from delta_rule_linear_gdn2_amd import binding

OPERATORS = ("gdn2_block_norm_fwd", "gdn2_block_norm_bwd", "gdn2_dropout", "gdn2_mixer_epilogue_bwd",
             "gdn2_mixer_prologue_bwd")


def _x(*shape):
    return torch.zeros(shape)


def _prologue():
    B, T, H, dk, dv, K = 1, 3, 2, 32, 64, 4
    key, value, fk, fv = _x(B, T, H, dk), _x(B, T, H, dv), _x(H * dk, K), _x(H * dv, K)
    return dict(xq=key, xk=key, xv=value, conv_q=fk, conv_k=fk, conv_v=fv, b_logit=key, w_logit=value, d_q=key, d_k=key,
                d_v=value, d_b=key, d_w=value)


CALLS = {"gdn2_block_norm_fwd": lambda: dict(x=_x(3, 16), u=_x(3, 16)),
         "gdn2_block_norm_bwd": lambda: dict(x_out=_x(3, 16), u=_x(3, 16), d_x_out=_x(3, 16), d_h=None),
         "gdn2_dropout": lambda: dict(x=_x(3, 16), p=0.1, seed=1),
         "gdn2_mixer_epilogue_bwd": lambda: dict(o=_x(3, 32), gate=_x(3, 32), weight=_x(32), d_y=_x(3, 32)),
         "gdn2_mixer_prologue_bwd": _prologue}


@pytest.mark.parametrize("name", OPERATORS)
def test_every_argument_by_keyword(name):
    with pytest.raises(ValueError, match="must be on a GPU"):
        getattr(binding, name)(**CALLS[name]())


@pytest.mark.parametrize("name", OPERATORS)
def test_a_missing_first_argument_is_named(name):
    kw = CALLS[name]()
    first = next(iter(kw))
    kw.pop(first)
    with pytest.raises(TypeError, match=f"'{first}'"):
        getattr(binding, name)(**kw)


@pytest.mark.parametrize("name", OPERATORS)
def test_the_signature_has_the_stream(name):
    assert inspect.signature(getattr(binding, name)).parameters["stream"].default is None
