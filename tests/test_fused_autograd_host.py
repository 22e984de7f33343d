"""The fused forward calls return tensors without autograd history; they say so when an input asks for one (the warning
comes before the device check, so no GPU is needed)."""
import warnings

import pytest
import torch

cr = pytest.importorskip("int4_quantized_linear_amd.convrot")

W, S = torch.zeros(64, 64, dtype=torch.int8), torch.ones(64)
X = torch.zeros(2, 64, dtype=torch.bfloat16)
CALLS = {
    "linear_act": lambda **kw: cr.linear_act(kw.pop("x", X), W, S, group=64, **kw),
    "linear_gated": lambda **kw: cr.linear_gated(kw.pop("x", X), W, S, W, S, group=64, **kw),
    "ffn_gated": lambda **kw: cr.ffn_gated(kw.pop("x", X), W, S, W, S, W, S, group=64, group_h=64, **kw),
}
NEEDS = [("linear_act", "x"), ("linear_act", "residual"), ("linear_act", "bias"), ("linear_gated", "x"),
         ("linear_gated", "bias_gate"), ("linear_gated", "bias_up"), ("ffn_gated", "x"), ("ffn_gated", "residual"),
         ("ffn_gated", "bias_gate"), ("ffn_gated", "bias_up"), ("ffn_gated", "bias_down")]


def _input(name):
    return torch.zeros(64) if name.startswith("bias") else X.clone()


@pytest.mark.parametrize("call,name", NEEDS)
def test_warns_where_history_is_lost(call, name):
    t = _input(name).requires_grad_()
    with pytest.warns(UserWarning, match="%s .*%s_backward" % (call, call)), pytest.raises(ValueError, match="is on cpu"):
        CALLS[call](**{name: t})


@pytest.mark.parametrize("call,name", NEEDS)
def test_silent_where_none_is_asked_for(call, name):
    """No gradient asked for, or inside torch.no_grad() or a torch.autograd.Function."""
    seen = []

    class Wrapped(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            with pytest.raises(ValueError, match="is on cpu"):
                CALLS[call](**{name: t})
            seen.append(t.requires_grad)
            return t.clone()

    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="is on cpu"):
            CALLS[call](**{name: _input(name)})
        t = _input(name).requires_grad_()
        with torch.no_grad(), pytest.raises(ValueError, match="is on cpu"):
            CALLS[call](**{name: t})
        Wrapped.apply(t)
    assert seen == [True]
