"""A backward call's bias gradients may share no byte with what the call reads or writes besides: for few tokens they
are written while other workgroups still read dy and pre (no GPU, nothing launched, fake pointers)."""
import pytest

from tests import test_fused_host as T
from tests.test_fused_host import A, D, G, H, bwd_args, ffn_bwd_args, gated_bwd_args, lib  # noqa: F401

# M = 32, N = 256, K = 512: dy of the block holds 32768 bytes, of the linears 16384, pre 16384 or 32768
CASES = [("convrot_linear_act_backward", bwd_args(**kw)) for kw in [
    dict(db=A), dict(db=A + 16384 - 4), dict(db=A - 1020), dict(db=G), dict(db=G + 16384 - 4), dict(db=A, act=0, pre=None)]]
CASES += [("convrot_linear_gated_backward", gated_bwd_args(**kw)) for kw in [
    dict(db1=A), dict(db2=A + 16384 - 4), dict(db1=G + 32768 - 4), dict(db2=G), dict(db1=H, db2=G - 1020)]]
CASES += [("convrot_ffn_gated_backward", ffn_bwd_args(**kw)) for kw in [
    dict(db1=A), dict(db2=A + 32768 - 4), dict(db3=A), dict(db1=G + 32768 - 4), dict(db2=G - 1020), dict(db3=A + 32768 - 4),
    dict(db3=G + 32768 - 4), dict(db3=A - 2044)]]

# next to them, and of no call's arrays: act "none" does not read pre
VALID = [("convrot_linear_act_backward", bwd_args(db=A + 16384)), ("convrot_linear_act_backward", bwd_args(db=A - 1024)),
         ("convrot_linear_act_backward", bwd_args(db=G, act=0)),
         ("convrot_linear_gated_backward", gated_bwd_args(db1=G + 32768, db2=A + 16384)),
         ("convrot_ffn_gated_backward", ffn_bwd_args(db1=A + 32768, db2=G + 32768, db3=G - 2048)),
         # dx in the place of dy or pre, which are read before it is written
         ("convrot_linear_act_backward", bwd_args(dx=A, db=H)), ("convrot_linear_act_backward", bwd_args(dx=G, db=H)),
         ("convrot_ffn_gated_backward", ffn_bwd_args(dx=G, db1=H))]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_bias_gradients_overlap_nothing(lib, i):  # noqa: F811
    name, args = CASES[i]
    rc = getattr(lib, name)(*args)
    assert rc == T.ERR["CONVROT_ERR_OVERLAP"] and name in lib.convrot_last_error().decode(), (args, rc)


@pytest.mark.parametrize("i", range(len(VALID)))
def test_neighbours_pass(lib, i):  # noqa: F811
    name, args = VALID[i]
    assert getattr(lib, name)(*args) == T.ERR["CONVROT_ERR_HIP"], lib.convrot_last_error().decode()
