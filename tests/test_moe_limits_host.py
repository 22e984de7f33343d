"""Sizes next to the limits of the mixture-of-experts calls, on the CPU: what is accepted is what one launch can hold, and what is
not is refused before anything is enqueued.  Pointers are fake, never dereferenced, and far enough apart for the largest arrays."""
import pytest

from tests import test_moe_host as H
from tests.test_moe_host import cr, lib  # noqa: F401  (lib is a fixture)

FAR = [i << 44 for i in range(1, 12)]
MOST = (1 << 26) - 1
ROWS = dict(zip(("dy", "off", "wq", "sw", "dx", "ws"), FAR), wsb=1 << 60)
LAYER = dict(zip(("dy", "pre", "d", "ex", "w", "wg", "sg", "wu", "su", "wd", "sd"), FAR), dx=1 << 50, dw=1 << 51, ws=1 << 52, wsb=1 << 60)

FITS = [("convrot_linear_grouped_backward", H.grouped_bwd(**ROWS, rows=rows, N=64, K=K, group=64, groups=groups))
        for rows, K, groups in [((1 << 24) - 1, 64, 4), (1 << 24, 64, 4), (MOST, 64, 1024), (MOST, 3840, 1024), (1 << 20, 131072, 4)]]
FITS += [("convrot_moe_ffn_gated_backward", H.moe_bwd(**LAYER, M=M, top=top, E_=8, F=64, K=64, group=64, gh=64))
         for M, top in [(1 << 21, 8), (MOST // 8, 8), (MOST // 2, 1)]]
FITS += [(n, f(M=MOST, E_=1, top=1, **at)) for n, f, at in (
    ("convrot_moe_route", H.route, dict(l=FAR[0], ex=FAR[1], w=FAR[2])),
    ("convrot_moe_route_backward", H.route_bwd, dict(l=FAR[0], ex=FAR[1], dw=FAR[2], dl=FAR[3])))]
TOO_MANY = [("convrot_linear_grouped_backward", H.grouped_bwd(**ROWS, rows=rows, N=64, K=K, group=64, groups=groups))
            for rows, K, groups in [(MOST + 1, 64, 4), (MOST, 4160, 4), (1 << 22, 131072, 4), ((1 << 24) - 64, 16384, 1024)]]
TOO_MANY += [("convrot_moe_ffn_gated_backward", H.moe_bwd(**LAYER, M=1 << 22, top=8, E_=8, F=8192, K=64, group=64, gh=64))]


@pytest.mark.parametrize("i", range(len(FITS)))
def test_accepted_up_to_the_device(lib, i):  # noqa: F811
    name, args = FITS[i]
    with pytest.raises(cr.ConvRotError) as e:
        cr._call(name, *args)
    assert cr.STATUS[e.value.status] == "CONVROT_ERR_HIP", str(e.value)


@pytest.mark.parametrize("i", range(len(TOO_MANY)))
def test_refused(lib, i):  # noqa: F811
    name, args = TOO_MANY[i]
    with pytest.raises(cr.ConvRotError) as e:
        cr._call(name, *args)
    assert cr.STATUS[e.value.status] == "CONVROT_ERR_SHAPE" and name in str(e.value), str(e.value)


def test_workspace_queries_agree():
    assert cr.workspace_bytes_grouped_backward(MOST, 1024, 64, 3840) >= MOST * 128
    assert cr.workspace_bytes_grouped_backward(MOST, 4, 64, 4160) == 0
    assert cr.workspace_bytes_moe_ffn_backward(1 << 22, 8, 8, 8192, 64) == 0
    # fp32 parts over the operand of the first contraction
    assert cr.workspace_bytes_moe_ffn_backward(9, 2, 4, 64, 128) > 18 * 64 * 4 + 18 * 128 * 4
