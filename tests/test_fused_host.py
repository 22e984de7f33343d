"""Host-side refusals of the fused linears (no GPU, nothing launched): every violated precondition
returns its status before anything is enqueued.  Pointers are fake and never dereferenced."""
import os

import pytest

cr = pytest.importorskip("int4_quantized_linear_amd.convrot")
ERR = {v: k for k, v in cr.STATUS.items()}

A, B, C, D, E, G, H = (0x10000000 * i for i in range(1, 8))     # fake, 256-byte aligned, far apart
MIS = A + 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cr.LIB_PATH):
        pytest.fail("libconvrot.so is not built; run python -m int4_quantized_linear_amd.build")
    if os.path.exists("/dev/kfd"):
        pytest.skip("host-only check (fake device pointers)")
    return cr.load()


def act_args(x=A, dt=1, xq=None, xs=None, M=32, N=256, K=512, group=256, wq=B, sw=C, bias=None, act=2, res=None,
             pre=None, y=D, ws=E, wsb=1 << 26):
    return (x, dt, xq, xs, M, N, K, group, wq, sw, bias, act, res, pre, y, ws, wsb, None)


def gated_args(x=A, dt=1, xq=None, xs=None, M=32, N=256, K=512, group=256, wg=B, sg=C, bg=None, wu=B, su=C, bu=None,
               act=2, pre=None, h=D, ws=E, wsb=1 << 26):
    return (x, dt, xq, xs, M, N, K, group, wg, sg, bg, wu, su, bu, act, pre, h, ws, wsb, None)


def ffn_args(x=A, dt=1, M=32, F=256, K=512, group=256, group_h=256, wg=B, sg=C, bg=None, wu=B, su=C, bu=None, wd=B,
             sd=C, bd=None, act=2, res=None, pre=None, y=D, ws=E, wsb=1 << 26):
    return (x, dt, M, F, K, group, group_h, wg, sg, bg, wu, su, bu, wd, sd, bd, act, res, pre, y, ws, wsb, None)


SHARED = [
    (dict(M=-1), "SHAPE"), (dict(K=100), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=131072 + 64), "SHAPE"),
    (dict(group=3), "GROUP"), (dict(group=512), "GROUP"), (dict(act=-1), "ACT"), (dict(act=5), "ACT"),
    (dict(dt=7), "DTYPE"), (dict(x=None), "NULL"), (dict(x=MIS), "ALIGN"), (dict(pre=D), "OVERLAP"),
    (dict(pre=D + 256), "OVERLAP"), (dict(pre=MIS), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(ws=E + 16), "WORKSPACE"),
    (dict(wsb=100), "WORKSPACE"), (dict(M=1 << 31), "SHAPE"),
]
CASES = [(n, f(**kw), s) for n, f in (("convrot_linear_act", act_args), ("convrot_linear_gated", gated_args),
                                      ("convrot_ffn_gated", ffn_args)) for kw, s in SHARED]
CASES += [("convrot_linear_act", act_args(**kw), s) for kw, s in [
    (dict(wq=None), "NULL"), (dict(sw=None), "NULL"), (dict(y=None), "NULL"), (dict(y=MIS), "ALIGN"),
    (dict(bias=MIS - 1), "ALIGN"), (dict(res=MIS), "ALIGN"), (dict(res=D + 512), "OVERLAP"),
    (dict(res=D - 512), "OVERLAP"), (dict(res=G, pre=G), "OVERLAP"), (dict(N=1 << 24), "SHAPE"),
    (dict(x=None, xq=A), "NULL"), (dict(x=None, xq=D, xs=C), "OVERLAP"), (dict(x=None, xq=G, xs=C, pre=G), "OVERLAP"),
    (dict(x=None, xq=A, xs=D + 64), "OVERLAP"), (dict(x=None, xq=A, xs=G + 4, pre=G), "OVERLAP")]]
CASES += [("convrot_linear_gated", gated_args(**kw), s) for kw, s in [
    (dict(wu=None), "NULL"), (dict(su=None), "NULL"), (dict(wg=None), "NULL"), (dict(sg=None), "NULL"),
    (dict(h=None), "NULL"), (dict(wu=MIS), "ALIGN"), (dict(bu=MIS - 1), "ALIGN"),
    (dict(pre=D - 32 * 256 * 2), "OVERLAP"), (dict(N=1 << 24), "SHAPE")]]
CASES += [("convrot_ffn_gated", ffn_args(**kw), s) for kw, s in [
    (dict(F=100), "SHAPE"), (dict(F=0), "SHAPE"), (dict(F=131072 + 64), "SHAPE"), (dict(group_h=5), "GROUP"),
    (dict(F=320, group_h=128), "SHAPE"), (dict(wd=None), "NULL"), (dict(sd=None), "NULL"), (dict(wu=None), "NULL"),
    (dict(bd=MIS - 1), "ALIGN"), (dict(res=MIS), "ALIGN"), (dict(res=D + 256), "OVERLAP"),
    (dict(pre=A), "OVERLAP"), (dict(res=G, pre=G), "OVERLAP")]]


def bwd_args(dy=A, pre=G, M=32, N=256, K=512, group=256, wq=B, sw=C, act=2, add=None, dx=D, db=None, ws=E,
             wsb=1 << 26):
    return (dy, pre, M, N, K, group, wq, sw, act, add, dx, db, ws, wsb, None)


def gated_bwd_args(dy=A, pre=G, M=32, N=256, K=512, group=256, wg=B, sg=C, wu=B, su=C, act=2, add=None, dx=D, db1=None,
                   db2=None, ws=E, wsb=1 << 26):
    return (dy, pre, M, N, K, group, wg, sg, wu, su, act, add, dx, db1, db2, ws, wsb, None)


def ffn_bwd_args(dy=A, pre=G, M=32, N=256, K=512, group=256, group_h=256, wg=B, sg=C, wu=B, su=C, wd=B, sd=C, act=2,
                 add=None, dx=D, db1=None, db2=None, db3=None, ws=E, wsb=1 << 26):
    return (dy, pre, M, N, K, group, group_h, wg, sg, wu, su, wd, sd, act, add, dx, db1, db2, db3, ws, wsb, None)


BACKWARD = [("convrot_linear_act_backward", bwd_args), ("convrot_linear_gated_backward", gated_bwd_args),
            ("convrot_ffn_gated_backward", ffn_bwd_args)]
CASES += [(n, f(**kw), s) for n, f in BACKWARD for kw, s in [
    (dict(M=-1), "SHAPE"), (dict(M=1 << 31), "SHAPE"), (dict(N=0), "SHAPE"), (dict(K=100), "SHAPE"),
    (dict(N=1 << 20), "SHAPE"), (dict(K=131072, M=(1 << 31) - 1, wsb=1 << 62), "SHAPE"), (dict(group=3), "GROUP"),
    (dict(K=320, group=128), "SHAPE"), (dict(act=5), "ACT"), (dict(act=-1), "ACT"), (dict(dy=None), "NULL"),
    (dict(pre=None), "NULL"), (dict(dx=None), "NULL"), (dict(dy=MIS), "ALIGN"), (dict(pre=MIS), "ALIGN"),
    (dict(dx=MIS), "ALIGN"), (dict(add=MIS), "ALIGN"), (dict(add=D + 256), "OVERLAP"), (dict(ws=None), "WORKSPACE"),
    (dict(ws=E + 16), "WORKSPACE"), (dict(wsb=100), "WORKSPACE")]]
CASES += [("convrot_linear_act_backward", bwd_args(**kw), s) for kw, s in [
    (dict(wq=None), "NULL"), (dict(sw=None), "NULL"), (dict(db=MIS - 1), "ALIGN"), (dict(db=D + 16), "OVERLAP"),
    (dict(db=H + 16, add=H), "OVERLAP")]]
CASES += [("convrot_linear_gated_backward", gated_bwd_args(**kw), s) for kw, s in [
    (dict(wu=None), "NULL"), (dict(su=None), "NULL"), (dict(db1=H, db2=H + 512), "OVERLAP"), (dict(db2=D), "OVERLAP"),
    (dict(act=0, pre=None), "NULL")]]
CASES += [("convrot_ffn_gated_backward", ffn_bwd_args(**kw), s) for kw, s in [
    (dict(wd=None), "NULL"), (dict(sd=None), "NULL"), (dict(wu=None), "NULL"), (dict(group_h=7), "GROUP"),
    (dict(N=320, group_h=128), "SHAPE"), (dict(N=100), "SHAPE"), (dict(db3=MIS - 1), "ALIGN"),
    (dict(db3=D), "OVERLAP"), (dict(db3=H, db1=H + 256), "OVERLAP"), (dict(db3=H, db2=H), "OVERLAP"),
    (dict(db3=G), "OVERLAP"), (dict(db3=H, add=H), "OVERLAP")]]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_refusals(lib, i):
    name, args, status = CASES[i]
    rc = getattr(lib, name)(*args)
    msg = lib.convrot_last_error().decode()
    assert rc == ERR["CONVROT_ERR_" + status] and name in msg, (name, args, rc, msg)


# calls that pass every check and stop at the missing device
VALID = [
    ("convrot_linear_act", act_args()), ("convrot_linear_act", act_args(res=D)),
    ("convrot_linear_act", act_args(M=4, N=1 << 24)),
    ("convrot_linear_act", act_args(x=None, xq=A, xs=C, ws=None, wsb=0, res=G, pre=H)),
    ("convrot_linear_gated", gated_args(pre=G, bg=C, bu=C)), ("convrot_ffn_gated", ffn_args(res=D, pre=G)),
    ("convrot_linear_act_backward", bwd_args(act=0, pre=None)), ("convrot_linear_act_backward", bwd_args(add=D, db=H)),
    ("convrot_linear_act_backward", bwd_args(M=0, db=H)),
    ("convrot_linear_gated_backward", gated_bwd_args(db1=H, db2=H + 1024)),
    ("convrot_ffn_gated_backward", ffn_bwd_args(add=A, db1=H, db2=H + 1024, db3=H + 2048)),
    ("convrot_ffn_gated_backward", ffn_bwd_args(dx=A, add=A))]
EMPTY = [
    ("convrot_linear_act", (None, 1, None, None, 0, 256, 512, 256, *[None] * 3, 0, *[None] * 4, 0, None)),
    ("convrot_linear_act", (None, 1, None, None, 5, 0, 512, 256, *[None] * 3, 0, *[None] * 4, 0, None)),
    ("convrot_linear_gated", (None, 1, None, None, 0, 256, 512, 256, *[None] * 6, 2, None, None, None, 0, None)),
    ("convrot_ffn_gated", (None, 1, 0, 256, 512, 256, 256, *[None] * 9, 2, *[None] * 4, 0, None)),
    ("convrot_linear_act_backward", (None, None, 0, 256, 512, 256, None, None, 2, *[None] * 4, 0, None)),
    ("convrot_linear_gated_backward", (None, None, 0, 256, 512, 256, *[None] * 4, 2, *[None] * 5, 0, None)),
    ("convrot_ffn_gated_backward", (None, None, 0, 256, 512, 256, 256, *[None] * 6, 2, *[None] * 6, 0, None))]


@pytest.mark.parametrize("name,args", VALID)
def test_valid_calls_reach_the_device(lib, name, args):
    assert getattr(lib, name)(*args) == ERR["CONVROT_ERR_HIP"], lib.convrot_last_error().decode()
    assert "hipGetDevice" in lib.convrot_last_error().decode()


@pytest.mark.parametrize("name,args", EMPTY)
def test_empty_inputs(lib, name, args):
    assert getattr(lib, name)(*args) == 0


def test_backward_workspace_queries(lib):
    for q in (lib.convrot_workspace_bytes_backward, lib.convrot_workspace_bytes_gated_backward,
              lib.convrot_workspace_bytes_ffn_backward):
        assert q(-1, 256, 512) == 0 and q(4, 0, 512) == 0 and q(4, 256, 100) == 0 and q(4, 1 << 20, 512) == 0
        assert q(0, 256, 512) == 0 and q((1 << 31) - 1, 256, 131072) == 0
    for M, N, K in [(1, 64, 64), (12, 8192, 5120), (2048, 25600, 5120), (4096, 16128, 5376)]:
        assert lib.convrot_workspace_bytes_backward(M, N, K) >= 2 * M * N
        assert lib.convrot_workspace_bytes_gated_backward(M, N, K) >= 4 * M * N
        w = lib.convrot_workspace_bytes_ffn_backward(M, N, K)
        assert w % 256 == 0 and w >= 6 * M * N
        args = list(ffn_bwd_args(M=M, N=N, K=K, group=64, group_h=64, dy=1 << 40, pre=2 << 40, ws=3 << 40, dx=4 << 40,
                                 wsb=w))
        assert lib.convrot_ffn_gated_backward(*args) == ERR["CONVROT_ERR_HIP"]
        args[-2] = w - 1
        assert lib.convrot_ffn_gated_backward(*args) == ERR["CONVROT_ERR_WORKSPACE"]


def test_workspace_queries(lib):
    up = lambda n: (n + 255) // 256 * 256
    for q in (lib.convrot_workspace_bytes_gated, lib.convrot_workspace_bytes_ffn):
        assert q(-1, 256, 512) == 0 and q(4, -1, 512) == 0 and q(4, 256, 100) == 0 and q(1 << 31, 256, 512) == 0
    assert lib.convrot_workspace_bytes_ffn(4, 100, 512) == 0
    for M, F, K in [(1, 25600, 5120), (12, 5376, 2688), (300, 5376, 2688), (2048, 25600, 5120)]:
        assert lib.convrot_workspace_bytes_gated(M, F, K) >= up(M * K) + up(4 * M)
        w = lib.convrot_workspace_bytes_ffn(M, F, K)
        assert w % 256 == 0 and w >= up(2 * M * F) + up(M * F) + up(4 * M)
        args = list(ffn_args(M=M, F=F, K=K, group=128, x=1 << 40, y=2 << 40, ws=3 << 40, wsb=w))
        assert lib.convrot_ffn_gated(*args) == ERR["CONVROT_ERR_HIP"]
        args[-2] = w - 1
        assert lib.convrot_ffn_gated(*args) == ERR["CONVROT_ERR_WORKSPACE"]
