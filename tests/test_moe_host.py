"""Host-side refusals of the mixture-of-experts calls (no GPU, nothing launched): every violated precondition returns
its status before anything is enqueued; the same calls under sanitizers; the binding's own checks; the warning about autograd.
Pointers are fake and never dereferenced."""
import os
import warnings

import pytest
import torch

from tests import test_host_sanitizers as S

cr = pytest.importorskip("int4_quantized_linear_amd.convrot")
ERR = {v: k for k, v in cr.STATUS.items()}

A, B, C, D, E, G, H, J = (0x40000000 * i for i in range(1, 9))     # fake, 256-byte aligned, far apart
MIS = A + 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(cr.LIB_PATH):
        pytest.fail("libconvrot.so is not built; run python -m int4_quantized_linear_amd.build")
    if os.path.exists("/dev/kfd"):
        pytest.skip("host-only check (fake device pointers)")
    return cr.load()


def route(l=A, dt=0, M=32, E_=64, top=8, score=0, norm=1, scale=1.0, bias=None, ex=B, w=C):
    return (l, dt, M, E_, top, score, norm, scale, bias, ex, w, None)


def route_bwd(dw=C, l=A, dt=0, M=32, E_=64, top=8, score=0, norm=1, scale=1.0, ex=B, dl=D):
    return (dw, l, dt, M, E_, top, score, norm, scale, ex, dl, None)


def grouped(x=A, dt=1, xq=None, xs=None, rows=32, N=256, K=512, group=256, off=G, groups=4, wq=B, sw=C, y=D, ws=E, wsb=1 << 26):
    return (x, dt, xq, xs, rows, N, K, group, off, groups, wq, sw, y, ws, wsb, None)


def grouped_bwd(dy=A, rows=32, N=256, K=512, group=256, off=G, groups=4, wq=B, sw=C, add=None, dx=D, ws=E, wsb=1 << 26):
    return (dy, rows, N, K, group, off, groups, wq, sw, add, dx, ws, wsb, None)


def moe(x=A, dt=1, ex=G, w=H, M=32, top=2, E_=8, F=256, K=512, group=256, gh=256, wg=B, sg=C, wu=B, su=C, wd=B, sd=C, act=2,
        res=None, pre=None, d=None, y=D, ws=E, wsb=1 << 27):
    return (x, dt, ex, w, M, top, E_, F, K, group, gh, wg, sg, wu, su, wd, sd, act, res, pre, d, y, ws, wsb, None)


def moe_bwd(dy=A, pre=J, d=J + (1 << 28), ex=G, w=H, M=32, top=2, E_=8, F=256, K=512, group=256, gh=256, wg=B, sg=C, wu=B, su=C,
            wd=B, sd=C, act=2, add=None, dx=D, dw=None, ws=E, wsb=1 << 27):
    return (dy, pre, d, ex, w, M, top, E_, F, K, group, gh, wg, sg, wu, su, wd, sd, act, add, dx, dw, ws, wsb, None)


SIZES = [dict(M=-1), dict(M=1 << 26), dict(M=1 << 40), dict(E_=0), dict(E_=1025), dict(top=0), dict(top=-1),
         dict(top=9, E_=8), dict(top=33, E_=64), dict(M=1 << 22, top=16, E_=64)]
CASES = [(n, f(**kw), "SHAPE") for n, f in (("convrot_moe_route", route), ("convrot_moe_route_backward", route_bwd),
                                            ("convrot_moe_ffn_gated", moe), ("convrot_moe_ffn_gated_backward", moe_bwd))
         for kw in SIZES]
CASES += [("convrot_moe_route", route(**kw), s) for kw, s in [
    (dict(dt=2), "DTYPE"), (dict(score=2), "SCORE"), (dict(score=-1), "SCORE"), (dict(l=None), "NULL"), (dict(ex=None), "NULL"),
    (dict(w=None), "NULL"), (dict(l=MIS), "ALIGN"), (dict(l=A + 1, dt=1), "ALIGN"), (dict(bias=MIS), "ALIGN"),
    (dict(ex=MIS), "ALIGN"), (dict(w=MIS), "ALIGN"), (dict(ex=C), "OVERLAP"), (dict(ex=A + 4), "OVERLAP"),
    (dict(w=A + 32 * 64 * 4 - 4), "OVERLAP"), (dict(bias=B), "OVERLAP"), (dict(bias=C + 32 * 8 * 4 - 4), "OVERLAP")]]
CASES += [("convrot_moe_route_backward", route_bwd(**kw), s) for kw, s in [
    (dict(dt=2), "DTYPE"), (dict(score=2), "SCORE"), (dict(dw=None), "NULL"), (dict(l=None), "NULL"), (dict(ex=None), "NULL"),
    (dict(dl=None), "NULL"), (dict(dl=MIS), "ALIGN"), (dict(dw=MIS), "ALIGN"), (dict(dl=A + 4), "OVERLAP"), (dict(dl=B), "OVERLAP"),
    (dict(dl=C - 4), "OVERLAP")]]
ROWS = [(dict(rows=-1), "SHAPE"), (dict(rows=1 << 26), "SHAPE"), (dict(groups=0), "SHAPE"), (dict(groups=1025), "SHAPE"),
        (dict(N=0), "SHAPE"), (dict(N=-1), "SHAPE"), (dict(K=100), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=131136), "SHAPE"),
        (dict(K=320), "SHAPE"), (dict(group=3), "GROUP"), (dict(group=512), "GROUP"), (dict(off=None), "NULL"),
        (dict(wq=None), "NULL"), (dict(sw=None), "NULL"), (dict(off=MIS), "ALIGN"), (dict(wq=MIS), "ALIGN"), (dict(sw=MIS), "ALIGN"),
        (dict(off=D + 4), "OVERLAP"), (dict(ws=None), "WORKSPACE"), (dict(ws=E + 16), "WORKSPACE"), (dict(wsb=100), "WORKSPACE")]
CASES += [(n, f(**kw), s) for n, f in (("convrot_linear_grouped", grouped), ("convrot_linear_grouped_backward", grouped_bwd))
          for kw, s in ROWS]
CASES += [("convrot_linear_grouped", grouped(**kw), s) for kw, s in [
    (dict(x=None), "NULL"), (dict(x=None, xq=A), "NULL"), (dict(x=None, xs=A), "NULL"), (dict(dt=7), "DTYPE"), (dict(x=MIS), "ALIGN"),
    (dict(y=None), "NULL"), (dict(y=MIS), "ALIGN"), (dict(N=1 << 24), "SHAPE"), (dict(rows=(1 << 26) - 1, N=(1 << 24) - 1), "SHAPE"),
    (dict(x=None, xq=D, xs=C), "OVERLAP"), (dict(x=None, xq=A, xs=D + 64), "OVERLAP")]]
CASES += [("convrot_linear_grouped_backward", grouped_bwd(**kw), s) for kw, s in [
    (dict(dy=None), "NULL"), (dict(dx=None), "NULL"), (dict(dy=MIS), "ALIGN"), (dict(dx=MIS), "ALIGN"), (dict(add=MIS), "ALIGN"),
    (dict(add=D + 16), "OVERLAP"), (dict(N=1 << 20), "SHAPE")]]
LAYER = [(dict(F=100), "SHAPE"), (dict(F=0), "SHAPE"), (dict(K=100), "SHAPE"), (dict(F=320, gh=128), "SHAPE"), (dict(gh=5), "GROUP"),
         (dict(group=0), "GROUP"), (dict(act=5), "ACT"), (dict(act=-1), "ACT"), (dict(M=1 << 20, K=4096), "SHAPE"), (dict(ex=None), "NULL"),
         (dict(w=None), "NULL"), (dict(wg=None), "NULL"), (dict(sg=None), "NULL"), (dict(wu=None), "NULL"), (dict(su=None), "NULL"),
         (dict(wd=None), "NULL"), (dict(sd=None), "NULL"), (dict(ex=MIS), "ALIGN"), (dict(w=MIS), "ALIGN"), (dict(wd=MIS), "ALIGN"),
         (dict(sd=MIS), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(ws=E + 64), "WORKSPACE"), (dict(wsb=1000), "WORKSPACE")]
CASES += [(n, f(**kw), s) for n, f in (("convrot_moe_ffn_gated", moe), ("convrot_moe_ffn_gated_backward", moe_bwd)) for kw, s in LAYER]
CASES += [("convrot_moe_ffn_gated", moe(**kw), s) for kw, s in [
    (dict(x=None), "NULL"), (dict(y=None), "NULL"), (dict(dt=3), "DTYPE"), (dict(x=MIS), "ALIGN"), (dict(res=MIS), "ALIGN"),
    (dict(pre=MIS), "ALIGN"), (dict(d=MIS), "ALIGN"), (dict(res=D + 16), "OVERLAP"), (dict(pre=D), "OVERLAP"), (dict(d=D + 256), "OVERLAP"),
    (dict(pre=J, d=J + 256), "OVERLAP"), (dict(pre=A), "OVERLAP"), (dict(d=A + 256), "OVERLAP"), (dict(res=J, d=J), "OVERLAP"),
    (dict(ex=D + 4), "OVERLAP"), (dict(w=D + 4), "OVERLAP"), (dict(pre=J, ex=J), "OVERLAP"), (dict(d=J, w=J), "OVERLAP")]]
CASES += [("convrot_moe_ffn_gated_backward", moe_bwd(**kw), s) for kw, s in [
    (dict(dy=None), "NULL"), (dict(pre=None), "NULL"), (dict(dx=None), "NULL"), (dict(d=None, dw=J), "NULL"), (dict(dy=MIS), "ALIGN"),
    (dict(pre=MIS), "ALIGN"), (dict(d=MIS), "ALIGN"), (dict(dx=MIS), "ALIGN"), (dict(add=MIS), "ALIGN"), (dict(dw=MIS), "ALIGN"),
    (dict(add=D + 16), "OVERLAP"), (dict(dw=D + 16), "OVERLAP"), (dict(dw=A), "OVERLAP"), (dict(dw=J), "OVERLAP"),
    (dict(dw=J + (1 << 28)), "OVERLAP"), (dict(dw=G), "OVERLAP"), (dict(dw=H), "OVERLAP"), (dict(add=J + (1 << 29), dw=J + (1 << 29)), "OVERLAP")]]

# calls that pass every check and stop at the missing device
VALID = [("convrot_moe_route", route()), ("convrot_moe_route", route(l=A + 2, dt=1, bias=J)), ("convrot_moe_route_backward", route_bwd()),
         ("convrot_moe_route_backward", route_bwd(dl=A)), ("convrot_linear_grouped", grouped()),
         ("convrot_linear_grouped", grouped(x=None, xq=A, xs=J, ws=None, wsb=0, N=33)), ("convrot_linear_grouped", grouped(y=A)),
         ("convrot_linear_grouped_backward", grouped_bwd()), ("convrot_linear_grouped_backward", grouped_bwd(add=D, N=33)),
         ("convrot_linear_grouped_backward", grouped_bwd(dx=A)), ("convrot_moe_ffn_gated", moe()), ("convrot_moe_ffn_gated", moe(res=D)),
         ("convrot_moe_ffn_gated", moe(y=A, pre=J, d=J + (1 << 28))), ("convrot_moe_ffn_gated_backward", moe_bwd()),
         ("convrot_moe_ffn_gated_backward", moe_bwd(add=D, d=None)), ("convrot_moe_ffn_gated_backward", moe_bwd(dx=A, dw=J + (1 << 29)))]
EMPTY = [("convrot_moe_route", route(M=0, l=None, ex=None, w=None)), ("convrot_moe_route_backward", route_bwd(M=0, dw=None, dl=None)),
         ("convrot_linear_grouped", grouped(rows=0, x=None, ws=None, y=None, off=None)),
         ("convrot_linear_grouped_backward", grouped_bwd(rows=0, dy=None, ws=None, dx=None)),
         ("convrot_moe_ffn_gated", moe(M=0, x=None, ex=None, ws=None, y=None)),
         ("convrot_moe_ffn_gated_backward", moe_bwd(M=0, dy=None, ws=None, dx=None))]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_refused(lib, i):
    name, args, status = CASES[i]
    with pytest.raises(cr.ConvRotError) as e:
        cr._call(name, *args)
    assert cr.STATUS[e.value.status] == "CONVROT_ERR_" + status, str(e.value)
    assert name in str(e.value)


@pytest.mark.parametrize("name,args", EMPTY)
def test_empty_is_a_no_op(lib, name, args):
    assert cr._call(name, *args) == 0


@pytest.mark.parametrize("i", range(len(VALID)))
def test_valid_calls_reach_the_device(lib, i):
    with pytest.raises(cr.ConvRotError) as e:
        cr._call(VALID[i][0], *VALID[i][1])
    assert cr.STATUS[e.value.status] == "CONVROT_ERR_HIP", str(e.value)


def test_workspace_queries(lib):
    assert cr.workspace_bytes_grouped(32, 4, 256, 512) >= 32 * 512 + 32 * 4
    assert cr.workspace_bytes_grouped_backward(32, 4, 256, 512) >= 32 * 256 * 2
    assert cr.workspace_bytes_grouped_backward(0, 4, 256, 512) == 0 and cr.workspace_bytes_moe_ffn_backward(0, 1, 4, 64, 64) == 0
    for bad in ((-1, 4, 256, 512), (1 << 26, 4, 256, 512), (1, 0, 256, 512), (1, 1025, 256, 512), (1, 1, 0, 512), (1, 1, 8, 100)):
        assert cr.workspace_bytes_grouped(*bad) == 0 and cr.workspace_bytes_grouped_backward(*bad) == 0
    for bad in ((-1, 2, 4, 64, 64), (1, 0, 4, 64, 64), (1, 5, 4, 64, 64), (1, 33, 64, 64, 64), (1, 1, 1025, 64, 64), (1, 1, 4, 65, 64),
                (1, 1, 4, 64, 0), (1 << 20, 1, 4, 64, 2048)):
        assert cr.workspace_bytes_moe_ffn(*bad) == 0 and cr.workspace_bytes_moe_ffn_backward(*bad) == 0
    # codes of x, h and its codes, and d in 16 bits with a scale per 64 channels
    assert cr.workspace_bytes_moe_ffn(9, 2, 4, 64, 128) > 9 * 128 + 18 * 64 * 3 + 18 * 128 * 2 + 18 * 2 * 4


def test_binding_checks():
    """Shapes, types and devices the binding refuses before the library sees a pointer."""
    f = torch.zeros
    with pytest.raises(ValueError, match="score is one of"):
        cr.moe_route(f(2, 4), 1, score="tanh")
    with pytest.raises(ValueError, match="is on cpu"):
        cr.moe_route(f(2, 4), 1)
    with pytest.raises(ValueError, match="is on cpu"):
        cr.moe_route_backward(f(2, 1), f(2, 4), f(2, 1, dtype=torch.int32))
    w, s = f(3, 64, 64, dtype=torch.int8), f(3, 64)
    with pytest.raises(ValueError, match="is on cpu"):
        cr.linear_grouped(f(2, 64), w, s, f(4, dtype=torch.int32), group=64)
    with pytest.raises(ValueError, match="give x"):
        cr.linear_grouped(None, w, s, f(4, dtype=torch.int32), group=64)
    with pytest.raises(ValueError, match="act is one of"):
        cr.moe_ffn_gated(f(2, 64), f(2, 1, dtype=torch.int32), f(2, 1), w, s, w, s, w, s, act="tanh", group=64, group_h=64)


W, SC = torch.zeros(3, 64, 64, dtype=torch.int8), torch.ones(3, 64)
X, EX, WT = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1)
HISTORY = {
    ("moe_route", "logits"): lambda t: cr.moe_route(t, 2),
    ("linear_grouped", "x"): lambda t: cr.linear_grouped(t, W, SC, torch.zeros(4, dtype=torch.int32), group=64),
    ("moe_ffn_gated", "x"): lambda t: cr.moe_ffn_gated(t, EX, WT, W, SC, W, SC, W, SC, group=64, group_h=64),
    ("moe_ffn_gated", "residual"): lambda t: cr.moe_ffn_gated(X, EX, WT, W, SC, W, SC, W, SC, residual=t, group=64, group_h=64),
    ("moe_ffn_gated", "weights"): lambda t: cr.moe_ffn_gated(X, EX, t[:, :1].float(), W, SC, W, SC, W, SC, group=64, group_h=64),
}


@pytest.mark.parametrize("call,name", HISTORY)
def test_warns_where_history_is_lost(call, name):
    run = HISTORY[call, name]
    with pytest.warns(UserWarning, match="%s .*%s_backward" % (call, call)), pytest.raises(ValueError, match="is on cpu"):
        run(X.clone().requires_grad_())
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="is on cpu"):
            run(X.clone())
        with torch.no_grad(), pytest.raises(ValueError, match="is on cpu"):
            run(X.clone().requires_grad_())


def _c_arg(value, ctype):
    return "%ff" % value if isinstance(value, float) else S._c_arg(value, ctype)


def _driver() -> str:
    call = lambda name, args: "%s(%s)" % (name, ", ".join(_c_arg(a, t) for a, t in zip(args, cr.SIGNATURES[name][0])))
    lines = ["#include <stdint.h>", "#include <stdio.h>", '#include "convrot.h"', "int main(void) {", "    int bad = 0;"]
    cases = [(n, a, ERR["CONVROT_ERR_" + s]) for n, a, s in CASES]
    cases += [(n, a, ERR["CONVROT_ERR_HIP"]) for n, a in VALID] + [(n, a, 0) for n, a in EMPTY]
    for i, (name, args, status) in enumerate(cases):
        lines.append('    if (%s != %d) { fprintf(stderr, "case %d %s: %%s\\n", convrot_last_error()); ++bad; }'
                     % (call(name, args), status, i, name))
    values = [1 << 62, 1 << 40, (1 << 31) - 1, (1 << 26) - 1, 1 << 20, 131072, -1, 0, 1, 17, 64]
    lines += ["    const int64_t v[] = {%s};" % ", ".join("(int64_t)%dll" % x for x in values), "    volatile size_t sink = 0;",
              "    const int n = (int)(sizeof v / sizeof v[0]);",
              "    for (int a = 0; a < n; ++a) for (int b = 0; b < n; ++b) for (int c = 0; c < n; ++c) for (int d = 0; d < n; ++d) {",
              "        sink += convrot_workspace_bytes_grouped(v[a], v[b], v[c], v[d]);",
              "        sink += convrot_workspace_bytes_grouped_backward(v[a], v[b], v[c], v[d]);",
              "        for (int t = -1; t < 34; t += 7) {",
              "            sink += convrot_workspace_bytes_moe_ffn(v[a], t, v[b], v[c], v[d]);",
              "            sink += convrot_workspace_bytes_moe_ffn_backward(v[a], t, v[b], v[c], v[d]);", "        }", "    }",
              "    (void)sink;", '    if (!bad) printf("all checks held\\n");', "    return bad != 0;", "}"]
    return "\n".join(lines) + "\n"


def test_host_code_under_asan_ubsan(tmp_path):
    if not (os.path.exists(S.HIPCC) and os.path.exists(S.CLANG)):
        pytest.skip("ROCm toolchain not available")
    if os.path.exists("/dev/kfd"):
        pytest.skip("host-only check (fake device pointers)")
    from int4_quantized_linear_amd import build as B_
    objs = [os.path.join(B_.HERE, "_build", s.replace(".hip", ".o")) for s in B_.SOURCES if s != "convrot_abi.hip"]
    if not all(os.path.exists(o) for o in objs):
        B_.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    abi = str(tmp_path / "abi.o")
    S._run([S.HIPCC, "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=" + B_.ARCH, *B_.DEVICE_FLAGS,
            "-Wno-unused-command-line-argument", *san, "-c", S.ABI_SRC, "-o", abi])
    source = tmp_path / "driver.c"
    source.write_text(_driver())
    driver = str(tmp_path / "driver.o")
    S._run([S.CLANG, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
            "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", S.INCLUDE, "-I", os.path.join(S.ROCM, "include"),
            "-c", str(source), "-o", driver])
    exe = str(tmp_path / "driver")
    S._run([S.HIPCC, "--offload-arch=" + B_.ARCH, *san, "-o", exe, driver, abi, *objs])
    assert "all checks held" in S._run([exe], env=dict(S.SAN_ENV, ASAN_OPTIONS="detect_leaks=0")).stdout


@pytest.mark.parametrize("name", ["grad_tile_kernelILb1E", "grad_gemm_kernelILb1E"])
def test_grouped_gradients_leave_m0_to_their_loads(name, tmp_path_factory):
    """The gradient kernels' own loads into LDS write m0, which an asm block cannot declare: nothing else may use it."""
    import re
    if not os.path.exists(S.HIPCC):
        pytest.skip("ROCm toolchain not available")
    if os.path.exists("/dev/kfd"):
        pytest.skip("host-only check")
    from int4_quantized_linear_amd import build as B_
    out = str(tmp_path_factory.mktemp("asm") / "grad.s")
    S._run([S.HIPCC, *B_.COMMON, *B_.DEVICE_FLAGS, "--cuda-device-only", "-S", os.path.join(B_.CSRC, "grad_i8.hip"), "-o", out])
    with open(out) as f:
        body = re.search(r"^_Z\w*%s\w*:.*?^\.Lfunc_end" % name, f.read(), re.M | re.S).group(0)
    outside = re.sub(r";APP.*?;NO_APP|;#ASMSTART.*?;#ASMEND", "", body, flags=re.S)
    assert len(re.findall(r"s_mov_b32 m0,", body)) == len(re.findall(r"buffer_load_dwordx4 .*lds", body)) > 0
    assert "v_mfma" in outside and not re.search(r"\bm0\b", outside)
