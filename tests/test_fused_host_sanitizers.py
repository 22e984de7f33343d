"""The fused entry points' host code under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only): the refusals of
test_fused_host.py, empty inputs, calls that pass every check and stop at the missing device, and the size queries at their
edges.  Any report ends the driver with a non-zero status."""
import os

import pytest

from tests import test_host_sanitizers as S


def _driver() -> str:
    from tests import test_fused_host as T
    cr = T.cr
    call = lambda name, args: "%s(%s)" % (name, ", ".join(S._c_arg(a, t) for a, t in zip(args, cr.SIGNATURES[name][0])))
    lines = ["#include <stdint.h>", "#include <stdio.h>", '#include "convrot.h"', "int main(void) {", "    int bad = 0;"]
    cases = [(n, a, T.ERR["CONVROT_ERR_" + s]) for n, a, s in T.CASES]
    cases += [(n, a, T.ERR["CONVROT_ERR_HIP"]) for n, a in T.VALID] + [(n, a, 0) for n, a in T.EMPTY]
    for i, (name, args, status) in enumerate(cases):
        lines.append('    if (%s != %d) { fprintf(stderr, "case %d %s: %%s\\n", convrot_last_error()); ++bad; }'
                     % (call(name, args), status, i, name))
    values = [1 << 62, 1 << 40, 1 << 31, (1 << 31) - 1, 1 << 24, 1 << 20, 131072, -1, 0, 1, 17, 64]
    lines += ["    const int64_t v[] = {%s};" % ", ".join("(int64_t)%dll" % x for x in values),
              "    volatile size_t sink = 0;", "    const int n = (int)(sizeof v / sizeof v[0]);",
              "    for (int a = 0; a < n; ++a) for (int b = 0; b < n; ++b) for (int c = 0; c < n; ++c) {"]
    for q in ("act", "gated", "ffn", "backward", "gated_backward", "ffn_backward"):
        lines.append("        sink += convrot_workspace_bytes_%s(v[a], v[b], v[c]);" % q)
    lines += ["    }", "    (void)sink;", '    if (!bad) printf("all checks held\\n");', "    return bad != 0;", "}"]
    return "\n".join(lines) + "\n"


def test_fused_host_code_under_asan_ubsan(tmp_path):
    if not (os.path.exists(S.HIPCC) and os.path.exists(S.CLANG)):
        pytest.skip("ROCm toolchain not available")
    if os.path.exists("/dev/kfd"):
        pytest.skip("host-only check (fake device pointers)")
    pytest.importorskip("int4_quantized_linear_amd.convrot")
    from int4_quantized_linear_amd import build as B
    objs = [os.path.join(B.HERE, "_build", s.replace(".hip", ".o")) for s in B.SOURCES if s != "convrot_abi.hip"]
    if not all(os.path.exists(o) for o in objs):
        B.build()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    abi = str(tmp_path / "abi.o")
    S._run([S.HIPCC, "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=" + B.ARCH, *B.DEVICE_FLAGS,
            "-Wno-unused-command-line-argument", *san, "-c", S.ABI_SRC, "-o", abi])
    source = tmp_path / "driver.c"
    source.write_text(_driver())
    driver = str(tmp_path / "driver.o")
    S._run([S.CLANG, "-std=c11", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
            "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", S.INCLUDE, "-I", os.path.join(S.ROCM, "include"),
            "-c", str(source), "-o", driver])
    exe = str(tmp_path / "driver")
    S._run([S.HIPCC, "--offload-arch=" + B.ARCH, *san, "-o", exe, driver, abi, *objs])
    assert "all checks held" in S._run([exe], env=dict(S.SAN_ENV, ASAN_OPTIONS="detect_leaks=0")).stdout
