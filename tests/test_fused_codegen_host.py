"""What the gradient kernels' source assumes of the compiler, checked on the assembly it makes of them (CPU only)."""
import os
import re

import pytest

from tests import test_host_sanitizers as S

KERNELS = ("grad_tile_kernel", "grad_gemm_kernel")


@pytest.fixture(scope="module")
def bodies(tmp_path_factory):
    """name -> lines of the kernel's body outside the source's own asm blocks."""
    if not os.path.exists(S.HIPCC):
        pytest.skip("ROCm toolchain not available")
    if os.path.exists("/dev/kfd"):
        pytest.skip("host-only check")
    from int4_quantized_linear_amd import build as B
    out = str(tmp_path_factory.mktemp("asm") / "grad.s")
    S._run([S.HIPCC, *B.COMMON, *B.DEVICE_FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "grad_i8.hip"), "-o", out])
    with open(out) as f:
        text = f.read()
    got = {}
    for name in KERNELS:
        body = re.search(r"^_Z\w*%s\w*:.*?^\.Lfunc_end" % name, text, re.M | re.S).group(0)
        got[name] = (body, re.sub(r";APP.*?;NO_APP|;#ASMSTART.*?;#ASMEND", "", body, flags=re.S))
    return got


@pytest.mark.parametrize("name", KERNELS)
def test_only_the_loads_into_lds_use_m0(bodies, name):
    body, outside = bodies[name]
    assert len(re.findall(r"s_mov_b32 m0,", body)) == len(re.findall(r"buffer_load_dwordx4 .*lds", body)) > 0
    assert "v_mfma" in outside and not re.search(r"\bm0\b", outside)
