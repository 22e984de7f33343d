"""Which kernel the backward tests' sizes run on: the tile and slice choice is a model of measured constants, so a refit
could move a size to another kernel and leave one untested without any test failing.  The choice is compiled
for the host from its own source (256 CUs, as without a GPU) and compared with what the tests mean to cover."""
import os

import pytest

from tests import test_gpu_fused_backward_tiles as tiles
from tests import test_gpu_fused_precision as precision
from tests import test_host_sanitizers as S

# (M, N, K, gated) -> tokens per tile, some tiles whole, some sliced, ragged last step of a weight
WANT = {
    (12, 16128, 5376, 0): (64, 0, 1, 0), (300, 16128, 640, 0): (64, 0, 1, 0), (4096, 2048, 2048, 0): (64, 1, 0, 0),
    (1024, 5120, 5120, 0): (256, 0, 1, 0), (4096, 16128, 2048, 0): (256, 0, 1, 0), (5, 524288, 128, 0): (64, 0, 1, 0),
    (600, 1048575, 64, 0): (64, 0, 1, 1),
    (12, 25600, 1024, 1): (64, 0, 1, 0), (2752, 1000, 1536, 1): (64, 1, 0, 1), (4096, 1024, 4096, 1): (256, 1, 0, 0),
    (4096, 1001, 4096, 1): (256, 1, 0, 1), (1728, 65, 4864, 1): (256, 1, 0, 1), (2048, 25600, 5120, 1): (256, 0, 1, 0),
    (2048, 9001, 5120, 1): (256, 0, 1, 1), (1100, 16100, 1280, 1): (256, 0, 1, 1),
    # the blocks' two steps
    (4096, 4096, 2944, 0): (256, 1, 0, 0), (4096, 2944, 4096, 1): (256, 1, 0, 0),
    (1500, 4096, 3008, 0): (256, 0, 1, 0), (1500, 3008, 4096, 1): (256, 0, 1, 0),
    (2048, 5120, 9024, 0): (256, 1, 1, 0), (2048, 9024, 5120, 1): (256, 0, 1, 0),
}

DRIVER = """
#include "%s"
#include <stdio.h>
#include <stdlib.h>
int main(int argc, char **argv)
{
    for (int i = 1; i + 3 < argc; i += 4) {
        const long M = atol(argv[i]), N = atol(argv[i + 1]);
        const convrot::Plan p = convrot::make_plan(M, N, atoi(argv[i + 2]), atoi(argv[i + 3]) != 0);
        const int T = p.tiles_m * p.tiles_c;
        printf("%%d %%d %%d %%d\\n", p.bm, p.T_dp > 0, p.S > 1 && p.T_dp < T, N %% 64 != 0);
    }
    return 0;
}
"""


def test_tests_run_on_the_kernels_they_mean(tmp_path):
    if not os.path.exists(S.HIPCC):
        pytest.skip("ROCm toolchain not available")
    if os.path.exists("/dev/kfd"):
        pytest.skip("host-only check")
    from int4_quantized_linear_amd import build as B
    used = [(M, N, K, 0) for M, N, K, _ in precision.LINEAR]
    used += [(M, N, K, 1) for M, N, K, _ in precision.GATED + tiles.GATED]
    used += [s for M, K, F in tiles.BLOCKS for s in ((M, K, F, 0), (M, F, K, 1))]
    assert set(used) == set(WANT)
    source = tmp_path / "plans.hip"
    source.write_text(DRIVER % os.path.join(B.CSRC, "grad_i8.hip"))
    exe = str(tmp_path / "plans")
    S._run([S.HIPCC, "-O1", "-std=c++17", "--offload-arch=" + B.ARCH, *B.DEVICE_FLAGS, "-Wno-unused-command-line-argument",
            "-o", exe, str(source)])
    sizes = list(WANT)
    out = S._run([exe, *[str(v) for s in sizes for v in s]]).stdout.split("\n")
    got = {s: tuple(int(v) for v in line.split()) for s, line in zip(sizes, out)}
    assert got == WANT
