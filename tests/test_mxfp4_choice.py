"""Which kernels the sizes of the 4-bit product's GPU tests reach, by the library's
own rule (``csrc/grouped_plan.h``, compiled for the host): every kernel is compared
with the oracle at some size, in both output types."""
import subprocess

import pytest

from grouped_helpers import QUEUES
from mixture_experts_layer_exclusive_amd import build as B
from test_gpu_mxfp4 import CHOICES, DENSE, LARGE, WIDTHS

PROGRAM = r"""
#include "grouped_plan.h"
#include <cstdio>
using namespace moe;
int main() {
    long rows;
    int E, N, K, f32;
    while (scanf("%ld %d %d %d %d", &rows, &E, &N, &K, &f32) == 5) {
        const moe_grouped_t g{rows, E, N, K, f32 ? MOE_DTYPE_F32 : MOE_DTYPE_BF16};
        printf("%d\n", short_mxfp4(g) ? 9 : static_cast<int>(plan_mxfp4(g).v));
    }
}
"""
SPLIT32, SPLIT64, TILE64X128, TILE128, TILE256, HALVES64X128, HALVES128, TILE128X256, SHORT = 0, 1, 3, 4, 5, 6, 7, 8, 9


def sizes():
    for counts in QUEUES.values():
        for N, K in WIDTHS:
            if len(counts) * N * K > 4e7:
                N, K = min(N, 136), min(K, 288)
            yield sum(counts) + 8, len(counts), N, K
    for counts, N, K in LARGE.values():
        yield sum(counts) + 10, len(counts), N, K
    for rows, N, K in DENSE:
        yield rows, 1, N, K
    for _, rows, E, N, K in CHOICES:
        yield rows, E, N, K


@pytest.fixture(scope="module")
def variants(tmp_path_factory):
    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.hip").write_text(PROGRAM)
    r = subprocess.run([cc, "--cuda-host-only", "-std=c++17", "-O1", f"-I{B.INCLUDE}", f"-I{B.CSRC}",
                        str(d / "choice.hip"), "-o", str(d / "choice")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr

    def of(problems):
        text = "".join("%d %d %d %d %d\n" % p for p in problems)
        out = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, timeout=60)
        return [int(v) for v in out.stdout.split()]
    return of


def test_every_kernel_is_compared_with_the_oracle(variants):
    for f32 in (0, 1):
        seen = set(variants([(*s, f32) for s in sizes()]))
        assert seen == {SPLIT32, SPLIT64, TILE64X128, TILE128, TILE256, HALVES64X128, HALVES128, TILE128X256,
                        SHORT}


def test_sizes_meant_for_a_kernel_take_it(variants):
    names = dict(split32=SPLIT32, split64=SPLIT64, tile64x128=TILE64X128, tile128=TILE128, tile256=TILE256,
                 short=SHORT, halves64x128=HALVES64X128, halves128=HALVES128, tile128x256=TILE128X256)
    for name, rows, E, N, K in CHOICES:
        for f32 in (0, 1):
            assert variants([(rows, E, N, K, f32)]) == [names[name]], (name, rows, E, N, K)
