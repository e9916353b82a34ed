"""Which kernels of the scored routing and of its gradient the sizes of
test_gpu_scored_kernels reach, by the library's own rule (``csrc/scored_plan.h``, compiled
for the host): every kernel is compared with the oracle, with and without groups; and its
many tokens are more than the workgroups and waves take at a time."""
import itertools
import subprocess

import pytest

from mixture_experts_layer_exclusive_amd import build as B
from test_gpu_scored_kernels import BACK, LISTS, ROUTES

PROGRAM = r"""
#include "scored_plan.h"
#include <cstdio>
using namespace moe;
int main() {
    int E, k;
    while (scanf("%d %d", &E, &k) == 2) {
        moe_gating_t g{};
        g.E = E;
        g.k = k;
        const RouteKernel r = route_kernel(g);
        const RouteBackKernel b = route_back_kernel(g);
        printf("%d %d %d %d %d %d\n", r.lanes, r.per_lane, int(r.words), r.list, b.lanes, int(b.words));
    }
}
"""


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
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

    def of(sizes):
        text = "".join("%d %d\n" % s for s in sizes)
        out = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, timeout=60)
        rows = [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
        return [r[:4] for r in rows], [r[4:] for r in rows]
    return of


ALL_SIZES = [(E, k) for E in range(1, 257) for k in range(1, min(E, 32) + 1)]
SHAPES = [(4, 8), (8, 8), (16, 8), (16, 16)]


def test_every_routing_kernel_is_compared_with_the_oracle(kernels):
    possible = set(kernels(ALL_SIZES)[0])
    assert possible == {(*s, w, n) for s, w, n in itertools.product(SHAPES, (0, 1), (4, 8, 16))} | {(64, 4, 0, 0)}
    tested = set(kernels([(E, min(k, E)) for E, _, _ in ROUTES for k in LISTS])[0])
    # (the whole wave's: test_many_tokens_per_wave)
    assert tested == possible - {(64, 4, 0, 0)}


def test_groups_are_of_whole_lanes_and_of_others_in_every_shape(kernels):
    seen = set()
    for E, groups, _ in ROUTES:
        (lanes, per_lane, _, _), = kernels([(E, 1)])[0]
        assert E % groups == 0
        lanes_of_group = E // groups / per_lane
        seen.add((lanes, per_lane, lanes_of_group in (1, 2, 4, 8)))
    assert seen == {(*s, whole) for s in SHAPES for whole in (True, False)}


def test_every_gradient_kernel_is_compared_with_the_oracle(kernels):
    possible = set(kernels(ALL_SIZES)[1])
    assert possible == set(itertools.product((4, 8, 16, 32), (0, 1)))
    assert set(kernels(BACK)[1]) == possible


def test_many_tokens_are_several_rounds(kernels):
    for T, E, k in [(40001, 256, 8), (40001, 250, 3), (20011, 100, 12), (70001, 62, 4), (140001, 24, 4), (9001, 96, 17),
                    (8200, 256, 32), (9001, 3, 2), (12289, 2, 1), (16387, 1, 1)]:
        (lanes, _, _, _), = kernels([(E, k)])[0]
        assert T > 1024 * 4 * (64 // lanes)
