"""Which kernels the sizes of the GPU tests reach, by the library's own rule on
the CPU: every kernel that the grouped products can launch is compared with
the oracle at some size, and the sizes that are meant for a kernel take it."""
import pytest

import grouped_choice
from grouped_helpers import QUEUES
from mixture_experts_layer_exclusive_amd import build as B
from test_gpu_grouped import CHOICES, LARGE, WIDTHS, ragged
from test_gpu_grouped_streams import ALONE, AT_ONCE, CUT, JOINT, STREAMS

# Every instance of the kernels: (type, output, mode, variant) of a product,
# (type, mode, variant, queues cut into parts) of a gradient alone, and the two
# variants of a joint launch.
FORWARD = [("bf16", "bf16", "NT", v) for v in ("split32", "split64", "tile64x128", "tile128", "tile256")]
FORWARD += [("f32", "f32", "NT", v) for v in ("split32", "tile64")]
FORWARD += [("int8", out, "NT", v) for out in ("bf16", "f32")
            for v in ("split32", "split64", "tile64x128", "tile128", "tile256")]
GRADIENTS = [("bf16", "NN", v, False) for v in ("split32", "split64", "tile64x128", "tile128", "tile256")]
GRADIENTS += [("f32", "NN", v, False) for v in ("split32", "tile64")]
GRADIENTS += [("bf16", "TN", v, cut) for v in ("tile128", "tile256") for cut in (False, True)]
GRADIENTS += [("f32", "TN", "tile128", False), ("f32", "TN", "tile128", True), ("f32", "TN", "tile256", False)]
GRADIENTS += [("bf16", "joint", v, "tile128", cut) for v in ("split32", "tile64x128", "tile128") for cut in (False, True)]
GRADIENTS += [("f32", "joint", v, "tile64", cut) for v in ("split32", "tile64") for cut in (False, True)]
GRADIENTS += [("f32", "joint", "split32", "tile128", cut) for cut in (False, True)]


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    try:
        B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    return grouped_choice.build(str(tmp_path_factory.mktemp("choice")))


def instances(problem, runs):
    op, dtype = problem[:2]
    for r in runs:
        if r[0] == "joint":
            yield (dtype, "joint", r[1], r[2], r[3] > 1)
        elif r[0] == "NT":
            yield ("int8" if op == "int8" else dtype, dtype, "NT", r[1])
        else:
            yield (dtype, r[0], r[1], r[2] > 1)


def sizes_of_the_gpu_tests():
    """The sizes that test_gpu_grouped and test_gpu_grouped_streams compare with
    the oracle (rows outside the queues included, as they count for the rule)."""
    for counts in QUEUES.values():
        rows = sum(counts) + 8
        for dtype in ("bf16", "f32"):
            for N, K in WIDTHS:
                if len(counts) * N * K > 4e7:
                    N, K = min(N, 136), min(K, 264)
                yield ("matmul", dtype, rows, len(counts), N, K)
                yield ("backward", dtype, rows, len(counts), N, K)
            for N, K in [(8, 16), (64, 128), (72, 48), (136, 272), (256, 1040), (520, 64), (1000, 528)]:
                if len(counts) * N * K > 4e7:
                    N, K = min(N, 136), min(K, 272)
                yield ("int8", dtype, rows, len(counts), N, K)
    for counts, N, K in LARGE.values():
        for dtype in ("bf16", "f32"):
            yield ("matmul", dtype, sum(counts) + 10, len(counts), N, K)
            yield ("backward", dtype, sum(counts) + 10, len(counts), N, K)
    for dtype in ("bf16", "f32"):
        counts = LARGE["ragged"][0]
        yield ("int8", dtype, sum(counts) + 10, len(counts), 2056, 528)
        for rows, N, K in [(1, 8, 16), (1, 4096, 2048), (16, 1000, 8208), (33, 136, 131056), (300, 520, 4096),
                           (4100, 2056, 528)]:
            yield ("int8", dtype, rows, 1, N, K)
    yield from CHOICES
    for op, dtype, rows, E, N, K in STREAMS + JOINT + ALONE:
        yield (op, dtype, rows + 8, E, N, K)


def test_every_kernel_is_compared_with_the_oracle(exe):
    sizes = list(sizes_of_the_gpu_tests())
    seen = {i for p, runs in zip(sizes, grouped_choice.kernels(exe, sizes)) for i in instances(p, runs)}
    missing = [i for i in FORWARD + GRADIENTS if i not in seen]
    assert not missing, missing
    assert not seen - set(FORWARD + GRADIENTS), seen - set(FORWARD + GRADIENTS)


@pytest.mark.parametrize("problem", STREAMS)
def test_streams_walk_several_tiles_of_several_slices(exe, problem):
    op, dtype, rows, E, N, K = problem
    runs = grouped_choice.kernels(exe, [(op, dtype, rows + 8, E, N, K)])[0]
    mode, variant = runs[0][:2]
    assert variant == "tile256" and mode == ("NN" if op == "backward" else "NT")
    width, length = (K, N) if mode == "NN" else (N, K)
    of = 128 if op == "int8" else 64          # values of a slice
    columns = -(-width // 256)
    tiles = sum(-(-c // 256) for c in ragged(rows, E, seed=rows)) * columns
    assert tiles > 512 and length > 2 * of and length % of != 0 and width % 256 != 0


def test_streams_have_both_tile_orders():
    """Each of the forward, the 8-bit product by output and the input gradient."""
    kinds = {(op, dtype) for op, dtype, *_ in STREAMS}
    for kind in kinds:
        columns = [-(-(K if op == "backward" else N) // 256) for op, dtype, _, _, N, K in STREAMS if (op, dtype) == kind]
        assert min(columns) <= 8 < max(columns), kind


def test_sizes_of_the_other_streams_tests(exe):
    rows, E, N, K = AT_ONCE
    problems = [(op, "bf16", rows, E, N, K) for op in ("matmul", "int8", "backward")]
    runs = [r for rs in grouped_choice.kernels(exe, problems) for r in rs]
    assert [r[1] for r in runs] == ["tile256"] * 4
    cut = grouped_choice.kernels(exe, [("backward", "bf16", CUT["rows"], CUT["E"], CUT["N"], CUT["K"])])[0]
    assert cut[-1][-2] > 1


def test_cut_weight_gradient_alone(exe):
    (op, dtype, rows, E, N, K), = ALONE
    runs = grouped_choice.kernels(exe, [(op, dtype, rows + 8, E, N, K)])[0]
    assert runs[0][:2] == ("NN", "tile256") and runs[1][:2] == ("TN", "tile128") and runs[1][2] > 1


def test_joint_sizes_are_joint(exe):
    for p, runs in zip(JOINT, grouped_choice.kernels(exe, [(p[0], p[1], p[2] + 8, *p[3:]) for p in JOINT])):
        assert runs[0][0] == "joint" and runs[0][3] > 1, (p, runs)
