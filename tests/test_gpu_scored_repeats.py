"""The gradient of the scored routing where ids name an expert more than once: the
slots' gradients add up in the slots' order."""
import itertools

import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from test_gpu_scored import check_backward, f64, gpu, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sums", [True, False])
@pytest.mark.parametrize("E", [20, 30, 64, 100, 127, 200, 256])
def test_sums_in_the_order_of_the_slots(E, sums):
    """Sums whose float32 value depends on the order: a + 1 - a is 0, a - a + 1 is 1."""
    big = 2.0 ** 26
    for a, b, c in ((0, 1, 2), (0, 4, 8), (3, 8, 16), (1, 17, 18)):
        for values in itertools.permutations((big, 1.0, -big)):
            ids = np.tile(np.arange(19, dtype=np.int32), (9, 1))
            ids[:, [a, b, c]] = 19
            ids[4] = np.arange(19)            # a token without repeats
            dg = np.zeros((9, 19), np.float32)
            dg[:, [a, b, c]] = 4 * np.array(values, np.float32)
            dl = moe.route_scored_backward(gpu(np.zeros((9, E), np.float32)), gpu(ids), gpu(dg), score="sigmoid",
                                           renormalise=False, dscore_sums=gpu(np.zeros(E, np.float32)) if sums else None)
            want = np.float32(values[0])
            for v in values[1:]:
                want = np.float32(want + np.float32(v))
            got = f64(dl)[:, 19]
            assert (got[np.arange(9) != 4] == want).all() and got[4] == 0
            assert (f64(dl)[4, [a, b, c]] == values).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(3, 2), (8, 5), (30, 7), (62, 12), (128, 32), (250, 9), (256, 8)])
def test_against_the_definition(E, k, dtype):
    ids = np.random.default_rng(E).integers(0, min(E, 6), (33, k)).astype(np.int32)
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            for sums in (True, False):
                check_backward(logits_of(33, E, E), k, sums=sums, score=score, renormalise=renormalise, ids=ids, dtype=dtype)
