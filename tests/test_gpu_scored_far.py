"""Shares of chosen experts whose scores are tiny: a bias chooses experts whose logits
lie so far below the row's largest (softmax) or below zero (sigmoid) that their scores
are float32 denormals or zeros.  Their shares of each other are not tiny.

Bounds as in test_gpu_scored: the exponent of a share is the difference to the largest
chosen logit, at most D."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from test_gpu_scored import U, check_backward, check_route, f64, gpu, logits_of, near

pytestmark = pytest.mark.gpu

FAR = [60, 87, 92, 97, 102, 120, 300, 600]


def far_logits(E, chosen, by, seed):
    l = logits_of(33, E, seed)
    l[:, :chosen] -= by
    return l


def choosing(E, chosen):
    """Biases that choose the experts below `chosen`, in an order of their own."""
    b = np.zeros(E, np.float32)
    b[:chosen] = 8 + np.random.default_rng(chosen).permutation(chosen) / 4
    return b


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(3, 2), (24, 4), (30, 7), (64, 6), (126, 12), (256, 8), (250, 16), (256, 24)])
def test_gates(E, k, score):
    for by in FAR:
        l = far_logits(E, k, by, E + k)
        if score == "sigmoid":
            l[:, k:] -= by
        check_route(l, k, score=score, bias=choosing(E, k), scale=2.5)
        check_route(l, k, score=score, bias=choosing(E, k), renormalise=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gates_chosen_again_in_64_bits(score):
    """Equal biases: the choice is never certain in 32 bits."""
    b = np.zeros(64, np.float32)
    b[8:20] = 4
    for by in FAR[1:]:
        l = far_logits(64, 32, by, 3)
        # (equal logits and biases, whose order is that of the numbers, whatever the bits)
        l[:, 8:20] = l[:, 8:9]
        l[:, 8:14] -= 1
        b[8:14] = 5
        check_route(l, 8, score=score, bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gates_of_experts_without_a_score(score):
    """Chosen experts at minus infinity, all of them or all but one far below."""
    l = logits_of(20, 24, 1)
    l[:, :4] = -np.inf
    l[10:, 2] = -150.0
    b = choosing(24, 4)
    out = check_route(l, 4, score=score, bias=b)
    gates = out[1].cpu().numpy()
    assert (gates[:10] == 0).all() and (np.sort(gates[10:], 1) == [0, 0, 0, 1]).all()


def test_a_nan_enters_the_gates_of_all_experts_of_a_softmax():
    l = far_logits(24, 4, 95, 1)
    for value in (np.nan, np.inf):
        l[:, 23] = value
        for k in (4, 20):
            ids, gates, _ = moe.route_scored(k, logits=gpu(l), bias=gpu(choosing(24, k)))
            assert not (ids == 23).any() and torch.isnan(gates).all()


@pytest.mark.parametrize("E,k", [(3, 2), (24, 4), (256, 8), (250, 16), (256, 24)])
@pytest.mark.parametrize("score,by", [("softmax", 725), ("softmax", 900), ("softmax", 5000), ("sigmoid", 690)])
def test_gates_at_the_end_of_64_bits(E, k, score, by):
    """Scores that are denormals or zeros in 64 bits, too: the shares are those of
    exp(l - m)."""
    l = far_logits(E, k, by, E + k)
    ids, gates, _ = moe.route_scored(k, logits=gpu(l), bias=gpu(choosing(E, k)), score=score)
    assert (torch.sort(ids, 1).values.cpu() == torch.arange(k)).all()
    chosen = np.take_along_axis(l, ids.cpu().numpy().astype(np.int64), 1).astype(np.float64)
    w = np.exp(chosen - chosen.max(1, keepdims=True))
    near(f64(gates), w / w.sum(1, keepdims=True), 2 * U, "gates")


@pytest.mark.parametrize("E,k", [(3, 2), (24, 4), (256, 8), (256, 24)])
def test_sigmoid_gates_that_are_zero_in_64_bits(E, k):
    """1 / (1 + exp(725)): the exponential overflows 64 bits above 709.8."""
    for by in (725, 5000):
        l = far_logits(E, k, by, E + k)
        ids, gates, _ = moe.route_scored(k, logits=gpu(l), bias=gpu(choosing(E, k)), score="sigmoid")
        assert (torch.sort(ids, 1).values.cpu() == torch.arange(k)).all() and (gates == 0).all()


# ---- the gradient ------------------------------------------------------------------

@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(3, 2), (24, 4), (62, 7), (128, 12), (256, 8)])
def test_gradient(E, k, score, renormalise):
    for by in FAR:
        l = far_logits(E, k, by, E + k)
        ids = np.tile(np.random.default_rng(k).permutation(k).astype(np.int32), (len(l), 1))
        for sums in (True, False):
            check_backward(l, k, sums=sums, score=score, renormalise=renormalise, ids=ids, scale=2.5)


@pytest.mark.parametrize("sums", [True, False])
def test_gradient_of_gates_that_are_zero(sums):
    """No gradient through the gates of chosen experts whose scores are all zero: the
    others' and the sums' only."""
    for score, value in (("sigmoid", -5000.0), ("sigmoid", np.finfo(np.float32).min), ("sigmoid", -np.inf), ("softmax", -np.inf)):
        l = logits_of(20, 64, 5)
        l[:, :6] = value
        ids = np.tile(np.arange(6, dtype=np.int32), (20, 1))
        got = check_backward(l, 6, sums=sums, score=score, ids=ids)
        assert (got[:, :6] == 0).all() and (sums or (got == 0).all())
