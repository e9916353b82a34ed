"""Groups valued by sums where a bias is infinite: sums of infinities are infinities,
equal ones go to the lower group, and infinities of both signs sum to a NaN, which
comes last."""
import numpy as np
import pytest

from test_gpu_scored import check_route, logits_of

pytestmark = pytest.mark.gpu

INF = np.inf


def bias_of(E, at):
    b = np.zeros(E, np.float32)
    for e, v in at.items():
        b[e] = v
    return b


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(24, 4), (32, 4), (64, 4), (250, 5), (256, 8)])
def test_infinite_values_are_equal(E, groups, score):
    size = E // groups
    one, two = 1, 2 * size
    b = bias_of(E, {one: INF, two: INF, two + 1: INF})
    for k, kept in ((1, 1), (4, 1), (4, 2)):
        out = check_route(logits_of(20, E, E), k, bias=b, score=score, groups=groups, groups_kept=kept)
        ids = out[0].cpu().numpy()
        assert (ids < size).all() or kept == 2
        assert (ids[:, 0] == one).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(24, 4), (32, 4), (64, 4), (250, 5), (256, 8)])
def test_infinities_of_both_signs_come_last(E, groups, score):
    size = E // groups
    at = {e: -INF for e in range(size, 2 * size)}
    at[size] = INF                        # group 1: infinity and minus infinity
    at.update({e: -1000.0 for e in range(size)})
    b = bias_of(E, at)
    out = check_route(logits_of(20, E, E), 3, bias=b, score=score, groups=groups, groups_kept=groups - 1)
    assert not (out[0].cpu().numpy() // size == 1).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_infinite_biases_without_groups(score):
    b = bias_of(40, {3: INF, 17: INF, 5: -INF, 30: INF, 2: -INF})
    check_route(logits_of(20, 40, 1), 5, bias=b, score=score)
    check_route(logits_of(20, 40, 1), 5, bias=b, score=score, groups=8, groups_kept=3, group_top=1)
