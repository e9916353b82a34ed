"""Every kernel of the scored routing and of its gradient against the float64 oracle
(test_scored_choice shows that these sizes reach them), many tokens per workgroup and
wave, and rows of the combine's gradient that its lanes go over more than once.
Bounds as in test_gpu_scored."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from oracle import moe_scored as S
from test_gpu_scored import (DEV, TINY, U, bias_of, check_backward, check_combine, check_route, f64, gpu, logits_of, near,
                             score_error)

pytestmark = pytest.mark.gpu

# experts, groups (whole lanes where they can be), groups kept
ROUTES = [(4, 2, 1), (28, 7, 4), (30, 5, 3), (32, 4, 2), (33, 3, 2), (62, 2, 1), (64, 8, 4), (66, 6, 2), (100, 4, 2),
          (126, 7, 3), (128, 8, 4), (129, 3, 2), (160, 5, 3), (192, 12, 5), (250, 10, 4), (256, 8, 4)]
LISTS = [1, 3, 4, 5, 7, 8, 9, 12, 16]
BACK = [(4, 2), (20, 6), (31, 3), (32, 32), (36, 4), (61, 8), (64, 20), (68, 4), (100, 9), (127, 8), (128, 8), (128, 32),
        (132, 6), (160, 17), (201, 8), (256, 32)]


@pytest.mark.parametrize("k", LISTS)
@pytest.mark.parametrize("E,groups,kept", ROUTES)
def test_routing(E, groups, kept, k):
    if k > E:
        k = E
    l = logits_of(70, E, 7 * E + k)
    check_route(l, k, score="softmax")
    check_route(l, k, score="softmax", bias=bias_of(E, k), scale=2.5)
    check_route(l, k, score="sigmoid", bias=bias_of(E, k), renormalise=False)
    kept = max(kept, -(-k * groups // E))
    for score, top in (("sigmoid", 2), ("softmax", 1)):
        check_route(l, k, score=score, bias=bias_of(E, k), groups=groups, groups_kept=kept, group_top=top)
        check_route(l, k, score=score, groups=groups, groups_kept=kept, group_top=top)


def settled(logits, k, bias=None, score="softmax", groups=1, groups_kept=None, group_top=2):
    """Rows whose choice 64 bits settle: what it compares (values of groups, c of experts
    that stay) is equal because it is made of the same logits and biases, or differs by
    more than 2^-48.  A score in 64 bits is off by at most 3 roundings of values up to 1 and
    an exponential's ulp (a softmax's sum moves all of a row's scores by the same share), 4
    2^-53, its sum with a bias below 2 by one more of values up to 2, a sum of two of those
    by another: 2 (4 + 2) + 2 = 14 2^-53, a difference of two such by 28 2^-53 < 2^-48."""
    r = S.route(logits, k, score=score, bias=bias, groups=groups, groups_kept=groups_kept, group_top=group_top)
    T, E = logits.shape
    b = np.zeros(E) if bias is None else bias
    size = E // groups

    def apart(values, made_of):
        order = sorted(range(len(values)), key=lambda i: -values[i])
        return all(values[i] - values[j] > 2.0 ** -48 or made_of[i] == made_of[j] for i, j in zip(order, order[1:]))

    clear = np.zeros(T, bool)
    for t in range(T):
        c, parts = r["order"][t], [(float(v), float(w)) for v, w in zip(logits[t], b)]
        ok = True
        if groups_kept is not None and groups_kept < groups:
            best = [sorted(range(q * size, (q + 1) * size), key=lambda e: -c[e])[:group_top] for q in range(groups)]
            ok = apart([sum(c[e] for e in q) for q in best], [sorted(parts[e] for e in q) for q in best])
        live = sorted((e for e in range(E) if r["stay"][t, e]), key=lambda e: -c[e])[:k + 1]
        clear[t] = ok and apart([c[e] for e in live], [parts[e] for e in live])
    return clear


def check_settled(logits, k, bias=None, **cfg):
    """check_route of the rows that 64 bits settle; all rows are k different experts."""
    clear = settled(logits, k, bias=bias, **cfg)
    ids, _, _ = moe.route_scored(k, logits=gpu(logits), bias=gpu(bias), **cfg)
    assert (np.diff(np.sort(ids.cpu().numpy(), 1), axis=1) > 0).all()
    if clear.any():
        out = check_route(np.ascontiguousarray(logits[clear]), k, bias=bias, **cfg)
        assert (ids.cpu().numpy()[clear] == out[0].cpu().numpy()).all()


@pytest.mark.parametrize("k", LISTS)
@pytest.mark.parametrize("E,groups,kept", ROUTES)
def test_routing_in_64_bits(E, groups, kept, k):
    """Quarters: many equal scores; and scores that differ in their last float32 bits."""
    if k > E:
        k = E
    kept = max(kept, -(-k * groups // E))
    rng = np.random.default_rng(E + k)
    quarters = (rng.integers(-4, 5, (33, E)) / 4).astype(np.float32)
    base = rng.normal(size=(33, 1)).astype(np.float32)
    close = (base * (1 + rng.integers(-3, 4, (33, E)) * np.float32(2.0 ** -23))).astype(np.float32)
    for l, b in ((quarters, rng.integers(0, 2, E) / 2), (close, 0.25 + rng.integers(-2, 3, E) * 2.0 ** -25)):
        b = b.astype(np.float32)
        check_settled(l, k, score="sigmoid", bias=b)
        check_settled(l, k, score="softmax", bias=b, groups=groups, groups_kept=kept)
        check_settled(l, k, score="sigmoid", groups=groups, groups_kept=kept)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", BACK)
def test_gradient(E, k, dtype):
    l = logits_of(70, E, E)
    for score in ("softmax", "sigmoid"):
        for sums in (True, False):
            for renormalise in (True, False):
                check_backward(l, k, sums=sums, score=score, renormalise=renormalise, scale=2.5, dtype=dtype)


# ---- many tokens ------------------------------------------------------------------

def check_many(l, k, score, bias):
    """check_route without groups, for many tokens at once; the inputs are such that 64
    bits leave no choice open."""
    T, E = l.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    gates = torch.full((T, k), 3e4, device=DEV)
    _, _, _, sums = moe.route_scored(k, logits=gpu(l), score=score, bias=gpu(bias), ids=ids, gates=gates,
                                     with_score_sums=True)
    torch.cuda.synchronize()
    s = S.scores(l, score)
    c = s + bias.astype(np.float64)
    order = np.argsort(-c, axis=1, kind="stable")
    sorted_c = np.take_along_axis(c, order[:, :k + 1], 1)
    gap = sorted_c[:, :-1] - sorted_c[:, 1:]
    same = np.diff(np.take_along_axis(l, order[:, :k + 1], 1), axis=1) == 0
    assert ((gap > 2.0 ** -50) | ((gap == 0) & same)).all()
    want = order[:, :k]
    got = ids.cpu().numpy()
    assert (got == want).all(), np.argwhere(got != want)[:3]
    chosen = np.take_along_axis(s, want, 1)
    ref = chosen / chosen.sum(1, keepdims=True)
    e = score_error(l, score)
    near(f64(gates), ref, (2 * e + (k + 3) * U) * ref + TINY, "gates")
    near(f64(sums), s.sum(0), ((e + 64 * U) * s).sum(0) + TINY * T, "sums")


@pytest.mark.parametrize("T,E,k", [(40001, 256, 8), (40001, 250, 3), (20011, 100, 12), (70001, 62, 4), (140001, 24, 4)])
def test_choices_again_in_every_round(T, E, k):
    """More tokens than the workgroups take at a time, most of them (every one in two
    thirds of the rows) with scores that only 64 bits tell apart."""
    rng = np.random.default_rng(T + E)
    base = rng.normal(size=(T, 1)).astype(np.float32)
    l = (base * (1 + rng.integers(-3, 4, (T, E)) * np.float32(2.0 ** -23))).astype(np.float32)
    l[::3] = 2 * rng.normal(size=l[::3].shape)
    bias = (0.25 + rng.integers(-2, 3, E) * 2.0 ** -25).astype(np.float32)
    check_many(l, k, "sigmoid", bias)


@pytest.mark.parametrize("T,E,k", [(9001, 96, 17), (8200, 256, 32), (9001, 3, 2), (12289, 2, 1), (16387, 1, 1)])
def test_many_tokens_per_wave(T, E, k):
    check_many(logits_of(T, E, T), k, "softmax", bias_of(E, k))


# ---- the combine's gradient ---------------------------------------------------------

@pytest.mark.parametrize("k", [1, 2, 8, 9])
@pytest.mark.parametrize("T,d,dtype", [(300, 2112, torch.bfloat16), (257, 4096, torch.bfloat16), (300, 7168, torch.bfloat16),
                                       (300, 1025, torch.float32), (257, 2051, torch.float32), (300, 4099, torch.float32),
                                       (19, 8256, torch.bfloat16), (19, 16448, torch.bfloat16), (19, 4099, torch.float32),
                                       (19, 8193, torch.float32)])
def test_combine_backward_in_several_passes(T, d, dtype, k):
    check_combine(T, k, d, dtype, seed=d + k, away=0.1)
