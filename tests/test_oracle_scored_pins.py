"""Pins of the scored-routing oracle: torch's softmax, sigmoid, top-k and
automatic differentiation, differences, and the plain softmax routing it
contains."""
import numpy as np
import pytest
import torch

import oracle
from oracle import moe_scored as S

CONFIGS = [dict(score=s, renormalise=r, scale=c) for s in ("softmax", "sigmoid") for r in (True, False) for c in (1.0, 2.5)]


def logits_of(T, E, seed=0):
    return np.random.default_rng(seed).normal(size=(T, E)).astype(np.float32)


def test_scores_are_torchs():
    l = logits_of(20, 12) * 3
    t = torch.from_numpy(l).double()
    np.testing.assert_allclose(S.scores(l, "softmax"), torch.softmax(t, 1), rtol=1e-14)
    np.testing.assert_allclose(S.scores(l, "sigmoid"), torch.sigmoid(t), rtol=1e-14)
    empty = np.full((1, 4), -np.inf)
    assert (S.scores(empty, "softmax") == 0).all() and (S.scores(empty, "sigmoid") == 0).all()


def test_softmax_routing_is_the_layers_own():
    l = logits_of(50, 16, 1)
    ids, gates = oracle.topk_route(l, 4)
    r = S.route(l, 4)
    assert (r["ids"] == ids).all()
    # (that oracle's gates are rounded to float32 once)
    np.testing.assert_allclose(r["gates"], gates, rtol=2.0 ** -24)


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_by_masking(score, top):
    """The usual way: values of groups by topk, the other groups masked out."""
    T, E, G, kept, k = 40, 24, 4, 2, 5
    l = logits_of(T, E, 2)
    bias = 0.2 * logits_of(1, E, 3)[0]
    c = torch.from_numpy(S.scores(l, score)) + torch.from_numpy(bias).double()
    value = c.view(T, G, -1).topk(top, 2).values.sum(2)
    keep = torch.zeros(T, G).scatter_(1, value.topk(kept, 1).indices, 1.0).bool()
    c = c.view(T, G, -1).masked_fill(~keep[:, :, None], -np.inf).view(T, E)
    r = S.route(l, k, score=score, bias=bias, groups=G, groups_kept=kept, group_top=top)
    assert (r["ids"] == c.topk(k, 1).indices.numpy()).all()
    assert all(keep[t, e // (E // G)] for t in range(T) for e in r["ids"][t])


def test_ties_and_masked_rows():
    r = S.route(np.zeros((1, 6)), 3)
    assert r["ids"].tolist() == [[0, 1, 2]]
    r = S.route(np.zeros((1, 6)), 2, bias=np.array([0, 0, 1, 1, 0, 0.0]))
    assert r["ids"].tolist() == [[2, 3]]
    r = S.route(np.full((1, 6), -np.inf), 3, scale=2.0)
    assert r["ids"].tolist() == [[0, 1, 2]] and (r["gates"] == 0).all()
    l = np.array([[np.nan, 1.0, -np.inf, 0.0]])
    assert S.route(l, 4, score="sigmoid")["ids"].tolist() == [[1, 3, 0, 2]]


@pytest.mark.parametrize("cfg", CONFIGS)
def test_backward_is_the_derivative(cfg):
    T, E, k = 6, 9, 3
    l = torch.from_numpy(logits_of(T, E, 4)).double().requires_grad_(True)
    r = S.route(l.detach().numpy(), k, **cfg)
    ids = torch.from_numpy(r["ids"]).long()
    s = torch.softmax(l, 1) if cfg["score"] == "softmax" else torch.sigmoid(l)
    g = s.gather(1, ids)
    if cfg["renormalise"]:
        g = g / g.sum(1, keepdim=True)
    g = cfg["scale"] * g
    np.testing.assert_allclose(r["gates"], g.detach(), rtol=1e-12)
    rng = np.random.default_rng(5)
    dg, dsum = rng.normal(size=(T, k)), rng.normal(size=E)
    (want,) = torch.autograd.grad((g * torch.from_numpy(dg)).sum() + (s.sum(0) * torch.from_numpy(dsum)).sum(), l)
    got, terms = S.route_backward(l.detach().numpy(), r["ids"], dg, dscore_sums=dsum, **cfg)
    np.testing.assert_allclose(got, want, rtol=1e-10, atol=1e-13)
    assert (np.abs(got) <= terms * (1 + 1e-12)).all()


@pytest.mark.parametrize("cfg", CONFIGS)
def test_backward_by_differences(cfg):
    T, E, k = 3, 7, 2
    l = logits_of(T, E, 6).astype(np.float64)
    r = S.route(l, k, **cfg)
    rng = np.random.default_rng(7)
    dg, dsum = rng.normal(size=(T, k)), rng.normal(size=E)

    def loss(v):
        q = S.route(v, k, **cfg)
        assert (q["ids"] == r["ids"]).all()
        return (q["gates"] * dg).sum() + (q["sums"] * dsum).sum()

    got, _ = S.route_backward(l, r["ids"], dg, dscore_sums=dsum, **cfg)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - got[t, e]) < 1e-7


def test_combine_backward_is_the_derivative():
    T, k, d = 5, 3, 8
    rng = np.random.default_rng(8)
    y = torch.from_numpy(rng.normal(size=(T * k, d))).requires_grad_(True)
    g = torch.from_numpy(rng.normal(size=(T, k))).requires_grad_(True)
    pos = rng.permutation(T * k).astype(np.int32)
    dy = rng.normal(size=(T, d))
    out = (g[:, :, None] * y[torch.from_numpy(pos).long()].view(T, k, d)).sum(1)
    np.testing.assert_allclose(oracle.combine(y.detach().numpy(), pos, g.detach().numpy()), out.detach(), rtol=1e-12)
    want_y, want_g = torch.autograd.grad((out * torch.from_numpy(dy)).sum(), (y, g))
    dy_perm, dgates, _ = S.combine_backward(dy, y.detach().numpy(), pos, g.detach().numpy())
    np.testing.assert_allclose(dy_perm, want_y, rtol=1e-12)
    np.testing.assert_allclose(dgates, want_g, rtol=1e-12)


def test_combine_backward_of_an_expert_elsewhere():
    dy_perm, dgates, _ = S.combine_backward(np.ones((1, 4)), np.ones((2, 4)), np.array([1, -1]), np.array([[2.0, 3.0]]))
    assert np.isnan(dy_perm[0]).all() and (dy_perm[1] == 2).all() and dgates.tolist() == [[4.0, 0.0]]
