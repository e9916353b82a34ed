"""Routing by scores, its gradient and the combine's gradient on the GPU against
the float64 oracle (``oracle.moe_scored``).

Chosen experts are compared exactly: the order is decided in 64 bits on both
sides, and no two of the drawn scores agree to 48 bits but those that are equal.
Bounds of the floats, u = 2^-24:

* a softmax score: the exponent l - max is rounded once (|l - max| u in the
  result), exp is good to 2 ulp, the sum has at most E roundings, the quotient
  one: (D + E + 8) u, D the largest |l - max| of the row; a sigmoid 6 u
* a gate: a score, over a sum of k more of them if renormalised, times scale: two
  such errors and k + 3 roundings
* a score sum: a score's error and at most 64 roundings of partial sums
* a logit's gradient: products and sums of those, at most 2 E + 2 k + 16
  roundings and 4 scores, times the sum of the terms' absolute values
* a slot's dot product: d + 1 roundings
and what lies below 2^-126 may be anything below it.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from oracle import moe_scored as S

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 2.0 ** -126


def gpu(a, dtype=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def score_error(logits, score):
    """Relative error of a float32 score, [T, 1]."""
    l = np.asarray(logits, np.float64)
    if score == "sigmoid":
        return np.full((l.shape[0], 1), 6 * U)
    finite = np.where(np.isfinite(l), l, -np.inf)
    top = finite.max(1, keepdims=True)
    D = np.where(np.isfinite(l), top - np.where(np.isfinite(l), l, 0), 0).max(1, keepdims=True)
    return (np.minimum(D, 110) + l.shape[1] + 8) * U


def near(got, ref, bound, what):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0], got[bad][0], ref[bad][0], np.broadcast_to(bound, ref.shape)[bad][0])


def check_route(logits, k, bias=None, with_sums=True, **cfg):
    T, E = logits.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    gates = torch.full((T, k), 3e4, device=DEV)
    out = moe.route_scored(k, logits=gpu(logits), bias=gpu(bias), ids=ids, gates=gates, with_score_sums=with_sums, **cfg)
    torch.cuda.synchronize()
    r = S.route(logits, k, bias=bias, **cfg)
    got = out[0].cpu().numpy()
    assert (got == r["ids"]).all(), np.argwhere(got != r["ids"])[:3]
    e = score_error(logits, cfg.get("score", "softmax"))
    near(f64(out[1]), r["gates"], (2 * e + (k + 3) * U) * np.abs(r["gates"]) + TINY, "gates")
    if with_sums:
        near(f64(out[3]), r["sums"], ((e + 64 * U) * r["scores"]).sum(0) + TINY * max(T, 1), "sums")
    return out


def logits_of(T, E, seed, spread=2.0):
    return (spread * np.random.default_rng(seed).normal(size=(T, E))).astype(np.float32)


def bias_of(E, seed):
    return (0.1 * np.random.default_rng(1000 + seed).normal(size=E)).astype(np.float32)


GROUPS = [  # E, k, groups, kept, group_top
    (256, 8, 8, 4, 2), (256, 8, 8, 4, 1), (256, 32, 16, 3, 2), (24, 3, 3, 1, 2), (160, 6, 8, 3, 1), (60, 5, 5, 5, 2),
    (12, 4, 6, 2, 2), (9, 2, 9, 4, 2), (256, 12, 256, 20, 1), (8, 1, 2, 1, 2), (250, 7, 2, 1, 2), (64, 6, 8, 4, 2),
    (128, 4, 4, 2, 1), (48, 8, 3, 2, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,kept,top", GROUPS)
def test_groups(E, k, groups, kept, top, score):
    l = logits_of(77, E, E + k)
    check_route(l, k, bias=bias_of(E, E), score=score, groups=groups, groups_kept=kept, group_top=top, scale=2.5)
    check_route(l, k, score=score, groups=groups, groups_kept=kept, group_top=top, renormalise=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (2, 2), (3, 2), (8, 2), (31, 4), (64, 6), (65, 8), (128, 8), (129, 9),
                                 (200, 17), (255, 32), (256, 8), (256, 32)])
def test_no_groups(E, k, score):
    l = logits_of(65, E, 3 * E + k)
    check_route(l, k, score=score)
    check_route(l, k, score=score, bias=bias_of(E, k), renormalise=False, scale=0.5)


@pytest.mark.parametrize("T", [0, 1, 2, 3, 31, 32, 33, 127, 1000])
def test_tokens(T):
    check_route(logits_of(T, 40, T), 4, bias=bias_of(40, 0), score="sigmoid", groups=4, groups_kept=2)


def test_many_tokens():
    check_route(logits_of(5000, 256, 9), 8, bias=bias_of(256, 9), score="sigmoid", groups=8, groups_kept=4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties(score):
    """Quarters: many equal scores, in one group and across them."""
    rng = np.random.default_rng(4)
    l = (rng.integers(-4, 5, (300, 64)) / 4).astype(np.float32)
    check_route(l, 8, score=score)
    check_route(l, 8, score=score, groups=8, groups_kept=3)
    check_route(l, 8, score=score, groups=8, groups_kept=3, group_top=1)
    check_route(np.zeros((5, 64), np.float32), 8, score=score, groups=8, groups_kept=2)
    b = (rng.integers(0, 2, 64) / 2).astype(np.float32)
    check_route(np.zeros((5, 64), np.float32), 8, score=score, bias=b, groups=8, groups_kept=3)
    check_route(np.zeros((5, 64), np.float32), 8, score=score, bias=b)


def test_close_scores_are_in_order():
    """Scores that differ in their last float32 bits, or in none of them, but not
    in 64 bits."""
    rng = np.random.default_rng(5)
    base = rng.normal(size=(200, 1)).astype(np.float32)
    l = (base * (1 + rng.integers(-3, 4, (200, 64)) * np.float32(2.0 ** -23))).astype(np.float32)
    b = (0.25 + rng.integers(-2, 3, 64) * 2.0 ** -25).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        check_route(l, 8, score=score, bias=b)
        check_route(l, 8, score=score, bias=b, groups=8, groups_kept=3)
        check_route(l, 8, score=score, groups=8, groups_kept=3)


def test_far_logits():
    """Softmax and sigmoid scores over many orders of magnitude."""
    l = logits_of(100, 32, 6, spread=12.0)
    check_route(l, 4, score="softmax")
    check_route(l, 4, score="sigmoid", bias=bias_of(32, 6))
    check_route(l, 4, score="sigmoid", renormalise=False)


def test_masked_experts_and_rows():
    l = logits_of(40, 24, 7)
    l[:, 5] = -np.inf
    l[3] = -np.inf
    l[4, 1:] = -np.inf
    for score in ("softmax", "sigmoid"):
        for cfg in ({}, dict(groups=4, groups_kept=2), dict(bias=bias_of(24, 7)),
                    dict(bias=bias_of(24, 7), groups=4, groups_kept=2)):
            out = check_route(l, 3, score=score, **cfg)
            assert (f64(out[1])[3] == 0).all()
    low = np.where(np.isneginf(l), np.finfo(np.float32).min, l)
    check_route(low, 3, score="sigmoid", bias=bias_of(24, 7))
    b = bias_of(24, 8)
    b[[0, 7]] = -np.inf     # experts out of service
    out = check_route(np.where(np.isneginf(l), 0, l), 3, score="sigmoid", bias=b)
    assert not np.isin(out[0].cpu().numpy(), [0, 7]).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("cfg", [{}, dict(groups=4, groups_kept=2), dict(bias=True), dict(bias=True, groups=8, groups_kept=3),
                                 dict(groups=4, groups_kept=2, group_top=1)])
def test_any_bits_give_different_experts(score, cfg):
    rng = np.random.default_rng(8)
    l = rng.integers(0, 2 ** 32, (400, 24), dtype=np.uint32).view(np.float32).copy()
    l[::3] = np.where(rng.random((134, 24)) < 0.5, np.nan, np.inf)
    cfg = dict(cfg)
    bias = rng.integers(0, 2 ** 32, 24, dtype=np.uint32).view(np.float32) if cfg.pop("bias", False) else None
    ids, _, _ = moe.route_scored(6, logits=gpu(l), score=score, bias=gpu(bias), **cfg)
    ids = np.sort(ids.cpu().numpy(), 1)
    assert (ids[:, 0] >= 0).all() and (ids[:, -1] < 24).all() and (np.diff(ids, axis=1) > 0).all()


def test_nan_comes_last():
    l = logits_of(30, 16, 10)
    l[:, 3] = np.nan
    for cfg in ({}, dict(bias=bias_of(16, 1))):
        ids, gates, _ = moe.route_scored(15, logits=gpu(l), score="sigmoid", bias=gpu(cfg.get("bias")))
        assert not (ids == 3).any() and torch.isfinite(gates).all()
        ids, gates, _ = moe.route_scored(16, logits=gpu(l), score="sigmoid", bias=gpu(cfg.get("bias")))
        assert (ids[:, 15] == 3).all() and torch.isnan(gates).all()
    _, gates, _ = moe.route_scored(4, logits=gpu(l))
    assert torch.isnan(gates).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_product(dtype):
    """x and w_router: the logits are moe.route's, and the choice is made on them."""
    g = torch.Generator().manual_seed(0)
    x, w = (torch.randn(n, 128, generator=g).to(dtype).to(DEV) for n in (100, 48))
    w = w * 0.1
    ids, gates, logits, sums = moe.route_scored(4, x=x, w_router=w, score="sigmoid", groups=4, groups_kept=2,
                                                with_score_sums=True)
    _, _, plain = moe.route(4, x=x, w_router=w)
    assert torch.equal(logits, plain)
    a = moe.route_scored(4, logits=logits, score="sigmoid", groups=4, groups_kept=2, with_score_sums=True)
    assert torch.equal(a[0], ids) and torch.equal(a[1], gates) and torch.equal(a[3], sums)
    check_route(logits.cpu().numpy(), 4, score="sigmoid", groups=4, groups_kept=2)


def test_softmax_without_bias_is_route():
    l = gpu(logits_of(300, 64, 11))
    a, b = moe.route(6, logits=l), moe.route_scored(6, logits=l)
    assert torch.equal(a[0], b[0])
    near(f64(a[1]), f64(b[1]), 200 * U * f64(b[1]), "gates")


def test_workspace_is_enough_and_undefined():
    T, E = 700, 48
    l = gpu(logits_of(T, E, 12))
    n = moe.route_scored_workspace_size(T, E, 4)
    buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    a = moe.route_scored(4, logits=l, with_score_sums=True, ws=buf[:n])
    assert (buf[n:] == 0xFF).all()
    b = moe.route_scored(4, logits=l, with_score_sums=True)
    assert torch.equal(a[3], b[3])
    with pytest.raises(moe.MoeError, match="WORKSPACE"):
        moe.route_scored(4, logits=l, with_score_sums=True, ws=buf[:n - 4])


# ---- the gradient -------------------------------------------------------------

def check_backward(logits, k, seed=0, sums=True, dtype=torch.float32, ids=None, **cfg):
    T, E = logits.shape
    rng = np.random.default_rng(seed)
    ids = S.route(logits, k, score=cfg.get("score", "softmax"))["ids"] if ids is None else ids
    dg = rng.normal(size=(T, k)).astype(np.float32)
    ds = rng.normal(size=E).astype(np.float32) if sums else None
    dl = torch.full((T, E), 3e4, dtype=dtype, device=DEV)
    got = moe.route_scored_backward(gpu(logits), gpu(ids), gpu(dg), dscore_sums=gpu(ds), dtype=dtype, dlogits=dl, **cfg)
    torch.cuda.synchronize()
    assert got is dl
    ref, terms = S.route_backward(logits, ids, dg, dscore_sums=ds, **cfg)
    e = score_error(logits, cfg.get("score", "softmax"))
    half = 0 if dtype == torch.float32 else 2.0 ** -8
    bound = (4 * e + (2 * E + 2 * k + 16) * U) * terms
    near(f64(got), ref, bound * (1 + half) + half * np.abs(ref) + TINY, "dlogits")
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (3, 1), (8, 2), (62, 6), (64, 8), (65, 12), (130, 9), (255, 32), (256, 8)])
def test_backward(E, k, score, renormalise, dtype):
    l = logits_of(70, E, E)
    for sums in (True, False):
        check_backward(l, k, sums=sums, score=score, renormalise=renormalise, scale=2.5, dtype=dtype)


@pytest.mark.parametrize("T", [0, 1, 2, 5, 63, 4099])
def test_backward_tokens(T):
    check_backward(logits_of(T, 40, T), 4, score="sigmoid")


def test_backward_masked_and_far():
    l = logits_of(40, 24, 7)
    l[:, 5] = -np.inf
    l[3] = -np.inf
    l[4, 1:] = -np.inf
    far = logits_of(50, 24, 8, spread=10.0)
    for score in ("softmax", "sigmoid"):
        for r in (True, False):
            got = check_backward(l, 3, score=score, renormalise=r)
            assert (f64(got)[3] == 0).all() and (f64(got)[:, 5] == 0).all()
            check_backward(far, 3, score=score, renormalise=r)


def test_backward_of_chosen_experts_of_small_scores():
    """A bias chooses experts whose scores are tiny: their shares are not."""
    l = logits_of(30, 16, 9)
    l[:, :4] -= 80
    ids = np.tile(np.arange(4, dtype=np.int32), (30, 1))
    check_backward(l, 4, score="sigmoid", ids=ids)
    check_backward(l, 4, score="softmax", ids=ids)


def test_backward_by_differences():
    """Against differences of the forward itself."""
    T, E, k = 4, 12, 3
    l = logits_of(T, E, 3)
    rng = np.random.default_rng(1)
    dg, ds = rng.normal(size=(T, k)).astype(np.float32), rng.normal(size=E).astype(np.float32)
    for cfg in (dict(score="softmax"), dict(score="sigmoid", scale=2.0), dict(score="softmax", renormalise=False)):
        ids, *_ = moe.route_scored(k, logits=gpu(l), **cfg)
        got = f64(moe.route_scored_backward(gpu(l), ids, gpu(dg), dscore_sums=gpu(ds), **cfg))
        h = 2.0 ** -7
        # every token and expert at once: token t's loss depends on its own logits
        # only (sums: by one token's score at a time)
        for e in range(E):
            at = []
            for sign in (1, -1):
                v = l.copy()
                v[:, e] += np.float32(sign * h)
                same, g, _ = moe.route_scored(k, logits=gpu(v), **cfg)
                assert torch.equal(same, ids)
                at.append((f64(g) * dg).sum(1) + (S.scores(v, cfg["score"]) * ds).sum(1))
            # roundings: k gates of error 30 u each; curvature: third derivatives
            # below 8 of each of k + E terms
            bound = 2 * 40 * U * (np.abs(dg).sum(1) * 2 + 1) / (2 * h) + 8 * (np.abs(dg).sum(1) + np.abs(ds).sum()) * h * h / 6
            assert (np.abs((at[0] - at[1]) / (2 * h) - got[:, e]) <= bound).all()


def test_backward_same_expert_twice():
    """(not what a routing gives, but defined: the slots' gradients add up)"""
    l = logits_of(10, 8, 2)
    ids = np.tile(np.array([3, 3], np.int32), (10, 1))
    dg = np.random.default_rng(3).normal(size=(10, 2)).astype(np.float32)
    got = f64(moe.route_scored_backward(gpu(l), gpu(ids), gpu(dg), renormalise=False))
    ref, terms = S.route_backward(l, ids, dg, renormalise=False)
    near(got, ref, 100 * U * terms + TINY, "twice")


# ---- the combine's gradient ------------------------------------------------------

def check_combine(T, k, d, dtype, seed=0, away=0.0, order=None):
    rng = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(rng.normal(size=s)).to(dtype)  # noqa: E731
    dy, y = t(T, d), t(T * k, d)
    gates = rng.normal(size=(T, k)).astype(np.float32)
    pos = rng.permutation(T * k).astype(np.int32) if order is None else order
    pos = np.where(rng.random(T * k) < away, -1, pos).astype(np.int32)
    out = dict(dy_perm=torch.full((T * k, d), 3e4, dtype=dtype, device=DEV), dgates=torch.full((T, k), 3e4, device=DEV))
    g = moe.combine_backward(dy.to(DEV), gpu(pos), gpu(gates), y_perm=y.to(DEV), out=out)
    torch.cuda.synchronize()
    ref, dgates, terms = S.combine_backward(f64(dy), f64(y), pos, gates)
    near(f64(g["dgates"]), dgates, (d + 1) * U * terms + TINY, "dgates")
    got = f64(g["dy_perm"])
    none = np.isnan(ref)
    assert (got[none] == f64(torch.tensor(3e4, dtype=dtype))).all()
    half = U if dtype == torch.float32 else 2.0 ** -8 * (1 + 2 * U) + U
    near(got[~none], ref[~none], half * np.abs(ref[~none]) + TINY, "dy_perm")
    alone = moe.combine_backward(dy.to(DEV), gpu(pos), gpu(gates), y_perm=y.to(DEV), with_dy_perm=False)
    assert alone["dy_perm"] is None and torch.equal(alone["dgates"], g["dgates"])
    out = dict(dy_perm=torch.full((T * k, d), 3e4, dtype=dtype, device=DEV))
    other = moe.combine_backward(dy.to(DEV), gpu(pos), gpu(gates), with_dgates=False, out=out)
    assert other["dgates"] is None and torch.equal(other["dy_perm"], g["dy_perm"])


@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 9, 32])
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (192, torch.bfloat16), (2048, torch.bfloat16),
                                     (4160, torch.bfloat16), (1, torch.float32), (7, torch.float32),
                                     (520, torch.float32), (1025, torch.float32), (2052, torch.float32)])
def test_combine_backward(d, dtype, k):
    check_combine(19, k, d, dtype, seed=d + k)


@pytest.mark.parametrize("T", [0, 1, 2, 1001])
def test_combine_backward_tokens(T):
    check_combine(T, 2, 128, torch.bfloat16, seed=T)
    check_combine(T, 2, 36, torch.float32, seed=T)


@pytest.mark.parametrize("d", [2, 3, 4, 5, 6, 63, 64, 65, 67, 190, 192, 193, 255, 257])
def test_combine_backward_short_rows(d):
    """Rows of any number of floats, each beginning at any float, by 16, 64 and 256 lanes."""
    for T, k in ((1, 1), (17, 2), (33, 3), (101, 8), (5, 9)):
        check_combine(T, k, d, torch.float32, seed=d + T, away=0.2)


@pytest.mark.parametrize("d", [64, 128, 320, 384, 448])
def test_combine_backward_short_rows_bf16(d):
    for T, k in ((1, 1), (17, 2), (33, 3), (101, 8), (5, 9)):
        check_combine(T, k, d, torch.bfloat16, seed=d + T, away=0.2)


@pytest.mark.parametrize("d", [5, 6, 7, 67, 257, 1027])
def test_combine_backward_counts_every_column_once(d):
    """Small whole numbers, whose sums are exact, and an infinity in the columns that two
    loads hold."""
    rng = np.random.default_rng(d)
    T, k = 9, 2
    dy, y = (rng.integers(-4, 5, s).astype(np.float32) for s in ((T, d), (T * k, d)))
    pos = rng.permutation(T * k).astype(np.int32)
    y[pos[0], d - 4:] = dy[0, d - 4:] = 1.0
    y[pos[0], d - 4] = np.inf
    gates = np.ones((T, k), np.float32)
    g = moe.combine_backward(gpu(dy), gpu(pos), gpu(gates), y_perm=gpu(y))
    want = np.einsum("td,tkd->tk", dy, y[pos].reshape(T, k, d))
    assert np.isinf(want[0, 0]) and np.array_equal(g["dgates"].cpu().numpy(), want)
    assert np.array_equal(g["dy_perm"].cpu().numpy()[pos], np.repeat(dy, k, 0))


def test_combine_backward_with_experts_elsewhere():
    check_combine(50, 4, 128, torch.bfloat16, away=0.4)
    check_combine(50, 4, 10, torch.float32, away=1.0)


def test_combine_backward_of_dispatch():
    T, E, k = 200, 16, 4
    ids, _, _ = moe.route_scored(k, logits=gpu(logits_of(T, E, 1)))
    q = moe.dispatch(ids, E)
    check_combine(T, k, 256, torch.bfloat16, order=q["assign_pos"].cpu().numpy())


# ---- graphs, streams ---------------------------------------------------------------

def test_captured_and_replayed():
    """All of them in one captured graph, replayed on new inputs, with eager work
    and synchronisations between the replays."""
    T, E, k, d = 257, 64, 6, 128
    l, x = gpu(logits_of(T, E, 1)), torch.randn(T, d, device=DEV).bfloat16()
    y, dy = torch.randn(T * k, d, device=DEV).bfloat16(), torch.randn(T, d, device=DEV).bfloat16()
    bias, ds = gpu(bias_of(E, 1)), torch.randn(E, device=DEV)

    def step():
        ids, gates, _, sums = moe.route_scored(k, logits=l, score="sigmoid", bias=bias, groups=8, groups_kept=4,
                                               with_score_sums=True)
        q = moe.dispatch(ids, E, x=x, with_x_perm=True)
        g = moe.combine_backward(dy, q["assign_pos"], gates, y_perm=y)
        dl = moe.route_scored_backward(l, ids, g["dgates"], score="sigmoid", dscore_sums=ds)
        return ids, gates, sums, g["dy_perm"], g["dgates"], dl

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(5):
        l.copy_(gpu(logits_of(T, E, 20 + seed)))
        y.copy_(torch.randn(T * k, d, device=DEV).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = [h.clone() for h in held]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    T, E, k = 3000, 128, 8
    ins = [gpu(logits_of(T, E, s)) for s in (1, 2)]
    want = [moe.route_scored(k, logits=l, score="sigmoid", groups=4, groups_kept=2, with_score_sums=True) for l in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        got = []
        for s, l in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(moe.route_scored(k, logits=l, score="sigmoid", groups=4, groups_kept=2, with_score_sums=True))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
