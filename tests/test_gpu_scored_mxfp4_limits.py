"""Scored routing, the combine's gradient and the 4-bit floats where element numbers
and byte offsets pass 32 bits: sampled rows against the oracle.  And large calls at
once on two streams."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from grouped_helpers import check, f64, offsets_of
from oracle import moe_mxfp4 as M, moe_scored as S

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def samples(n, count=40):
    return np.unique(np.concatenate([np.random.default_rng(0).integers(0, n, count), [0, 1, n - 2, n - 1]]))


def test_routing_of_over_2_32_logit_bytes():
    T, E, k = 9_000_003, 256, 4
    l = torch.empty(T, E, device=DEV).normal_()
    assert l.numel() > 2 ** 31
    bias = torch.linspace(-0.1, 0.1, E, device=DEV)
    cfg = dict(score="sigmoid", scale=2.0)
    ids, gates, _, sums = moe.route_scored(k, logits=l, bias=bias, groups=8, groups_kept=4, with_score_sums=True, **cfg)
    at = samples(T)
    rows = l[torch.from_numpy(at).to(DEV)].cpu().numpy()
    r = S.route(rows, k, bias=bias.cpu().numpy(), groups=8, groups_kept=4, **cfg)
    assert (ids[torch.from_numpy(at).to(DEV)].cpu().numpy() == r["ids"]).all()
    np.testing.assert_allclose(f64(gates[torch.from_numpy(at).to(DEV)]), r["gates"], rtol=2e-6)
    # each score is good to 6 2^-24, and at most 64 roundings of partial sums
    ref = torch.zeros(E, dtype=torch.float64, device=DEV)
    for i in range(0, T, 1_000_000):
        ref += torch.sigmoid(l[i:i + 1_000_000].double()).sum(0)
    np.testing.assert_allclose(f64(sums), f64(ref), rtol=70 * 2.0 ** -24)
    dg = torch.randn(T, k, device=DEV)
    dl = moe.route_scored_backward(l, ids, dg, **cfg)
    pick = torch.from_numpy(at).to(DEV)
    want, terms = S.route_backward(rows, r["ids"], dg[pick].cpu().numpy(), **cfg)
    assert (np.abs(f64(dl[pick]) - want) <= 600 * 2.0 ** -24 * terms + 2.0 ** -126).all()


def test_combine_gradient_of_over_2_32_bytes():
    T, k, d = 300_007, 4, 2048
    dy, y = (torch.empty(n, d, dtype=torch.bfloat16, device=DEV).normal_() for n in (T, T * k))
    assert y.numel() > 2 ** 31
    gates = torch.randn(T, k, device=DEV)
    pos = torch.randperm(T * k, device=DEV).int()
    g = moe.combine_backward(dy, pos, gates, y_perm=y)
    at = samples(T)
    for t in at:
        p = pos[t * k:(t + 1) * k].long()
        ref, dgates, terms = S.combine_backward(f64(dy[t:t + 1]), f64(y[p]), np.arange(k), f64(gates[t:t + 1]))
        got = f64(g["dy_perm"][p])
        assert (np.abs(got - ref) <= 2.0 ** -8 * 1.01 * np.abs(ref) + 2.0 ** -126).all()
        assert (np.abs(f64(g["dgates"][t]) - dgates[0]) <= (d + 1) * 2.0 ** -24 * terms[0]).all()


def test_quantising_over_2_32_values():
    rows, cols = 70_001, 65_536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV).normal_()
    assert x.numel() > 2 ** 32
    codes, scales = moe.quantize_rows_mxfp4(x)
    at = samples(rows, 12)
    pick = torch.from_numpy(at).to(DEV)
    want, sw = M.quantize_rows(x[pick].float().cpu().numpy())
    assert (codes[pick].cpu().numpy() == want).all() and (scales[:, pick].cpu().numpy() == sw).all()
    del x
    v = moe.dequantize_rows_mxfp4(codes, scales)
    assert (f64(v[pick]) == M.dequantize_rows(want, sw)).all()


def test_product_of_over_2_32_bytes_of_codes():
    E, N, K = 40, 16384, 16384
    counts = [1, 0, 2] + [1] * 36 + [70]
    off = offsets_of(counts)
    R = int(off[-1])
    codes = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device=DEV)  # noqa: E731
    bytes_ = lambda *s: torch.randint(124, 131, s, dtype=torch.uint8, device=DEV)  # noqa: E731
    a, sa, w, sw = codes(R, K // 2), bytes_(K // 256, R, 8), codes(E, N, K // 2), bytes_(K // 256, E, N, 8)
    assert w.numel() > 2 ** 32
    c = moe.grouped_matmul_mxfp4(a, sa, w, sw, torch.from_numpy(off).to(DEV), out_dtype=torch.float32)
    cols = samples(N, 30)
    pick = torch.from_numpy(cols).to(DEV)
    for e in (0, 2, 21, 38, 39):
        lo, hi = int(off[e]), int(off[e + 1])
        ref, terms = M.matmul(a[lo:hi].cpu().numpy(), sa[:, lo:hi].cpu().numpy(), w[e][pick][None].cpu().numpy(),
                              sw[:, e][:, pick][:, None].cpu().numpy(), [0, hi - lo])
        check(c[lo:hi][:, pick], ref, terms, K, "f32", f"expert {e}")


def test_large_calls_at_once_on_two_streams():
    counts = [[2900, 1, 0, 2555, 3556], [4000, 4012, 0, 0, 1000]]
    N, K = 4360, 800
    made = []
    for i, c in enumerate(counts):
        g = torch.Generator(device=DEV).manual_seed(i)
        x = torch.randn(9012, K, generator=g, device=DEV).bfloat16()
        w = moe.quantize_rows_mxfp4(torch.randn(5 * N, K, generator=g, device=DEV).bfloat16())
        made.append((x, w[0].view(5, N, -1), w[1].view(-1, 5, N, 8), torch.from_numpy(offsets_of(c)).to(DEV)))

    def run(x, w, sw, off):
        a, sa = moe.quantize_rows_mxfp4(x)
        return moe.grouped_matmul_mxfp4(a, sa, w, sw, off)

    want = [run(*m) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(4):
        got = []
        for s, m in zip(streams, made):
            with torch.cuda.stream(s):
                got.append(run(*m))
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, counts):
            n = sum(c)
            assert torch.equal(a[:n], b[:n])
