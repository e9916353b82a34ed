"""Routing by scores, the combine's gradient and the 4-bit floats on the CPU:
argument checks of the C ABI and of the binding, before any HIP call (no kernel
is launched)."""
import ctypes
import os
import re

import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from mixture_experts_layer_exclusive_amd import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000    # never dereferenced
MIS = 0x10004  # not 16-byte aligned
BIG = 1 << 40
OK, INV, UNS, WS = L.MOE_OK, L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE_TOO_SMALL
F32, BF16 = L.MOE_DTYPE_F32, L.MOE_DTYPE_BF16


@pytest.fixture(scope="module")
def lib():
    return L.load()


def gat(T=64, d=128, dtype=BF16, E=64, k=6, score=0, groups=8, groups_kept=4, group_top=2, renormalise=1, scale=1.0):
    return L.MoeGating(T=T, d=d, dtype=dtype, E=E, k=k, score=score, groups=groups, groups_kept=groups_kept,
                       group_top=group_top, renormalise=renormalise, scale=scale)


def route(lib, g, x=None, w=None, li=A, lo=None, bias=A, ids=A, gates=A, sums=A, ws=A, n=BIG):
    return lib.moe_route_scored(ctypes.byref(g), x, w, li, lo, bias, ids, gates, sums, ws, n, None)


def back(lib, g, logits=A, ids=A, dgates=A, dsums=A, dtype=F32, dl=A):
    return lib.moe_route_scored_backward(ctypes.byref(g), logits, ids, dgates, dsums, dtype, dl, None)


def size(lib, g):
    n = ctypes.c_size_t(0)
    return lib.moe_route_scored_workspace_size(ctypes.byref(g), ctypes.byref(n)), n.value


def test_header_matches_binding():
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    for name in ("MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID"):
        assert int(re.search(name + r"\s*=\s*(\d+)", text).group(1)) == getattr(L, name)
    body = re.search(r"typedef struct \{([^}]*)\} moe_gating_t;", text).group(1)
    fields = re.findall(r"^\s*(int64_t|int32_t|float) (\w+);", body, re.M)
    types = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float}
    assert [(n, types[t]) for t, n in fields] == list(L.MoeGating._fields_)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=65), INV), (dict(score=2), INV), (dict(score=-1), INV),
    (dict(groups=0), INV), (dict(groups=7), INV), (dict(groups=-8), INV), (dict(groups_kept=0), INV),
    (dict(groups_kept=9), INV), (dict(group_top=0), INV), (dict(group_top=3), INV),
    (dict(k=17, groups_kept=2), INV),                    # only 16 experts stay
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(E=264), UNS), (dict(k=33, groups_kept=8), UNS), (dict(T=2 ** 24), UNS), (dict(T=2 ** 27, k=32), UNS),
])
def test_gating_validation(lib, bad, status):
    g = gat(**bad)
    assert size(lib, g)[0] == status
    assert route(lib, g) == status and back(lib, g) == status


def test_gating_of_the_router(lib):
    for bad, status in ((dict(d=0), INV), (dict(dtype=2), INV), (dict(d=100), UNS)):
        g = gat(**bad)
        assert route(lib, g, x=A, w=A, li=None, lo=A) == status
        assert size(lib, g)[0] == OK                     # (not looked at with logits)
    assert route(lib, gat(d=100, dtype=F32), x=A, w=A, li=None, lo=A, ids=None) == INV


def test_gating_pointers(lib):
    g = gat()
    for name in ("li", "ids", "gates"):
        assert route(lib, g, **{name: MIS}) == UNS
        assert route(lib, g, **{name: None}) == INV
    for name in ("bias", "sums", "ws"):
        assert route(lib, g, **{name: MIS}) == UNS
    assert route(lib, g, ws=None) == INV
    for name in ("x", "w", "lo"):
        args = dict(x=A, w=A, li=None, lo=A)
        assert route(lib, g, **{**args, name: None}) == INV
        assert route(lib, g, **{**args, name: MIS}) == UNS
    need = size(lib, g)[1]
    assert need > 0 and route(lib, g, n=need - 1) == WS
    for name in ("logits", "ids", "dgates", "dl"):
        assert back(lib, g, **{name: MIS}) == UNS
        assert back(lib, g, **{name: None}) == INV
    assert back(lib, g, dsums=MIS) == UNS
    assert back(lib, g, dtype=2) == INV
    assert lib.moe_route_scored(None, *[None] * 9, 0, None) == INV
    assert lib.moe_route_scored_backward(None, *[None] * 4, 0, None, None) == INV
    assert lib.moe_route_scored_workspace_size(ctypes.byref(g), None) == INV


def test_no_tokens_is_a_no_op(lib):
    g = gat(T=0)
    assert size(lib, g) == (OK, 0)
    assert route(lib, g, li=None, x=None, bias=None, ids=None, gates=None, sums=None, ws=None, n=0) == OK
    assert back(lib, g, None, None, None, None, F32, None) == OK


def prob(T=64, d=128, k=2, dtype=BF16):
    return L.MoeProblem(T=T, d=d, E=k, k=k, f=64, dtype=dtype)


def test_combine_backward_arguments(lib):
    call = lib.moe_combine_backward
    p = ctypes.byref(prob())
    ok = [A] * 6   # dy, y_perm, assign_pos, gates, dy_perm, dgates
    for i in range(6):
        args = ok[:i] + [MIS] + ok[i + 1:]
        assert call(p, *args, None) == UNS, i
    for i in (0, 1, 2, 3):
        args = ok[:i] + [None] + ok[i + 1:]
        assert call(p, *args, None) == INV, i
    assert call(p, A, A, A, A, None, None, None) == INV
    assert call(p, None, None, A, A, A, None, None) == INV
    assert call(ctypes.byref(prob(d=100)), *ok, None) == UNS
    assert call(ctypes.byref(prob(k=0)), *ok, None) == INV
    assert call(None, *ok, None) == INV
    assert call(ctypes.byref(prob(T=0)), *[None] * 6, None) == OK


def test_mxfp4_row_arguments(lib):
    for call in (lambda r, c, t, *p: lib.moe_quantize_rows_mxfp4(p[0], r, c, t, p[1], p[2], None),
                 lambda r, c, t, *p: lib.moe_dequantize_rows_mxfp4(p[1], p[2], r, c, t, p[0], None)):
        assert call(-1, 64, F32, A, A, A) == INV
        assert call(1, 0, F32, A, A, A) == INV
        assert call(1, -32, F32, A, A, A) == INV
        assert call(1, 64, 2, A, A, A) == INV
        assert call(1, 48, F32, A, A, A) == UNS
        assert call(1, (1 << 20) + 32, F32, A, A, A) == UNS
        assert call(2 ** 24, 32, F32, A, A, A) == UNS
        assert call(2 ** 24 - 1, 4096, F32, A, A, A) == UNS     # rows * cols above 2^35 - 2^11
        for i in range(3):
            for bad, st in ((None, INV), (MIS, UNS)):
                args = [A] * 3
                args[i] = bad
                assert call(4, 64, BF16, *args) == st, (i, bad)
        assert call(0, 64, BF16, None, None, None) == OK


def grp(rows=64, E=8, N=256, K=128, dtype=BF16):
    return L.MoeGrouped(rows=rows, E=E, N=N, K=K, dtype=dtype)


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), INV), (dict(E=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(dtype=2), INV),
    (dict(E=257), UNS), (dict(rows=2 ** 31), UNS), (dict(N=(1 << 20) + 8), UNS), (dict(K=(1 << 20) + 32), UNS),
    (dict(N=100), UNS), (dict(K=48), UNS), (dict(rows=2 ** 31 - 1, N=1 << 20, K=1 << 20), UNS),
])
def test_product_problem(lib, bad, status):
    assert lib.moe_grouped_matmul_mxfp4(ctypes.byref(grp(**bad)), *[A] * 6, None) == status


def test_product_pointers(lib):
    g = ctypes.byref(grp())
    for i in range(6):      # a, a_scales, w, w_scales, offsets, c
        for bad, st in ((None, INV), (MIS, UNS)):
            args = [A] * 6
            args[i] = bad
            assert lib.moe_grouped_matmul_mxfp4(g, *args, None) == st, (i, bad)
    assert lib.moe_grouped_matmul_mxfp4(None, *[A] * 6, None) == INV
    assert lib.moe_grouped_matmul_mxfp4(ctypes.byref(grp(rows=0)), None, None, None, None, A, None, None) == OK


# ---- the binding, on tensors without storage -----------------------------------------

META = "meta"
U8, I32 = torch.uint8, torch.int32


def t(*shape, dtype=torch.float32, device=META):
    return torch.empty(*shape, dtype=dtype, device=device)


def refuses(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_route_scored_arguments():
    T, E, k, d = 48, 16, 4, 128
    refuses("live on the GPU", moe.route_scored, k, logits=t(T, E))
    refuses("live on the GPU", moe.route_scored, k, x=t(T, d), w_router=t(E, d), bias=t(E))
    refuses("score", moe.route_scored, k, logits=t(T, E), score="relu")
    refuses("logits", moe.route_scored, k, logits=t(T, E, dtype=torch.bfloat16))
    refuses("logits", moe.route_scored, k, logits=t(T, E, 1))
    refuses("logits", moe.route_scored, k, logits=t(E, T).t())
    refuses("required", moe.route_scored, k, x=t(T, d))
    refuses("w_router", moe.route_scored, k, x=t(T, d), w_router=t(E, d + 1))
    refuses("bias", moe.route_scored, k, logits=t(T, E), bias=t(E + 1))
    refuses("bias", moe.route_scored, k, logits=t(T, E), bias=t(E, dtype=torch.float64))
    refuses("bias", moe.route_scored, k, logits=t(T, E), bias=t(E, device="cpu"))
    refuses("ids", moe.route_scored, k, logits=t(T, E), ids=t(T, k, dtype=torch.int64))
    refuses("gates", moe.route_scored, k, logits=t(T, E), gates=t(T, k + 1))
    refuses("score_sums", moe.route_scored, k, logits=t(T, E), with_score_sums=True, score_sums=t(T))
    refuses("ws", moe.route_scored, k, logits=t(T, E), with_score_sums=True, ws=t(64, device="cpu"))
    refuses("topk_ids", moe.route_scored_backward, t(T, E), t(T, k), t(T, k))
    refuses("dgates", moe.route_scored_backward, t(T, E), t(T, k, dtype=I32), t(T, k + 1))
    refuses("dscore_sums", moe.route_scored_backward, t(T, E), t(T, k, dtype=I32), t(T, k), dscore_sums=t(k))
    refuses("dlogits", moe.route_scored_backward, t(T, E), t(T, k, dtype=I32), t(T, k), dtype=torch.bfloat16, dlogits=t(T, E))
    refuses("dtype", moe.route_scored_backward, t(T, E), t(T, k, dtype=I32), t(T, k), dtype=torch.float16)
    refuses("live on the GPU", moe.route_scored_backward, t(T, E), t(T, k, dtype=I32), t(T, k))


def test_combine_backward_tensors():
    T, k, d = 48, 4, 128
    dy, y, pos, g = t(T, d), t(T * k, d), t(T * k, dtype=I32), t(T, k)
    refuses("live on the GPU", moe.combine_backward, dy, pos, g, y_perm=y)
    refuses("y_perm is required", moe.combine_backward, dy, pos, g)
    refuses("is required", moe.combine_backward, dy, pos, g, y_perm=y, with_dy_perm=False, with_dgates=False)
    refuses("y_perm", moe.combine_backward, dy, pos, g, y_perm=t(T * k, d, dtype=torch.bfloat16))
    refuses("assign_pos", moe.combine_backward, dy, t(T * k, dtype=torch.int64), g, y_perm=y)
    refuses("gates", moe.combine_backward, dy, pos, t(T, k, dtype=torch.float64), y_perm=y)
    refuses("dy", moe.combine_backward, t(T, d, dtype=torch.float16), pos, g, y_perm=y)
    refuses("dy_perm", moe.combine_backward, dy, pos, g, y_perm=y, out=dict(dy_perm=t(T, d)))
    refuses("dgates", moe.combine_backward, dy, pos, g, y_perm=y, out=dict(dgates=t(T * k)))


def test_mxfp4_tensors():
    R, K, E, N = 40, 544, 4, 24
    c, s = t(R, K // 2, dtype=U8), t(3, R, 8, dtype=U8)
    w, ws, off = t(E, N, K // 2, dtype=U8), t(3, E, N, 8, dtype=U8), t(E + 1, dtype=I32)
    refuses("live on the GPU", moe.quantize_rows_mxfp4, t(R, K))
    refuses("src", moe.quantize_rows_mxfp4, t(R, K, dtype=torch.float16))
    refuses("src", moe.quantize_rows_mxfp4, t(K, R).t())
    refuses("codes", moe.quantize_rows_mxfp4, t(R, K), codes=t(R, K, dtype=U8))
    refuses("scales", moe.quantize_rows_mxfp4, t(R, K), scales=t(R, K // 32, dtype=U8))
    refuses("live on the GPU", moe.dequantize_rows_mxfp4, c, s)
    refuses("scales", moe.dequantize_rows_mxfp4, c, t(2, R, 8, dtype=U8))
    refuses("dtype", moe.dequantize_rows_mxfp4, c, s, dtype=torch.float16)
    refuses("out", moe.dequantize_rows_mxfp4, c, s, out=t(R, K))
    refuses("live on the GPU", moe.grouped_matmul_mxfp4, c, s, w, ws, off)
    refuses("a must be", moe.grouped_matmul_mxfp4, c, s, w[0], ws, off)
    refuses("a must be", moe.grouped_matmul_mxfp4, c, s, w, ws)
    refuses("a_scales", moe.grouped_matmul_mxfp4, c, s.transpose(0, 1), w, ws, off)
    refuses("w_scales", moe.grouped_matmul_mxfp4, c, s, w, ws[:, :, :, :4], off)
    refuses("w:", moe.grouped_matmul_mxfp4, c, s, t(E, N, K, dtype=U8), ws, off)
    refuses("offsets", moe.grouped_matmul_mxfp4, c, s, w, ws, t(E, dtype=I32))
    refuses("out_dtype", moe.grouped_matmul_mxfp4, c, s, w, ws, off, out_dtype=torch.float16)
    refuses("c:", moe.grouped_matmul_mxfp4, c, s, w, ws, off, c=t(R, N))
