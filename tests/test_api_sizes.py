"""Sizes past the 32 bits that the C ABI takes them in are refused by the binding, on
tensors without storage: cut to their low bits they would be others, which the library
would take."""
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe

U8, I8, I32, F32, BF16 = torch.uint8, torch.int8, torch.int32, torch.float32, torch.bfloat16
HUGE = 2 ** 32


def t(*shape, dtype=F32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def refuses(fn, *args, **kw):
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        fn(*args, **kw)


def test_rows_to_quantise():
    for n in (HUGE + 64, 2 ** 31):
        refuses(moe.quantize_rows_mxfp4, t(2, n, dtype=BF16))
        refuses(moe.quantize_rows_mxfp4, t(2, n))
        refuses(moe.dequantize_rows_mxfp4, t(2, n // 2, dtype=U8), t((n + 255) // 256, 2, 8, dtype=U8))
        refuses(moe.quantize_rows_int8, t(2, n))
        refuses(moe.quantize_rows_fp8, t(2, n, dtype=BF16))


def test_products():
    K, S = HUGE + 32, HUGE // 256 + 1
    refuses(moe.grouped_matmul_mxfp4, t(4, K // 2, dtype=U8), t(S, 4, 8, dtype=U8), t(2, 8, K // 2, dtype=U8),
            t(S, 2, 8, 8, dtype=U8), t(3, dtype=I32))
    refuses(moe.grouped_matmul_mxfp4, t(4, 32, dtype=U8), t(1, 4, 8, dtype=U8), t(HUGE + 8, 32, dtype=U8),
            t(1, HUGE + 8, 8, dtype=U8))
    refuses(moe.grouped_matmul_mxfp4, t(4, 32, dtype=U8), t(1, 4, 8, dtype=U8), t(HUGE + 2, 8, 32, dtype=U8),
            t(1, HUGE + 2, 8, 8, dtype=U8), t(HUGE + 3, dtype=I32))
    refuses(moe.grouped_matmul_int8, t(4, K, dtype=I8), t(4), t(8, K, dtype=I8), t(8))
    refuses(moe.grouped_matmul, t(4, K), t(2, 8, K), t(3, dtype=I32))
    refuses(moe.grouped_matmul_backward, t(4, K), t(2, 8, K), t(3, dtype=I32), t(4, 8))
    refuses(moe.grouped_workspace_size, 2, 4, HUGE + 2, 8, 64, BF16)


def test_routing():
    E = HUGE + 8
    refuses(moe.route_scored, 2, logits=t(1, E))
    refuses(moe.route_scored, HUGE + 2, logits=t(1, 8))
    refuses(moe.route_scored, 2, x=t(1, HUGE + 64), w_router=t(8, HUGE + 64))
    for cfg in (dict(groups=HUGE + 1), dict(groups_kept=HUGE + 1), dict(group_top=HUGE + 1), dict(groups=-HUGE + 1)):
        refuses(moe.route_scored, 2, logits=t(1, 8), **cfg)
    refuses(moe.route_scored_backward, t(1, E), t(1, 2, dtype=I32), t(1, 2))
    refuses(moe.route_scored_workspace_size, 4, E, 2)
    refuses(moe.route, 2, logits=t(1, E))
    refuses(moe.dispatch, t(1, 2, dtype=I32), E)


def test_combine():
    d = HUGE + 64
    refuses(moe.combine_backward, t(1, d), t(2, dtype=I32), t(1, 2), y_perm=t(2, d))
    refuses(moe.combine, t(2, d), t(2, dtype=I32), t(1, 2))
