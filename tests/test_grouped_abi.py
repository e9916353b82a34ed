"""The grouped products' entry points on the CPU: argument checks of the C
ABI and of the binding, before any HIP call (no kernel is launched)."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from mixture_experts_layer_exclusive_amd import _lib as L
from mixture_experts_layer_exclusive_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000    # never dereferenced
MIS = 0x10004  # not 16-byte aligned
BIG = 1 << 40
INV, UNS, WS = L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE_TOO_SMALL


def grp(rows=64, E=8, N=256, K=128, dtype=L.MOE_DTYPE_BF16):
    return L.MoeGrouped(rows=rows, E=E, N=N, K=K, dtype=dtype)


@pytest.fixture(scope="module")
def lib():
    return L.load()


def size(lib, g, op):
    n = ctypes.c_size_t(0)
    return lib.moe_grouped_workspace_size(ctypes.byref(g), op, ctypes.byref(n)), n.value


def all_calls(lib, g):
    p = ctypes.byref(g)
    return [lib.moe_grouped_matmul(p, A, A, A, A, A, BIG, None),
            lib.moe_grouped_matmul_backward(p, A, A, A, A, A, A, A, BIG, None),
            lib.moe_grouped_matmul_int8(p, A, A, A, A, A, A, A, BIG, None)]


def test_header_constants_match_binding():
    text = open(os.path.join(ROOT, "include", "moe.h")).read()
    for name in ("MOE_GROUPED_OP_MATMUL", "MOE_GROUPED_OP_BACKWARD", "MOE_GROUPED_OP_INT8"):
        assert int(re.search(name + r"\s*=\s*(\d+)", text).group(1)) == getattr(L, name)
    assert 1 << int(re.search(r"#define MOE_GROUPED_MAX_DIM \(1 << (\d+)\)", text).group(1)) == L.MOE_GROUPED_MAX_DIM


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), INV), (dict(E=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(N=-8), INV),
    (dict(dtype=2), INV), (dict(dtype=-1), INV),
    (dict(E=257), UNS), (dict(rows=2 ** 31), UNS),
    (dict(N=(1 << 20) + 8), UNS), (dict(K=(1 << 20) + 16), UNS),
    (dict(N=100), UNS), (dict(K=100), UNS),
    (dict(rows=2 ** 31 - 1, N=1 << 20, K=1 << 20), UNS),
])
def test_problem_validation(lib, bad, status):
    g = grp(**bad)
    for op in (1, 2, 3):
        assert size(lib, g, op)[0] == status
    assert all_calls(lib, g) == [status] * 3


def test_row_lengths_by_type(lib):
    assert size(lib, grp(N=12, K=4, dtype=L.MOE_DTYPE_F32), 1)[0] == L.MOE_OK
    assert size(lib, grp(N=10, K=4, dtype=L.MOE_DTYPE_F32), 1)[0] == UNS
    assert size(lib, grp(N=8, K=24), 2)[0] == L.MOE_OK
    assert size(lib, grp(N=8, K=24), 3)[0] == UNS   # int8: K a multiple of 16
    assert size(lib, grp(N=8, K=48), 3)[0] == L.MOE_OK
    assert size(lib, grp(N=8, K=(1 << 17) - 16), 3)[0] == L.MOE_OK
    assert size(lib, grp(N=8, K=1 << 17), 3)[0] == UNS
    assert size(lib, grp(N=8, K=1 << 17), 1)[0] == L.MOE_OK


def test_large_sizes_are_accepted(lib):
    # 2^32 elements of output, of weights, and rows up to the int32 limit
    assert size(lib, grp(rows=1 << 22, E=1, N=1024, K=64), 1)[0] == L.MOE_OK
    assert size(lib, grp(rows=64, E=256, N=4096, K=4096), 2)[0] == L.MOE_OK
    assert size(lib, grp(rows=2 ** 31 - 1, E=1, N=8, K=8), 1)[0] != INV


def test_workspace_query(lib):
    g = grp()
    assert lib.moe_grouped_workspace_size(ctypes.byref(g), 1, None) == INV
    assert lib.moe_grouped_workspace_size(None, 1, ctypes.byref(ctypes.c_size_t())) == INV
    assert size(lib, g, 0)[0] == INV and size(lib, g, 4)[0] == INV
    assert moe.grouped_workspace_size(1, 64, 8, 256, 128, torch.bfloat16) == size(lib, g, 1)[1]
    with pytest.raises(ValueError):
        moe.grouped_workspace_size(1, 64, 8, 256, 128, torch.float16)
    with pytest.raises(moe.MoeError):
        moe.grouped_workspace_size(1, 64, 8, 100, 128, torch.bfloat16)


def test_null_and_misaligned_pointers(lib):
    g = ctypes.byref(grp())
    ok = [A, A, A, A]
    for i in range(4):
        for bad, st in ((None, INV), (MIS, UNS)):
            args = ok[:i] + [bad] + ok[i + 1:]
            assert lib.moe_grouped_matmul(g, *args, A, BIG, None) == st, (i, bad)
    # backward: (a, w, offsets, dc, da, dw)
    back = lib.moe_grouped_matmul_backward
    for i in range(4):
        args = [A] * 6
        args[i] = None
        assert back(g, *args, A, BIG, None) == INV, i
    for i in range(6):
        args = [A] * 6
        args[i] = MIS
        assert back(g, *args, A, BIG, None) == UNS, i
    assert back(g, A, A, A, A, None, None, A, BIG, None) == INV
    # int8: (a, a_scales, w, w_scales, offsets, c)
    for i in range(6):
        for bad, st in ((None, INV), (MIS, UNS)):
            args = [A] * 6
            args[i] = bad
            assert lib.moe_grouped_matmul_int8(g, *args, A, BIG, None) == st, (i, bad)
    # quantise
    q = lib.moe_quantize_rows_int8
    assert q(A, -1, 64, 1, A, A, None) == INV
    assert q(A, 4, 0, 1, A, A, None) == INV
    assert q(A, 4, 64, 5, A, A, None) == INV
    assert q(A, 4, 72, 1, A, A, None) == UNS
    assert q(A, 4, (1 << 20) + 16, 1, A, A, None) == UNS
    assert q(A, 1 << 24, 64, 1, A, A, None) == UNS
    for i in range(3):
        for bad, st in ((None, INV), (MIS, UNS)):
            p = [A, A, A]
            p[i] = bad
            assert q(p[0], 4, 64, 1, p[1], p[2], None) == st
    assert q(None, 0, 64, 1, None, None, None) == L.MOE_OK


def test_no_rows_is_a_no_op(lib):
    g = ctypes.byref(grp(rows=0))
    assert lib.moe_grouped_matmul(g, None, None, None, None, None, 0, None) == L.MOE_OK
    assert lib.moe_grouped_matmul_int8(g, None, None, None, None, A, None, None, 0, None) == L.MOE_OK


def test_workspace_too_small(lib):
    # (a dense weight gradient over many rows splits them)
    for kw, op in ((dict(rows=16, E=1, N=256, K=8192), 1), (dict(rows=100000, E=1, N=256, K=256), 2),
                   (dict(rows=16, E=1, N=256, K=8192), 3)):
        g = grp(**kw)
        st, n = size(lib, g, op)
        assert st == L.MOE_OK
        if n == 0:
            continue
        p = ctypes.byref(g)
        fn, count = {1: (lib.moe_grouped_matmul, 4), 2: (lib.moe_grouped_matmul_backward, 6),
                     3: (lib.moe_grouped_matmul_int8, 6)}[op]
        assert fn(p, *[A] * count, A, n - 1, None) == WS
        assert fn(p, *[A] * count, None, n, None) == INV


# ---- the binding -------------------------------------------------------------

BF, F32, I32, I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
R, E, N, K = 48, 8, 64, 128


def t(*shape, dtype=BF, device="meta"):
    return torch.empty(*shape, dtype=dtype, device=device)


def raises(fn, match):
    with pytest.raises(ValueError, match=match):
        fn()


def call_matmul(**o):
    a = dict(a=t(R, K), w=t(E, N, K), offsets=t(E + 1, dtype=I32), **{})
    a.update(o)
    return moe.grouped_matmul(a["a"], a["w"], a["offsets"], ws=a.get("ws"), c=a.get("c"))


def call_backward(**o):
    a = dict(a=t(R, K), w=t(E, N, K), offsets=t(E + 1, dtype=I32), dc=t(R, N), kw={})
    a.update(o)
    return moe.grouped_matmul_backward(a["a"], a["w"], a["offsets"], a["dc"], out=a.get("out"), **a["kw"])


def call_int8(**o):
    a = dict(a=t(R, K, dtype=I8), sa=t(R, dtype=F32), w=t(E, N, K, dtype=I8), sw=t(E, N, dtype=F32),
             offsets=t(E + 1, dtype=I32), dt=BF)
    a.update(o)
    return moe.grouped_matmul_int8(a["a"], a["sa"], a["w"], a["sw"], a["offsets"], out_dtype=a["dt"], c=a.get("c"))


@pytest.mark.parametrize("call", [call_matmul, call_backward, call_int8])
def test_consistent_arguments_reach_the_device_check(call):
    raises(call, "live on the GPU")


@pytest.mark.parametrize("over,name", [
    (dict(a=t(R, K + 8)), "w"), (dict(a=t(R, K, dtype=F32)), "w"), (dict(a=t(R, K, dtype=torch.float16)), "a"),
    (dict(a=t(K)), "a must be"), (dict(w=t(N, K)), "a must be"), (dict(offsets=t(E, dtype=I32)), "offsets"),
    (dict(offsets=t(E + 1, dtype=torch.int64)), "offsets"), (dict(offsets=t(E + 1, dtype=I32, device="cpu")), "offsets"),
    (dict(c=t(R, N + 8)), "c"), (dict(c=t(R, N, dtype=F32)), "c"), (dict(a=t(K, R).t()), "a must be contiguous"),
    (dict(ws=t(64, dtype=torch.uint8, device="cpu")), "ws"),
])
def test_matmul_rejects(over, name):
    raises(lambda: call_matmul(**over), name)


@pytest.mark.parametrize("over,name", [
    (dict(dc=t(R, N + 8)), "w"), (dict(dc=t(R + 1, N)), "a"), (dict(a=None), "a for dw"), (dict(w=None), "w is required"),
    (dict(kw=dict(with_da=False, with_dw=False)), "with_da or with_dw"),
    (dict(out=dict(da=t(R, N))), "da"), (dict(out=dict(dw=t(E, K, N))), "dw"), (dict(dc=t(N)), "dc"),
])
def test_backward_rejects(over, name):
    raises(lambda: call_backward(**over), name)


def test_backward_one_gradient_needs_one_input():
    raises(lambda: call_backward(a=None, kw=dict(with_dw=False)), "live on the GPU")
    raises(lambda: call_backward(w=None, kw=dict(with_da=False)), "live on the GPU")


@pytest.mark.parametrize("over,name", [
    (dict(a=t(R, K)), "a"), (dict(w=t(E, N, K)), "w"), (dict(sa=t(R, 1, dtype=F32)), "a_scales"),
    (dict(sw=t(N, dtype=F32)), "w_scales"), (dict(dt=torch.float16), "out_dtype"), (dict(offsets=None), "without offsets"),
    (dict(w=t(N, K, dtype=I8)), "w"), (dict(c=t(R, N, dtype=F32)), "c"), (dict(sa=t(R)), "a_scales"),
])
def test_int8_rejects(over, name):
    raises(lambda: call_int8(**over), name)


def test_int8_dense_arguments():
    raises(lambda: call_int8(offsets=None, w=t(N, K, dtype=I8), sw=t(N, dtype=F32)), "live on the GPU")


def test_quantize_rejects():
    raises(lambda: moe.quantize_rows_int8(t(4, 64)), "live on the GPU")
    raises(lambda: moe.quantize_rows_int8(t(4, 64, dtype=torch.float16)), "src")
    raises(lambda: moe.quantize_rows_int8(t(4, 4, 64)), "src must be")
    raises(lambda: moe.quantize_rows_int8(t(4, 64), codes=t(4, 64, dtype=torch.uint8)), "codes")
    raises(lambda: moe.quantize_rows_int8(t(4, 64), scales=t(5, dtype=F32)), "scales")


# ---- the host layer under sanitizers ------------------------------------------

@pytest.mark.skipif("MOE_LIBRARY" in os.environ, reason="already in the sanitized child")
def test_host_layer_is_clean_under_sanitizers(tmp_path):
    try:
        B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    if not B.asan_runtime():
        pytest.skip("clang AddressSanitizer runtime not found")
    env = dict(os.environ)
    env.update(MOE_LIBRARY=B.build_host_sanitized(str(tmp_path)), LD_PRELOAD=B.asan_runtime(),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "tests/test_grouped_abi.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "passed" in r.stdout
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-6000:]
