"""The waits for direct global-to-LDS loads, as the compiler sees them: the
loads are inline assembly, so nothing but the wait itself tells the compiler
that LDS has changed.  A wait has to keep LDS accesses on their side of it.
Compiled for the device here, never run."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_exclusive_amd import build as B

# Each kernel accesses an LDS word, waits, and accesses the same word again:
# merged with the first access unless the wait stands between them.
PROBE = """
#include "lds_dma.h"
using namespace moe;
extern "C" __global__ void read_after_vmcnt(const char* in, int* out) {
    __shared__ __attribute__((aligned(1024))) char smem[1024];
    lds_dma16(in + threadIdx.x * 16, __builtin_amdgcn_readfirstlane(lds_addr(smem)));
    const int a = reinterpret_cast<int*>(smem)[threadIdx.x];
    wait_vmcnt<0>();
    out[threadIdx.x] = a - reinterpret_cast<int*>(smem)[threadIdx.x];
}
extern "C" __global__ void read_after_vmcnt_lgkm(const char* in, int* out) {
    __shared__ __attribute__((aligned(1024))) char smem[1024];
    lds_dma16(in + threadIdx.x * 16, __builtin_amdgcn_readfirstlane(lds_addr(smem)));
    const int a = reinterpret_cast<int*>(smem)[threadIdx.x];
    wait_vmcnt_lgkm0<63>();
    out[threadIdx.x] = a - reinterpret_cast<int*>(smem)[threadIdx.x];
}
extern "C" __global__ void write_after_vmcnt(const char* in, int* out) {
    __shared__ __attribute__((aligned(1024))) char smem[1024];
    lds_dma16(in + threadIdx.x * 16, __builtin_amdgcn_readfirstlane(lds_addr(smem)));
    reinterpret_cast<int*>(smem)[threadIdx.x] = 1;
    wait_vmcnt<3>();
    reinterpret_cast<int*>(smem)[threadIdx.x] = 2;
    wait_vmcnt<0>();
    out[threadIdx.x] = reinterpret_cast<int*>(smem)[threadIdx.x ^ 1];
}
"""


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("waits")
    (d / "probe.hip").write_text(PROBE)
    r = subprocess.run([cc, *B.HIPCC_FLAGS, "--cuda-device-only", "-S", str(d / "probe.hip"), "-o", str(d / "probe.s")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    text = (d / "probe.s").read_text()
    return {m.group(1): m.group(2) for m in re.finditer(r"^(\w+):(.*?)s_endpgm", text, re.M | re.S)}


@pytest.mark.parametrize("name,access,wait", [
    ("read_after_vmcnt", r"\bds_read", r"s_waitcnt vmcnt\(0\)"),
    ("read_after_vmcnt_lgkm", r"\bds_read", r"s_waitcnt lgkmcnt\(0\)"),
    ("write_after_vmcnt", r"\bds_write", r"s_waitcnt vmcnt\(3\)"),
])
def test_lds_accesses_stay_on_their_side_of_a_wait(kernels, name, access, wait):
    body = kernels[name]
    at = [m.start() for m in re.finditer(access, body)]
    assert len(at) == 2, body
    assert re.search(wait, body[at[0]:at[1]]), body


def test_split_kernels_wait_between_their_loads_and_lds_accesses(tmp_path):
    """The split kernel's waves load, read and reuse their own part of LDS with
    no barrier in between: in its code every LDS access after a load into LDS
    has a wait for loads before it."""
    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path / "grouped.s"
    r = subprocess.run([cc, *B.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "grouped.hip"), "-o", str(out)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    text = out.read_text()
    found = 0
    for m in re.finditer(r"^(\w*grouped_split_kernel\w*):(.*?)\.end_amdhsa_kernel", text, re.M | re.S):
        found += 1
        loads = reads = writes = 0
        pending = False
        for e in re.findall(r"buffer_load_dwordx4 [^\n]* lds|s_waitcnt vmcnt\(\d+\)|ds_read|ds_write", m.group(2)):
            if e.startswith("buffer"):
                pending = True
                loads += 1
            elif e.startswith("s_waitcnt"):
                pending = False
            else:
                assert not pending, (m.group(1), e)
                reads += e == "ds_read"
                writes += e == "ds_write"
        assert loads and reads and writes
    assert found >= 10, found
