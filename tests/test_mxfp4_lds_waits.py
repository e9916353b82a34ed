"""The 4-bit product's split kernels, whose waves load, read and reuse their own part
of LDS with no barrier in between: in their code every LDS access after a load into LDS
(of operands or of scales) has a wait for loads before it.  Compiled for the device
here, never run."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_exclusive_amd import build as B


@pytest.fixture(scope="module")
def text(tmp_path_factory):
    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("waits") / "mxfp4.s"
    r = subprocess.run([cc, *B.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "grouped_mxfp4.hip"),
                        "-o", str(out)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return out.read_text()


def kernels(text, name):
    return {m.group(1): m.group(2) for m in re.finditer(r"^(\w*%s\w*):(.*?)\.end_amdhsa_kernel" % name, text, re.M | re.S)}


def test_split_kernels_wait_between_their_loads_and_lds_accesses(text):
    found = kernels(text, "grouped_split_kernel")
    assert len(found) == 4
    for name, body in found.items():
        wide = narrow = reads = writes = 0
        pending = False
        for e in re.findall(r"buffer_load_dword(?:x4)? [^\n]* lds|s_waitcnt vmcnt\(\d+\)|ds_read|ds_write", body):
            if e.startswith("buffer"):
                pending = True
                wide += "x4" in e
                narrow += "x4" not in e
            elif e.startswith("s_waitcnt"):
                pending = False
            else:
                assert not pending, (name, e)
                reads += e == "ds_read"
                writes += e == "ds_write"
        assert wide and narrow and reads and writes


def test_nothing_spills(text):
    assert "scratch_" not in text and "buffer_store_dword v" not in re.sub(r"buffer_store_dwordx4", "", text)
    assert set(re.findall(r"\.vgpr_spill_count: +(\d+)", text)) == {"0"}
    assert set(re.findall(r"\.private_segment_fixed_size: +(\d+)", text)) == {"0"}


def test_products_are_block_scaled(text):
    """Every matrix instruction is the scaled one on two 4-bit operands, and the byte of
    the scales that belongs to each of a slice's four steps is used."""
    for body in kernels(text, "grouped_(?:split|tile|mxfp4_short)_kernel").values():
        ops = re.findall(r"v_mfma_\w+[^\n]*", body)
        assert ops and all("v_mfma_scale_f32_32x32x64_f8f6f4" in o and "cbsz:4 blgp:4" in o for o in ops)
        if len(ops) < 16:
            continue    # (the kernel for short reductions has a slice of its own length)
        used = {re.sub(r".*?(op_sel:\[\d,\d,\d\] )?(op_sel_hi:\[\d,\d,\d\]).*", r"\1\2", o) for o in ops}
        assert len(used) == 4, used
