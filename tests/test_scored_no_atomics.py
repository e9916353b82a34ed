"""The scored routing's kernels use no atomic operation, in memory or in LDS, so that the
same inputs give the same bits.  Compiled for the device here, never run."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_exclusive_amd import build as B


@pytest.mark.parametrize("source", ["route_scored.hip", "combine.hip", "quant_mxfp4.hip"])
def test_no_atomics(tmp_path, source):
    try:
        cc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = tmp_path / "kernels.s"
    r = subprocess.run([cc, *B.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, source), "-o", str(out)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    text = out.read_text()
    assert "s_endpgm" in text
    assert not re.findall(r"^\s+(?:(?:global|buffer|flat)_atomic_\w+|ds_(?:add|sub|inc|dec|min|max|and|or|xor|cmpst|wrxchg)_\w+)",
                          text, re.M)
