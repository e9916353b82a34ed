"""How many loads the 4-bit product's kernels leave in flight at their waits, from the
generated code: loads into LDS come back in the order they were sent, so a wait for all
but N has the older ones in LDS, and N may be at most the loads sent after the slice that
is read next.  Compiled for the device here, never run.

Split kernels (a ring of two slices for each wave, no barriers): two slices of L loads are
sent, then each wait has one younger slice behind it.  Tile kernels: the first slice of NL
loads and a part of the second go out first; within a slice's turn a barrier after the last
reads frees its stage, the refilling loads begin, and before the next slice is read a wait
leaves those, and a barrier follows."""
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
    out = tmp_path_factory.mktemp("counts") / "mxfp4.s"
    r = subprocess.run([cc, *B.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "grouped_mxfp4.hip"),
                        "-o", str(out)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return out.read_text()


EVENTS = re.compile(r"^\s+(?:(buffer_load_dword(?:x4)? [^\n]* lds)|s_waitcnt vmcnt\((\d+)\)( lgkmcnt\(0\))?|(s_barrier)|(ds_read)|(ds_write)"
                    r"|s_waitcnt (lgkmcnt\(0\))|((?:buffer|global)_store))", re.M)


def events(body):
    """load, (wait, N), barrier, read, write, drain (of LDS accesses), store; from the
    first load into LDS on."""
    out = []
    for load, n, both, barrier, read, write, drain, store in EVENTS.findall(body):
        if load:
            out.append("load")
        elif n:
            out.append(("wait", int(n)))
            if both:
                out.append("drain")
        elif barrier or read or write or drain or store:
            out.append("barrier" if barrier else "read" if read else "write" if write else "drain" if drain else "store")
    return out[out.index("load"):]


def check_split(body, copies):
    records, since = [], 0
    for e in events(body):
        if e == "load":
            since += 1
        elif e[0] == "wait":
            records.append((since, e[1]))
            since = 0
        elif e == "read":
            # (nothing is read between a slice's loads and the wait for them)
            assert since == 0 or records[-1][1] == 0
    assert since == 0
    while records and records[-1] == (0, 0):
        records.pop()
    assert len(records) == 4 * copies, records
    sizes = []
    for i in range(0, len(records), 4):
        (first, n0), (a, n1), (b, n2), (c, n3) = records[i:i + 4]
        L = first // 2
        assert (first, a, b, c) == (2 * L, L, L, L) and n3 == 0, records[i:i + 4]
        assert max(n0, n1, n2) <= L, records[i:i + 4]
        sizes.append(L)
    return sizes


def check_tile(body):
    ev = events(body)
    first = next(i for i, e in enumerate(ev) if e[0] == "wait" and e[1] > 0)
    sent = ev[:first].count("load")
    # (waits with loads left over: the one before the first slice, the one of the loop)
    left = [i for i, e in enumerate(ev) if e[0] == "wait" and e[1] > 0]
    assert len(left) == 2, [ev[i] for i in left]
    assert all(ev[i + 1] == "barrier" for i in left)
    loop = ev[first + 1:]
    NL = loop.count("load")
    assert sent >= NL and ev[first][1] <= sent - NL, (sent, NL, ev[first])
    at = left[1] - first - 1
    free = max(i for i in range(1, at) if loop[i] == "barrier")
    assert loop[free - 1] == "drain"
    between = loop[free + 1:at]
    assert "read" not in between and "write" not in between, between
    assert loop[at][1] <= between.count("load"), (loop[at], between.count("load"))
    # all of a slice's loads are sent before the outputs are stored
    assert "load" not in loop[loop.index("store"):]
    return NL, loop[at][1]


def kernels(text, name):
    return {m.group(1): m.group(2) for m in re.finditer(r"^(\w*%s\w*):(.*?)\.end_amdhsa_kernel" % name, text, re.M | re.S)}


def test_split_kernels(text):
    found = kernels(text, "grouped_split_kernel")
    assert len(found) == 4
    # loads of a slice: codes of 32 columns (4) and of 8, 16 or 32 rows (1, 2, 4), two of
    # scales; or of 64 columns and rows (16) and 4
    seen = sorted(tuple(sorted(check_split(body, 3 if "Li1ELi1E" in name else 1))) for name, body in found.items())
    assert seen == [(7, 8, 10), (7, 8, 10), (20,), (20,)]


def test_tile_kernels(text):
    found = kernels(text, "grouped_tile_kernel")
    assert len(found) == 12
    for name, body in found.items():
        NL, left = check_tile(body)
        assert 0 < left < NL


def test_a_wait_for_too_few_would_be_found(text):
    for name, body in kernels(text, "grouped_split_kernel").items():
        copies = 3 if "Li1ELi1E" in name else 1
        n = {int(v) for v in re.findall(r"s_waitcnt vmcnt\((\d+)\)", body[body.index(" lds"):])} - {0}
        for v in n:
            at = body.index(" lds")
            bad = body[:at] + re.sub(r"vmcnt\(%d\)" % v, "vmcnt(%d)" % (v + 1), body[at:])
            with pytest.raises(AssertionError):
                check_split(bad, copies)
    for body in kernels(text, "grouped_tile_kernel").values():
        at = body.index(" lds")
        waits = [m for m in re.finditer(r"s_waitcnt vmcnt\((\d+)\)", body[at:]) if m.group(1) != "0"]
        for m in waits:
            bad = body[:at + m.start()] + "s_waitcnt vmcnt(%d)" % (int(m.group(1)) + 1) + body[at + m.end():]
            with pytest.raises(AssertionError):
                check_tile(bad)
