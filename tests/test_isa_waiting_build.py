"""What the race checks compare: the waiting build's tiled fp8 kernels and its routing
and sorting kernels really differ from the library's, on their gfx950 assembly (no
GPU needed)."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_weight_only_uint32_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
FULL_WAIT = "s_waitcnt vmcnt(0) expcnt(0) lgkmcnt(0)"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")


def kernels(source, debug):
    """{mangled name: assembly lines} of a source in the library's or the waiting build."""
    from int4_weight_only_uint32_amd import build
    d = tempfile.mkdtemp(prefix="qg_isa_")
    try:
        out = os.path.join(d, "k.s")
        flags = [f for f in build.FLAGS if f not in ("-shared", "-fPIC")] + [f"-DQG_DEBUG_SYNC={debug}"]
        subprocess.run([HIPCC] + flags + ["-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S", "-o", out,
                                          os.path.join(CSRC, source)], check=True, capture_output=True, timeout=600)
        with open(out) as f:
            text = f.read()
    finally:
        shutil.rmtree(d, ignore_errors=True)
    return {name: [l.strip() for l in body.split("\n")]
            for name, body in re.findall(r"^(_Z\S+):.*?\n(.*?)^\.Lfunc_end", text, re.S | re.M)}


def test_tiled_fp8_loads_land_one_by_one():
    """After each load to LDS the wave waits, before its next one and before the next MFMA;
    in the library's build nearly none of them is waited for there."""
    share = {}
    for debug in (0, 1):
        for name, body in kernels("qg_fp8.hip", debug).items():
            if not re.search(r"fp8_(tiled|two_tiles)_kernel", name):
                continue
            loads = waited = 0
            pending = False
            for line in body:
                if re.match(r"buffer_load_\S+.*\blds\b", line):
                    loads, pending = loads + 1, True
                elif line.startswith(FULL_WAIT):
                    waited, pending = waited + pending, False
                elif line.startswith("v_mfma"):
                    pending = False
            share.setdefault(name, []).append(waited / loads)
    assert len(share) == 2 * (7 + 3)
    for name, (here, waiting) in share.items():
        assert waiting == 1.0 and here < 0.25, (name, here, waiting)


def test_routing_and_sorting_wait_where_lanes_meet():
    """The routing kernel of each width: in the exact and the ordinary path; the placing
    of the sort: on both sides of the counts' step."""
    counts = {}
    for debug in (0, 1):
        for name, body in kernels("qg_moe.hip", debug).items():
            counts.setdefault(name, []).append(sum(l.startswith(FULL_WAIT) for l in body))
    for part, least, n in (("moe_route_kernel", 3, 5), ("moe_sort_one_kernel", 2, 2), ("moe_sort_place_kernel", 2, 1)):
        of = [c for name, c in counts.items() if part in name]
        assert len(of) == n, (part, counts)
        for here, waiting in of:
            assert waiting - here >= least, (part, here, waiting)
