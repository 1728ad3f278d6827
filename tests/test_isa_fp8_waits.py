"""The counted waits of the streaming fp8 kernels, on their gfx950 assembly (no
GPU needed).

A wave of fp8_stream_kernel has a ring of P stages in LDS, L loads each, and
before it reads a stage it waits until at most (P - 1) L loads are in flight.  That
is right only if the compiled code issues the first P stages' loads before the
first such wait and exactly L between one wait and the next."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "int4_weight_only_uint32_amd", "csrc", "qg_fp8.hip")
HIPCC = "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")


@pytest.fixture(scope="module")
def asm():
    from int4_weight_only_uint32_amd import build
    d = tempfile.mkdtemp(prefix="qg_isa_")
    try:
        out = os.path.join(d, "fp8.s")
        flags = [f for f in build.FLAGS if f not in ("-shared", "-fPIC")]
        subprocess.run([HIPCC] + flags + ["-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S", "-o", out, SRC],
                       check=True, capture_output=True, timeout=600)
        with open(out) as f:
            return f.read()
    finally:
        shutil.rmtree(d, ignore_errors=True)


def test_streaming_kernels_counted_waits(asm):
    seen = 0
    for name, body in re.findall(r"^(_Z\S*fp8_stream_kernel\S*):.*?\n(.*?)^\.Lfunc_end", asm, re.S | re.M):
        mt, nt, nw, p = (int(x) for x in re.search(r"kernelILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
        stage = 2 * nt + 2 * mt + 2               # W and A tiles, two loads of scales
        loads, waits = 0, []
        for line in body.split("\n"):
            if re.search(r"\bbuffer_load_\S+.*\blds\b", line):
                loads += 1
            m = re.search(r"s_waitcnt vmcnt\((\d+)\)\s*$", line)
            if m and int(m.group(1)) == (p - 1) * stage:
                waits.append(loads)
                loads = 0
        # one wait per stage of the unrolled ring; in front of the first, P stages;
        # what follows the last is the last stage's refill
        assert waits == [p * stage] + [stage] * (p - 1), (name, waits)
        assert loads == stage, (name, loads)
        seen += 1
    assert seen == 2 * 7, seen


def test_tiled_kernels_do_not_spill(asm):
    """A spill in the scheduled loop goes through memory and its waits stall the loads
    in flight (2.8 times slower where it happened)."""
    kernels = re.findall(r"\.name:\s+(\S*fp8_(?:tiled|two_tiles)_kernel\S*).*?\.vgpr_spill_count:\s+(\d+)", asm, re.S)
    assert len(kernels) == 2 * (7 + 3)
    for name, spills in kernels:
        assert int(spills) == 0, name
