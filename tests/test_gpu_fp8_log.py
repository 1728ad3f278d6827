"""QGEMM_LOG names the kernel that an fp8 product runs, both tiles where it has two."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_first_dispatch_line_names_both_tiles():
    code = (
        "import torch, int4_weight_only_uint32_amd as qg\n"
        "def run(M, N, K=128):\n"
        "    f8 = torch.float8_e4m3fn\n"
        "    a, w = torch.ones(M, K, device='cuda').to(f8), torch.ones(N, K, device='cuda').to(f8)\n"
        "    qg.fp8_gemm(a, torch.ones(M, 1, device='cuda'), w, torch.ones(-(-N // 128), 1, device='cuda'))\n"
        "for M, N in ((1024, 17408), (1024, 19500), (1024, 21900), (1024, 26000), (1024, 32768), (4, 256)):\n"
        "    run(M, N)\n"
        "torch.cuda.synchronize()\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, QGEMM_LOG="1", PYTHONPATH=root)
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    said = {}
    for line in r.stderr.splitlines():
        if line.startswith("[qgemm] first dispatch ok: qgemm_fp8"):
            head, kernel = line.split(": ", 2)[1:]
            said[int(head.split("N=")[1].split()[0])] = kernel
    assert said == {
        17408: "tiled, 256 x 256, from column 16384 on 64 x 128, 2 groups over k",
        19500: "tiled, 256 x 256, from column 16384 on 128 x 128, 2 groups over k",
        21900: "tiled, 256 x 256, from column 16384 on 128 x 256",
        26000: "tiled, 256 x 256",
        32768: "tiled, 256 x 256",
        256: "streaming, 16 x 16, 4 waves over k"}, said
