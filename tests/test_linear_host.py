"""CPU tests of the 4-bit linear map's host side (no HIP call is made)."""
import os
import subprocess
import sys

import pytest

import quantized_mixture_experts_fp32_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# sizes that moe_linear_w4 refuses: N below or between row tiles, K off the
# groups, each limit
REFUSED = [(100, 8, 1280), (100, 8, 4096), (1, 15, 4096), (1, 15, 2176), (5000, 24, 4096),
           (64, 1, 1024), (100, 4096, 4100), (100, 4096, 1), (1, 16, 1 << 20),
           (1 << 23, 16, 128), (1, 1 << 28, 128), (1 << 17, 16, 1 << 17), (1 << 17, 1 << 17, 128),
           ((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1), (-1, 16, 128), (4, 0, 128), (4, 16, -128)]


@pytest.mark.parametrize("T,N,K", REFUSED)
def test_workspace_query_of_refused_sizes(T, N, K):
    """0 bytes, in a process of its own: a query that divides by the count of
    row tiles would end it."""
    code = ("import quantized_mixture_experts_fp32_amd as moe;"
            f"print(moe.moe_linear_w4_ws_bytes({T}, {N}, {K}))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=60,
                       cwd=ROOT)
    assert r.returncode == 0 and r.stdout.split() == ["0"], (r.returncode, r.stdout, r.stderr)
    lib = moe.load_library()
    assert lib.moe_linear_w4(0x10000, T, N, K, 128, 0x10000, 0x10000, None, 0x10000, 0, None, 0,
                             None) in (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED)


def test_workspace_query_of_accepted_sizes():
    """Some accepted size needs a workspace, of the split group sums' size."""
    for T, N, K in ((2501, 4096, 4096), (1500, 8208, 256), (4096, 2048, 2048)):
        assert moe.moe_linear_w4_ws_bytes(T, N, K) == T * (K // 128) * 8
    assert moe.moe_linear_w4_ws_bytes(1, 16, 128) == 0
