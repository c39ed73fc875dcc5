"""CPU tests of the 4-bit linear map's host side (no HIP call is made)."""
import os
import subprocess
import sys

import pytest

import quantized_mixture_experts_fp32_amd as moe
from linear_shapes import LISTED, SHAPES

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


@pytest.mark.parametrize("name,T,K,N", LISTED)
def test_shapes_run_the_kernel_that_they_are_listed_for(name, T, K, N):
    """What the GPU tests of a kernel's shapes reach: a change of the kernel
    choice has to come with shapes for what it moved."""
    assert moe.moe_linear_w4_kernel(T, N, K) == name


def test_kernels_in_use():
    """Only listed kernels run, over the range of sizes; refused and empty
    sizes run none; the GEMM alone has a workspace."""
    seen = set()
    for T in (1, 2, 5, 16, 17, 33, 48, 64, 65, 97, 200, 333, 515, 1024, 1500, 2501, 4096):
        for K in (128, 256, 640, 1024, 1664, 2048, 2176, 4096, 5248, 8192, 14336):
            for N in (16, 272, 784, 2064, 4112, 8208, 12304, 25712, 50304):
                name = moe.moe_linear_w4_kernel(T, N, K)
                seen.add(name)
                assert (moe.moe_linear_w4_ws_bytes(T, N, K) > 0) == name.startswith("gemm")
    assert seen <= set(SHAPES) and len(seen) >= 14, seen ^ set(SHAPES)
    for T, N, K in (*REFUSED, (0, 16, 128)):
        assert moe.moe_linear_w4_kernel(T, N, K) == ""
