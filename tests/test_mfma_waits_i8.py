"""CPU test of libmoe_wq_i8.so's GPU code: no instruction takes an MFMA's result
before it is there (as test_mfma_waits.py has it for libmoe_wq.so).

Its matrix instruction, 16 x 16 x 64 in 8-bit integers, takes 4 passes, as the
16 x 16 x 32 in bf16 does: 8 steps."""
import os
import subprocess

import pytest

import quantized_mixture_experts_fp32_amd as moe
import test_mfma_waits as waits

LIB = os.path.join(moe.HERE, "libmoe_wq_i8.so")


def test_library_waits_for_its_matrix_results(tmp_path, monkeypatch):
    objdump = os.path.join(waits.LLVM, "llvm-objdump")
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(LIB):
        from quantized_mixture_experts_fp32_amd import build
        build.build()
    monkeypatch.setitem(waits.STEPS, "16x16x64", 8)
    kernels = mfmas = 0
    for n, code in enumerate(waits.device_objects(LIB)):
        path = tmp_path / f"{n}.o"
        path.write_bytes(code)
        r = subprocess.run([objdump, "-d", "--mcpu=gfx950", str(path)], capture_output=True,
                           text=True, check=True)
        for name, body in waits.parse(r.stdout).items():
            count = sum(ins.startswith("v_mfma") for ins, _, _ in body)
            if count:
                kernels, mfmas = kernels + 1, mfmas + count
                found = waits.early_uses(body)
                assert not found, (name, [(hex(a), hex(b), c, d) for a, b, c, d in found[:5]])
    assert kernels >= 8 and mfmas >= 200, (kernels, mfmas)
