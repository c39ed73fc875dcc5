"""CPU test of the built library's GPU code: no instruction takes an MFMA's
result before it is there.

The hardware does not wait for a matrix instruction's result when a vector
instruction reads or overwrites it; the compiler counts the steps and inserts
s_nop, but has been seen to count along a branch's fall-through only, so that
a result read behind a branch came too early.  This walks every path from every
MFMA of the library and counts the steps up to the first use.

Steps needed: what the compiler puts between an MFMA and its use in straight
code, passes + 4: 12 for 32x32x16 (8 passes), 8 for 16x16x32 (4 passes).  A
chain of MFMAs on one accumulator is the hardware's own business.
"""
import os
import re
import struct
import subprocess

import pytest

import quantized_mixture_experts_fp32_amd as moe

LLVM = os.environ.get("ROCM_LLVM_BIN", "/opt/rocm/llvm/bin")
STEPS = {"16x16x32": 8, "32x32x16": 12}
INSN = re.compile(r"^\s+([a-z]\w+)\s*(.*?)\s*//\s*([0-9A-F]+):")
VREG = re.compile(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b")


def device_objects(path):
    """The gfx950 code objects in a library's offload bundles."""
    blob = open(path, "rb").read()
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := blob.find(magic, at)) >= 0:
        n, = struct.unpack_from("<Q", blob, at + 24)
        p = at + 32
        for _ in range(n if n < 16 else 0):
            off, size, idlen = struct.unpack_from("<QQQ", blob, p)
            name = blob[p + 24:p + 24 + idlen]
            p += 24 + idlen
            if b"gfx950" in name and size:
                yield blob[at + off:at + off + size]
        at += len(magic)


def parse(listing):
    """{function: [(mnemonic, operands, address)]} of an llvm-objdump listing."""
    out, body = {}, None
    for line in listing.splitlines():
        if line.endswith(">:"):
            body = out.setdefault(line.split("<")[1][:-2], [])
        elif body is not None and (m := INSN.match(line)):
            body.append((m[1], m[2], int(m[3], 16)))
    return out


def regs(text):
    r = set()
    for a, b, c in VREG.findall(text):
        r.update((int(c),) if c else range(int(a), int(b) + 1))
    return r


def early_uses(body):
    """(MFMA address, address of the use, steps passed, steps needed) of every
    use of an MFMA's result that comes too early on some path."""
    index = {addr: i for i, (_, _, addr) in enumerate(body)}
    sets = []
    for ins, args, addr in body:  # (reads, writes) of vector registers
        first, _, rest = args.partition(",")
        if ins.startswith("v_mfma"):
            ops = re.findall(r"v\[\d+:\d+\]|v\d+|[^,\s]+", args)
            sets.append((regs(ops[1]) | regs(ops[2]), regs(ops[0])))
        elif re.match(r"v_(swap|permlane\d+_swap)", ins):
            sets.append((regs(args), regs(args)))
        elif ins.startswith(("ds_write", "global_store", "buffer_store", "scratch_store",
                             "global_load_lds", "global_atomic")):
            sets.append((regs(args), set()))
        elif ins.startswith(("v_", "ds_", "global_", "buffer_", "scratch_", "flat_")):
            reads = regs(args) if ins.startswith(("v_fmac", "v_pk_fmac", "v_dot")) else regs(rest)
            sets.append((reads, regs(first)))
        else:
            sets.append((set(), set()))
    found = []
    for i, (ins, args, addr) in enumerate(body):
        if not ins.startswith("v_mfma"):
            continue
        need = next(n for shape, n in STEPS.items() if shape in ins)
        paths, seen = [(i + 1, 0, frozenset(sets[i][1]))], {}
        while paths:
            j, passed, live = paths.pop()
            while j < len(body) and passed < need and live:
                if seen.get((j, live), need) <= passed:
                    break
                seen[j, live] = passed
                op, a, at = body[j]
                reads, writes = sets[j]
                mfma = op.startswith("v_mfma")
                if reads & live or (writes & live and not mfma):
                    found.append((addr, at, passed, need))
                    break
                live = live - writes
                passed += int(a) + 1 if op == "s_nop" else 1
                if op == "s_endpgm":
                    break
                if op.startswith(("s_branch", "s_cbranch")):
                    off = int(a.split()[0]) & 0xFFFF
                    to = index[at + 4 + 4 * (off - 0x10000 if off & 0x8000 else off)]
                    if op == "s_branch":
                        j = to
                        continue
                    paths.append((to, passed, live))
                j += 1
    return found


def test_library_waits_for_its_matrix_results(tmp_path):
    objdump = os.path.join(LLVM, "llvm-objdump")
    if not os.path.exists(objdump):
        pytest.skip("no llvm-objdump")
    if not os.path.exists(moe.LIB_PATH):
        from quantized_mixture_experts_fp32_amd import build
        build.build()
    kernels = mfmas = 0
    for n, code in enumerate(device_objects(moe.LIB_PATH)):
        path = tmp_path / f"{n}.o"
        path.write_bytes(code)
        r = subprocess.run([objdump, "-d", "--mcpu=gfx950", str(path)], capture_output=True,
                           text=True, check=True)
        for name, body in parse(r.stdout).items():
            count = sum(ins.startswith("v_mfma") for ins, _, _ in body)
            if count:
                kernels, mfmas = kernels + 1, mfmas + count
                found = early_uses(body)
                assert not found, (name, [(hex(a), hex(b), c, d) for a, b, c, d in found[:5]])
    assert kernels >= 20 and mfmas >= 1000, (kernels, mfmas)


LISTING = """
0000000000001000 <k>:
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]  // 000000001000: D3B50000
\ts_cbranch_execz 2                                           // 000000001008: BF880002 <k+0x14>
\ts_nop 6                                                     // 00000000100C: BF800006
\tv_add_f32_e32 v20, v21, v22                                 // 000000001010: 02282D15
\tv_mul_f32_e32 v4, v2, v5                                    // 000000001014: 0A080B02
\ts_endpgm                                                    // 000000001018: BF810000
"""


def test_walk_finds_a_use_behind_a_branch():
    """The fall-through takes 9 steps, the branch around it 1; with the wait in
    front of the branch, or the branch taken out, nothing is early."""
    body = parse(LISTING)["k"]
    assert early_uses(body) == [(0x1000, 0x1014, 1, 8)]
    assert early_uses([body[0], ("s_nop", "6", 0x1004), *body[1:]]) == []
    assert early_uses([body[0], *body[2:]]) == []
    assert early_uses([body[0], ("v_mov_b32_e32", "v1, v9", 0x1004), *body[2:]]) == [
        (0x1000, 0x1004, 0, 8)]  # overwritten while in flight
    chain = ("v_mfma_f32_16x16x32_bf16", "v[0:3], v[8:11], v[12:15], v[0:3]", 0x1004)
    assert early_uses([body[0], chain, *body[2:]]) == []
    reads = ("v_mfma_f32_16x16x32_bf16", "v[4:7], v[0:3], v[12:15], v[4:7]", 0x1004)
    assert early_uses([body[0], reads, *body[2:]]) == [(0x1000, 0x1004, 0, 8)]
