"""CPU tests of the shared expert's calls around their kernels: what is recorded
on a side stream, which kernel takes the largest sizes, what a workspace holds,
and the two libraries."""
import contextlib
import ctypes
import os
import re
import shutil

import pytest
import torch

import quantized_mixture_experts_fp32_amd as moe
from quantized_mixture_experts_fp32_amd import build as package_build


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        package_build.build()
    return moe.load_library()


class Enough(Exception):
    pass


def shared_block(d, f):
    block = moe.GatedFfn.__new__(moe.GatedFfn)
    block.d, block.f = d, f
    block.w_gate_up, block.w_down = torch.zeros(2 * f, d), torch.zeros(d, f)
    return block


# ------------------------------------------------------------- a side stream
@pytest.mark.parametrize("with_shared", [True, False])
def test_shared_weights_are_recorded_on_the_stream(monkeypatch, with_shared):
    """The products of a shared expert read its weights on the call's stream, so
    memory that the caller drops after the call must not be handed out before."""
    layer = moe.MoeLayer.__new__(moe.MoeLayer)
    layer.d, layer.wr = 128, torch.zeros(8, 128)
    block = shared_block(128, 16)
    residual, gain = torch.zeros(4, 128), torch.zeros(128)
    seen = []

    @contextlib.contextmanager
    def launch_on(stream, values):
        seen.extend(v for v in values if v is not None)
        raise Enough
        yield

    monkeypatch.setattr(moe, "_launch_on", launch_on)
    with pytest.raises(Enough):
        layer.forward_block(residual, gain, shared=block if with_shared else None,
                            stream=object())
    want = [residual, gain] + ([block.w_gate_up, block.w_down] if with_shared else [])
    assert {id(t) for t in seen} == {id(t) for t in want}


def test_a_block_that_kept_nothing():
    with pytest.raises(ValueError, match="keep=False"):
        shared_block(128, 16).backward_block(torch.zeros(4, 128), None)


# ---------------------------------------------------------- the largest launches
def threads(name, T, N):
    """Of the linear map's launch: 512 for 16 features (few tokens), or a tile's
    256 (rows times features up to 128 x 128 by one group of waves) or 512."""
    if name == "direct":
        return -(-N // 16) * 512
    bm, bn, k2 = re.fullmatch(r"tile (\d+)x(\d+)( k2)?", name).groups()
    bm, bn = int(bm), int(bn)
    block = 256 if bm * bn < 128 * 128 or (bm, bn, k2) == (128, 128, None) else 512
    return -(-T // bm) * -(-N // bn) * block


@pytest.mark.parametrize("K", [16, 48])
def test_every_size_can_be_launched(lib, K):
    """A launch has fewer than 2^32 threads (a HIP limit)."""
    for T in (1, 2, 8, 9, 16, 17, 32, 33, 63, 64, 65, 129):
        for N in ((1 << 27) - 16, (1 << 27) - 8, 1 << 27, (1 << 27) + 8, (1 << 28) - 8):
            if T * N >= 1 << 34:
                continue
            name = moe.moe_linear_i8_kernel(T, N, K)
            assert name and threads(name, T, N) < 1 << 32, (T, N, name)
    assert moe.moe_linear_i8_kernel(16, (1 << 27) - 16, K) == "direct"
    assert moe.moe_linear_i8_kernel(1, (1 << 27) - 8, K) != "direct"
    # (the few-token kernel forms up to 8 tokens' codes by itself, the tiles do not)
    assert moe.moe_linear_i8_ws_bytes(1, (1 << 27) - 16, K) == 0
    assert moe.moe_linear_i8_ws_bytes(1, 1 << 27, K) >= K + 4


# ------------------------------------------------------------- the workspaces
def needed(lib, T, d, f, do_f32, x_i8, kept):
    """What the gradient asks for, from its refusal of a workspace of no bytes."""
    p = ctypes.c_void_p(0x10000)
    rc = lib.moe_gated_ffn_bwd(p, int(do_f32), p, p if x_i8 else None, p if kept else None, p, p,
                               T, d, f, p, p, p, 0, p, 0, None)
    assert rc == moe.MOE_ERR_WORKSPACE, rc
    return int(re.search(rb"< (\d+) bytes", lib.moe_last_error())[1])


@pytest.mark.parametrize("form", [(0, 0, 0), (0, 0, 1), (1, 1, 0)])
@pytest.mark.parametrize("d,f", [(2048, 1024), (256, 1824), (264, 2288), (4096, 136), (72, 136),
                                 (2224, 152)])
def test_a_workspace_serves_smaller_batches(lib, d, f, form):
    """A workspace for T tokens is large enough for fewer of them, whichever
    kernels these choose."""
    last = 0
    step = lambda T: 1 if T < 300 else 37 if T < 3000 else 173  # noqa: E731
    T = 1
    while T < 17000:
        at = moe.moe_gated_ffn_bwd_ws_bytes(T, d, f, *form)
        assert at >= last and at >= needed(lib, T, d, f, *form), (T, last, at)
        last, T = at, T + step(T)


def test_a_workspace_is_not_larger_than_needed(lib):
    """The largest need of so many or fewer tokens: here found one by one."""
    for T in (4, 131, 512, 700, 1024, 2600):
        most = max(needed(lib, t, 2048, 1024, 0, 0, 0) for t in range(1, T + 1))
        assert moe.moe_gated_ffn_bwd_ws_bytes(T, 2048, 1024) == most
    for T in (64, 8000):
        assert moe.moe_gated_ffn_bwd_ws_bytes(T, 4096, 2048, 0, False, True) == needed(
            lib, T, 4096, 2048, 0, 0, 1)


# ---------------------------------------------------------- the two libraries
@pytest.mark.parametrize("there", [(), ("libmoe_wq.so",), ("libmoe_wq_i8.so",)])
def test_a_missing_library_is_named(lib, tmp_path, monkeypatch, there):
    for name in there:
        shutil.copy(os.path.join(moe.HERE, name), tmp_path / name)
    monkeypatch.setattr(moe, "_lib", None)
    monkeypatch.setattr(moe, "LIB_PATH", str(tmp_path / "libmoe_wq.so"))
    missing = "libmoe_wq_i8.so" if there == ("libmoe_wq.so",) else "libmoe_wq.so"
    with pytest.raises(RuntimeError, match=f"{missing} not built: run"):
        moe.load_library()


@pytest.mark.parametrize("fails", ["linear_i8.hip build", "libmoe_wq_i8.so link",
                                   "libmoe_wq.so link", None])
def test_a_failed_build_replaces_neither_library(tmp_path, monkeypatch, fails):
    """The libraries are of one build: both new, or both as they were."""
    libs = [tmp_path / "libmoe_wq.so", tmp_path / "libmoe_wq_i8.so"]
    for p in libs:
        p.write_text("old")

    def run(what, cmd):
        if what == fails:
            raise RuntimeError(what)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return ""

    monkeypatch.setattr(package_build, "_run", run)
    monkeypatch.setattr(package_build, "LIB", str(libs[0]))
    monkeypatch.setattr(package_build, "LIB_I8", str(libs[1]))
    if fails:
        with pytest.raises(RuntimeError, match=fails):
            package_build.build()
    else:
        package_build.build()
    assert [p.read_text() for p in libs] == ["old" if fails else "new"] * 2
    assert sorted(os.listdir(tmp_path)) == ["libmoe_wq.so", "libmoe_wq_i8.so"]
