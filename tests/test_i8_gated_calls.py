"""CPU tests of the shared expert's calls around their kernels: what is recorded
on a side stream, and which kernel takes the largest sizes."""
import contextlib
import os
import re

import pytest
import torch

import quantized_mixture_experts_fp32_amd as moe


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from quantized_mixture_experts_fp32_amd import build
        build.build()
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
