"""CPU tests of the shared expert's calls around their kernels: what is recorded
on a side stream."""
import contextlib

import pytest
import torch

import quantized_mixture_experts_fp32_amd as moe


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
