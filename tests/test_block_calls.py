"""How the operators around the routed experts are called: every parameter by
name, as their signatures show them (CPU: refused before any launch; GPU: equal
to the positional calls)."""
import inspect

import pytest
import torch

import quantized_mixture_experts_fp32_amd as moe

DEV = "cuda:0"
CALLS = ("moe_linear_w4", "moe_rmsnorm", "moe_rmsnorm_bwd", "moe_combine_residual",
         "moe_combine_residual_bwd", "moe_dispatch", "moe_dispatch_bwd", "moe_combine_bwd")


def inputs(name, device):
    """The required arguments of a call, in order."""
    g = torch.Generator().manual_seed(3)
    T, d, k = 4, 128, 2
    n = lambda *s: torch.randn(*s, generator=g).to(device)  # noqa: E731
    pos = torch.randperm(T * k, generator=g).to(torch.int32).to(device)
    codes = torch.randint(0, 256, (16, 64), generator=g, dtype=torch.uint8).to(device)
    w = torch.rand(T, k, generator=g).to(device)
    return {
        "moe_linear_w4": dict(x=n(T, d).to(torch.bfloat16), codes=codes,
                              scales=(w.new_ones(16, 1) * 0.1).half()),
        "moe_rmsnorm": dict(x=n(T, d)),
        "moe_rmsnorm_bwd": dict(dout=n(T, d), x=n(T, d)),
        "moe_combine_residual": dict(residual=n(T, d), y_pairs=n(T * k, d), pair_pos=pos,
                                     topk_w=w),
        "moe_combine_residual_bwd": dict(dout=n(T, d), y_pairs=n(T * k, d), pair_pos=pos,
                                         topk_w=w),
        "moe_dispatch": dict(x=n(T, d), pair_pos=pos, k=k),
        "moe_dispatch_bwd": dict(dxs=n(T * k, d), pair_pos=pos, k=k),
        "moe_combine_bwd": dict(dout=n(T, d), y_pairs=n(T * k, d), pair_pos=pos, topk_w=w),
    }[name]


@pytest.mark.parametrize("name", CALLS)
def test_calls_by_name_reach_the_checks(name):
    """A call with every argument by name gets as far as the device check."""
    with pytest.raises(ValueError, match="expected a GPU"):
        getattr(moe, name)(**inputs(name, "cpu"))


@pytest.mark.parametrize("name", CALLS)
def test_signatures_show_what_the_calls_take(name):
    call = getattr(moe, name)
    sig = inspect.signature(call)
    lead = next(iter(sig.parameters))
    assert sig.parameters["stream"].kind is inspect.Parameter.KEYWORD_ONLY
    with pytest.raises(TypeError, match=f"'{lead}'"):
        call()
    with pytest.raises(TypeError, match=f"'{lead}_'"):
        call(**{lead + "_": torch.zeros(4, 128)})
    with pytest.raises(ValueError, match="a tensor is needed"):
        call(**{**inputs(name, "cpu"), lead: None})


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_calls_by_name_equal_positional_calls(name):
    print(f"by name: {name}", flush=True)
    args = inputs(name, DEV)
    want = flat(getattr(moe, name)(*args.values()))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for kw in ({}, dict(stream=side)):
        got = flat(getattr(moe, name)(**args, **kw))
        torch.cuda.synchronize()
        assert len(got) == len(want)
        for a, b in zip(want, got):
            assert torch.equal(a, b)
