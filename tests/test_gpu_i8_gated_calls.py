"""GPU tests of the 8-bit linear map at its largest sizes and over the range of its
scales."""
import pytest
import torch

import i8_gated_ref as ref
import quantized_mixture_experts_fp32_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.mark.parametrize("T", [1, 16])
def test_few_tokens_and_most_features(T):
    """From 2^27 features on the kernel for few tokens would need 2^32 threads: a
    tile takes them.  The bounds are those of every linear map here."""
    N, K = (1 << 27) + 24, 16
    print(f"linear_i8 T={T} N={N} K={K} {moe.moe_linear_i8_kernel(T, N, K)}", flush=True)
    g = torch.Generator(DEV).manual_seed(T)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF16)
    codes = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    scales = torch.rand(N, generator=g, device=DEV) + 0.5
    out = moe.moe_linear_i8(x, codes, scales)
    assert out.shape == (T, N)
    xq, xs = moe.moe_quantize_i8(x, group=0)
    for at in (0, N // 3 // 8 * 8, (1 << 26) - 64, (1 << 27) - 64, N - 128):
        s = slice(at, at + 128)
        want, e = ref.linear_i8(xq, xs, codes[s], scales[s], None)
        ref.check(f"columns from {at}", out[:, s], want, ref.stored(want, e, False))


@pytest.mark.parametrize("T,N,K", [(1, 40, 64), (8, 40, 512), (16, 72, 256), (17, 264, 256),
                                   (300, 520, 272)])
@pytest.mark.parametrize("ex,ew", [(-112, -14), (-100, -24), (100, -60), (60, -110), (-110, 30)])
def test_scales_far_apart(T, N, K, ex, ew):
    """Rows and weights of very different sizes, whose two scales' product alone would
    be below fp32's normal numbers or round there: the bounds are the same four fp32
    steps (and a sum below 2^-126 half a step of the smallest number, twice)."""
    print(f"linear_i8 T={T} N={N} K={K} x 2^{ex} w 2^{ew}", flush=True)
    g = torch.Generator(DEV).manual_seed(T + N + K)
    x = (torch.randn(T, K, generator=g, device=DEV) * 2.0 ** ex).to(BF16)
    w = torch.randn(N, K, generator=g, device=DEV) * 2.0 ** ew
    codes, scales = moe.moe_quantize_i8(w, group=0)
    xq, xs = moe.moe_quantize_i8(x, group=0)
    assert codes.any() and xq.any()
    want, e = ref.linear_i8(xq, xs, codes, scales, None)
    for kw in (dict(x=x), dict(x=xq, x_scales=xs)):
        got = moe.moe_linear_i8(codes=codes, scales=scales, out_dtype=moe.MOE_OUT_F32, **kw)
        ref.check("out", got, want, e + 2.0 ** -149)


@pytest.mark.parametrize("T", [1, 8, 16, 17, 300])
def test_nothing_times_large_scales(T):
    """Sums of 0 stay 0 where the product of the two scales is above fp32's range."""
    N, K = 72, 256
    print(f"linear_i8 T={T} N={N} K={K}", flush=True)
    x, w = torch.zeros(T, K, device=DEV), torch.zeros(N, K, device=DEV)
    x[:, :K // 2] = 2.0 ** 120
    w[::2, K // 2:] = 2.0 ** 40       # meets x's zeros
    w[1::2, :K // 2] = 2.0 ** -100
    codes, scales = moe.moe_quantize_i8(w, group=0)
    bias = torch.randn(N, device=DEV)
    got = moe.moe_linear_i8(x.to(BF16), codes, scales, bias, out_dtype=moe.MOE_OUT_F32)
    assert torch.equal(got[:, ::2], bias[::2].expand(T, -1))
    xq, xs = moe.moe_quantize_i8(x, group=0)
    want, e = ref.linear_i8(xq, xs, codes, scales, bias)
    ref.check("out", got, want, e)
