"""GPU tests of the 8-bit linear map at its largest sizes."""
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
