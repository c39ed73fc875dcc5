"""The 4-bit linear map's kernels at what each of them can get wrong: scales of
very different sizes in a row, groups without weight, large values."""
import pytest
import torch

import block_ref as ref
import quantized_mixture_experts_fp32_amd as moe
from block_ref import assert_within, f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def note(msg):
    print(msg, flush=True)


def is_gemm(T, K, N):
    """Only the GEMM needs a workspace."""
    return moe.moe_linear_w4_ws_bytes(T, N, K) > 0


def reference(x, codes, scales, bias=None):
    """(y, bound) for any of the kernels.  The tile and streaming kernels sum
    each group apart: block_ref.linear's count.  The GEMM carries one total
    through all groups: per group the MFMA steps over 128 products and up to 3
    parts of the group's sum (an MFMA may align its products to the largest and
    cut them there, so each counts twice), the step to the group's unit (a
    quotient and a product, 4 roundings); once the group sums' own 128 and 4 at
    the end.  Terms as there, up to 440 / 8 times |s x|."""
    y, bound = ref.linear(x, codes, scales, bias)
    T, K = x.shape
    N, G = codes.shape[-2], K // 128
    if is_gemm(T, K, N):
        s = scales.reshape(N, G).view(torch.float16).double().abs()
        ax = f64(x).abs().reshape(T, G, 128).sum(2)
        roundings = G * (2 * (128 + 3) + 4) + 128 + 4
        bound = ref.U * roundings * (440.0 / 8) * (ax @ s.t().contiguous())
        if bias is not None:
            bound = bound + ref.U * y.abs()
    return y, bound


# one tile, one GEMM in tiles of 96 or 128 tokens, one with a longer K
SHAPES = [(40, 1024, 208), (1500, 256, 8208), (2501, 1280, 2064), (1500, 2560, 4112)]
# scales of the groups of K, in turn over the rows
STEPS = {"down": (0, -20), "up": (-20, 0), "stairs": (0, -7, -14, -21),
         "there and back": (-2, -24, -2), "one apart": (0, -1, 0, -2)}


def inputs(T, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).to(DEV)
    # as a quantizer writes them: no -8
    low, high = codes & 15, codes >> 4
    codes = torch.where(low == 8, 9, low) | (torch.where(high == 8, 9, high) << 4)
    return g, x, codes.contiguous()


@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_scales_of_different_sizes(T, K, N, steps):
    """Neighbouring groups whose scales are up to 2^22 apart, and values below
    the smaller of 2^110 and 2^120 / K: finite, and within the bound."""
    note(f"linear unequal scales T={T} K={K} N={N} {steps}")
    g, x, codes = inputs(T, K, N, T + K)
    x = x.clamp(-3.9, 3.9) * min(2.0 ** 107, 2.0 ** 117 / K)
    G = K // 128
    e = torch.tensor(STEPS[steps])
    at = (torch.arange(G)[None, :] + torch.arange(N)[:, None]) % len(e)
    s = torch.pow(2.0, e[at].float()) * (1 + torch.rand(N, G, generator=g)).clamp_max(1.99)
    s[1::3] *= -1
    scales = s.to(torch.float16).to(DEV)
    x = x.to(BF).to(DEV)
    out = moe.moe_linear_w4(x, codes, scales, out_dtype=moe.MOE_OUT_F32)
    y, bound = reference(x, codes, scales)
    assert float(y.abs().max()) < 2.0 ** 126 and torch.isfinite(out).all()
    assert_within(out, y, bound, "unequal scales")


@pytest.mark.parametrize("T,K,N", SHAPES)
def test_group_without_weight_contributes_nothing(T, K, N):
    """The activations of a group whose scale is 0 do not enter, however large
    they are next to the others."""
    note(f"linear groups without weight T={T} K={K} N={N}")
    g, x, codes = inputs(T, K, N, 2 * T + K)
    G = K // 128
    scales = (torch.rand(N, G, generator=g) * 0.1 + 0.05).to(torch.float16)
    scales[:, 1::2] = 0
    scales[5] = 0
    x.view(T, G, 128)[:, 1::2] *= 2.0 ** 40
    x, scales = x.to(BF).to(DEV), scales.to(DEV)
    out = moe.moe_linear_w4(x, codes, scales, out_dtype=moe.MOE_OUT_F32)
    y, bound = reference(x, codes, scales)
    assert_within(out, y, bound, "groups without weight")
    assert (out[:, 5] == 0).all()
