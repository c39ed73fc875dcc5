"""GPU tests of the 8-bit rows (codes and scales bit for bit), the norm and its
gradient read from a checkpoint, and the 8-bit linear map."""
import numpy as np
import pytest
import torch

import i8_gated_ref as ref
import quantized_mixture_experts_fp32_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def rows(T, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g) * scale
    x *= 1 + 20 * (torch.rand(K, generator=g) < 0.02)
    return x.to(dtype)


def behind(t, fill):
    """t on the GPU with `fill` in the memory after it."""
    room = torch.full((t.numel() + 4096,), fill, dtype=t.dtype, device=DEV)
    v = room[:t.numel()].view(t.shape)
    v.copy_(t)
    return v


SHAPES = [(1, 8), (1, 128), (3, 136), (2, 2048), (5, 2056), (17, 4096), (33, 120), (2, 8192),
          (3, 8200), (257, 520), (1000, 1032)]


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("T,K", SHAPES)
def test_quantize_bit_for_bit(T, K, group, dtype):
    print(f"quantize_i8 T={T} K={K} group={group} {dtype}", flush=True)
    x = rows(T, K, dtype, T + K)
    if T > 2:
        x[1] = 0
        x[2, :3] = 0
    want, ws = ref.quantize(x.float().numpy(), group)
    room = torch.full((T * K + 4096,), 99, dtype=torch.int8, device=DEV)
    codes, scales = moe.moe_quantize_i8(behind(x, float("nan")), group,
                                        codes=room[:T * K].view(T, K))
    assert np.array_equal(codes.cpu().numpy(), want)
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert (room[T * K:] == 99).all()
    for code, out in ((moe.MOE_OUT_F32, torch.float32), (moe.MOE_OUT_BF16, BF16)):
        back = moe.moe_dequantize_i8(codes, scales, out_dtype=code)
        s = torch.from_numpy(ws)
        s = s[:, None] if group == 0 else s.repeat_interleave(128, 1)[:, :K]
        assert torch.equal(back.cpu(), (torch.from_numpy(want).float() * s).to(out))


@pytest.mark.parametrize("group", [128, 0])
def test_quantize_extreme_values(group):
    """Zeros, the smallest and largest values, ties, infinities and NaN."""
    print(f"quantize_i8 extremes group={group}", flush=True)
    K = 256
    x = torch.zeros(12, K)
    x[1, 5] = 2.0 ** -119
    x[2, 5] = 2.0 ** -120
    x[3] = torch.arange(K) - 127.5      # halves: ties to even in group 0 or near them
    x[4, 0], x[4, 1:128] = 127.0, torch.arange(127) - 63.5
    x[5, 7] = float("inf")
    x[6, 130] = float("nan")
    x[7, 0] = 3.4e38
    x[8] = -3.4e38
    x[9, 9] = -float("inf")
    x[10] = 1e-40
    x[11] = torch.linspace(-1, 1, K)
    want, ws = ref.quantize(x.numpy(), group)
    codes, scales = moe.moe_quantize_i8(x.to(DEV), group)
    assert np.array_equal(codes.cpu().numpy(), want)
    assert np.array_equal(scales.cpu().numpy(), ws, equal_nan=True)
    back = moe.moe_dequantize_i8(codes, scales, out_dtype=moe.MOE_OUT_F32).cpu()
    bad = ~torch.isfinite(x).view(12, -1, group or K).all(2)
    bad = bad.repeat_interleave(group or K, 1)
    assert torch.isnan(back[bad]).all() and torch.isfinite(back[~bad]).all()


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 136), (16, 2048), (300, 4096), (513, 2056), (5, 8192)])
def test_norm_from_a_checkpoint(T, d, dtype):
    """moe_rmsnorm and its gradient on codes equal the same calls on the
    restored values bit for bit: one kernel body, fp32 values either way."""
    print(f"norm_i8 T={T} d={d} {dtype}", flush=True)
    f32 = dtype == torch.float32
    code = moe.MOE_OUT_F32 if f32 else moe.MOE_OUT_BF16
    codes, scales = moe.moe_quantize_i8(rows(T, d, dtype, d, 3.0).to(DEV))
    x = moe.moe_dequantize_i8(codes, scales, out_dtype=moe.MOE_OUT_F32)
    g = torch.Generator().manual_seed(1)
    gain = (1 + 0.3 * torch.randn(d, generator=g)).to(DEV)
    dout = torch.randn(T, d, generator=g).to(dtype).to(DEV)
    dres = torch.randn(T, d, generator=g).to(dtype).to(DEV)
    got = moe.moe_rmsnorm(codes, gain, eps=1e-5, out_dtype=code, x_scales=scales)
    assert torch.equal(got, moe.moe_rmsnorm(x, gain, eps=1e-5, out_dtype=code))
    dx, dgain = moe.moe_rmsnorm_bwd(dout, codes, gain, eps=1e-5, dres=dres, x_scales=scales,
                                    dx_dtype=code)
    wx, wgain = moe.moe_rmsnorm_bwd(dout, x, gain, eps=1e-5, dres=dres.float())
    assert dx.dtype == dtype
    # one fp32 body; the compiler may join a product and a sum in one of them:
    # a few steps of the terms (rstd u, the projection, dres)
    rstd = (x.double().pow(2).mean(1, keepdim=True) + 1e-5).rsqrt()
    u = dout.double() * gain.double()
    terms = (rstd * (u.abs() + (x.double() * rstd).abs() * (u * x.double() * rstd).abs().mean(
        1, keepdim=True)) + dres.double().abs())
    bound = (d + 16) * 2 ** -23 * terms + (0 if f32 else 2 ** -8) * wx.double().abs()
    assert ((dx.double() - wx.double()).abs() <= bound).all()
    h = (dout.double() * x.double() * rstd).abs().sum(0)
    assert ((dgain.double() - wgain.double()).abs() <= (d + T) * 2 ** -23 * h).all()


LINEAR = [(1, 8, 16), (1, 2048, 2048), (2, 520, 272), (3, 264, 4096), (16, 1000, 1024),
          (17, 136, 144), (33, 3000, 512), (64, 4096, 4096), (65, 264, 2064), (130, 520, 1040),
          (300, 1032, 528), (1100, 2056, 4096), (2048, 1024, 2048)]


def linear_inputs(T, N, K, bias, seed=0):
    x = rows(T, K, BF16, seed + T)
    w = rows(N, K, torch.float32, seed + N, K ** -0.5)
    b = rows(1, N, torch.float32, seed + 7)[0] if bias else None
    return x, w, b


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear_i8(T, N, K, f32):
    """Both forms of x; the sum is exact, so fp32 results are within four
    roundings."""
    bias = (T + N // 8) % 2 == 0
    print(f"linear_i8 T={T} N={N} K={K} f32={f32} bias={bias}", flush=True)
    x, w, b = linear_inputs(T, N, K, bias)
    codes, scales = moe.moe_quantize_i8(w.to(DEV), group=0)
    codes = behind(codes, 77)
    q, sx = moe.moe_quantize_i8(x.to(DEV), group=0)
    b = None if b is None else b.to(DEV)
    code = moe.MOE_OUT_F32 if f32 else moe.MOE_OUT_BF16
    room = torch.full((T * N + 4096,), 5.0, dtype=torch.float32 if f32 else BF16, device=DEV)
    got = moe.moe_linear_i8(behind(x, float("nan")), codes, scales, bias=b, out_dtype=code,
                            out=room[:T * N].view(T, N))
    assert (room[T * N:] == 5.0).all()
    want, bound = ref.linear_i8(q, sx, codes, scales, b)
    ref.check("linear_i8", got, want, ref.stored(want, bound, f32) + 1e-300)
    again = moe.moe_linear_i8(behind(q, 77), codes, scales, bias=b, out_dtype=code, x_scales=sx)
    assert torch.equal(got, again)


@pytest.mark.parametrize("T", [1, 16, 64, 70])
def test_linear_i8_longest_sum(T):
    """Every code at the end of its range, the longest K: the int32 sum holds."""
    N, K = 8, (1 << 17) - 16
    print(f"linear_i8 longest T={T}", flush=True)
    q = torch.full((T, K), 127, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -127, dtype=torch.int8, device=DEV)
    one = torch.ones(max(T, N), device=DEV)
    got = moe.moe_linear_i8(q, w, one[:N], out_dtype=moe.MOE_OUT_F32, x_scales=one[:T])
    assert torch.equal(got, torch.full_like(got, float(-127 * 127 * K)))


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_linear_i8_rows_that_are_not_finite(T):
    """A token with an infinity or NaN gives NaN, its neighbours what they
    would without it; a token of zeros gives the bias."""
    N, K = 264, 512
    print(f"linear_i8 not finite T={T}", flush=True)
    x, w, b = linear_inputs(T, N, K, True)
    x, b = x.to(DEV), b.to(DEV)
    codes, scales = moe.moe_quantize_i8(w.to(DEV), group=0)
    clean = moe.moe_linear_i8(x, codes, scales, bias=b, out_dtype=moe.MOE_OUT_F32)
    x[T // 2, 3] = float("inf") if T % 2 else float("nan")
    got = moe.moe_linear_i8(x, codes, scales, bias=b, out_dtype=moe.MOE_OUT_F32)
    keep = torch.arange(T, device=DEV) != T // 2
    assert torch.isnan(got[T // 2]).all() and torch.equal(got[keep], clean[keep])
    x[T // 2] = 0
    got = moe.moe_linear_i8(x, codes, scales, bias=b, out_dtype=moe.MOE_OUT_F32)
    assert torch.equal(got[T // 2], b) and torch.equal(got[keep], clean[keep])


def test_no_rows():
    codes, scales = moe.moe_quantize_i8(torch.zeros(0, 256, device=DEV))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)
    assert moe.moe_dequantize_i8(codes, scales).shape == (0, 256)
    w, s = moe.moe_quantize_i8(torch.ones(16, 256, device=DEV), group=0)
    assert moe.moe_linear_i8(torch.zeros(0, 256, device=DEV, dtype=BF16), w, s).shape == (0, 16)
    dx, dgain = moe.moe_rmsnorm_bwd(torch.zeros(0, 256, device=DEV), codes,
                                    torch.ones(256, device=DEV), x_scales=scales)
    assert dx.shape == (0, 256) and (dgain == 0).all()


def test_offsets_beyond_32_bits():
    """Rows whose bytes begin past 4 GiB."""
    T, K = 1 << 20, 4224
    print("quantize_i8 past 4 GiB", flush=True)
    x = torch.zeros(T, K, dtype=BF16, device=DEV)
    last = rows(2, K, BF16, 3)
    x[-2:] = last.to(DEV)
    codes, scales = moe.moe_quantize_i8(x)
    want, ws = ref.quantize(last.float().numpy(), 128)
    assert np.array_equal(codes[-2:].cpu().numpy(), want)
    assert np.array_equal(scales[-2:].cpu().numpy(), ws)
    x.fill_(1.0)
    moe.moe_dequantize_i8(codes, scales, out=x)
    assert (x[:T - 2:65537] == 0).all()
    s = torch.from_numpy(ws).repeat_interleave(128, 1)[:, :K]
    assert torch.equal(x[-2:].cpu(), (torch.from_numpy(want).float() * s).to(BF16))
