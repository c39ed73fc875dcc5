"""The 4-bit linear map's kernels at what each of them can get wrong: scales of
very different sizes in a row, groups without weight, large values, infinities
and NaN, workspaces, streams and graphs.  linear_shapes lists shapes by the
kernel that they run (checked on the CPU)."""
import pytest
import torch

import block_ref as ref
import quantized_mixture_experts_fp32_amd as moe
from block_ref import assert_within, f64
from linear_shapes import EACH, LISTED

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


# ------------------------------------------------------------- every kernel
def quantized(T, K, N, seed):
    """x bf16, codes and scales as a quantizer writes them for normal weights
    of 1 / sqrt(K), and a bias; made on the device."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    low, high = codes & 15, codes >> 4
    codes = torch.where(low == 8, 9, low) | (torch.where(high == 8, 9, high) << 4)
    scales = (1 + torch.rand(N, K // 128, generator=g, device=DEV)) * 0.3 / K ** 0.5
    return x, codes, scales.to(torch.float16), torch.randn(N, generator=g, device=DEV)


def slices(N):
    """Row ranges: the first, two inside, the last (whole row tiles)."""
    if N <= 4096:
        return [(0, N)]
    mid = N // 32 * 16
    return [(0, 528), (2032, 2320), (mid, mid + 272), (N - 528, N)]


@pytest.mark.parametrize("out_dtype", [moe.MOE_OUT_BF16, moe.MOE_OUT_F32])
@pytest.mark.parametrize("name,T,K,N", LISTED)
def test_every_kernel(name, T, K, N, out_dtype):
    note(f"linear {name} T={T} K={K} N={N} out={out_dtype}")
    x, codes, scales, bias = quantized(T, K, N, T + K + N)
    guard = torch.full((T * N + 1024,), -7.0, dtype=F32 if out_dtype else BF, device=DEV)
    out = guard[512:512 + T * N].view(T, N)
    moe.moe_linear_w4(x, codes, scales, bias=bias, out=out, out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert (guard[:512] == -7.0).all() and (guard[512 + T * N:] == -7.0).all()
    for a, b in slices(N):
        W = codes[a:b].contiguous(), scales[a:b].contiguous()
        y, bound = ref.linear(x, *W, bias[a:b].contiguous())
        if name.startswith("gemm"):
            G = K // 128
            s = f64(scales[a:b])
            ax = f64(x).abs().reshape(T, G, 128).sum(2)
            bound = (ref.U * (G * (2 * (128 + 3) + 4) + 132) * 55 * (ax @ s.t().contiguous())
                     + ref.U * y.abs())
        assert_within(out[:, a:b], y, bound, f"rows {a}..{b}")
        # in rms: 16 times an fp32 rounding (256 of them) of a partial sum of
        # some 1500 sigma, and in the GEMM of the total (335 sigma a group),
        # against 335 sigma a group; four times that, and the store
        G = K // 128 if name.startswith("gemm") else 0
        tol = 4 * 16 * (1500 ** 2 + G * 335 ** 2) ** 0.5 / 335 * ref.U
        rel = float((f64(out[:, a:b]) - y).norm() / y.norm())
        assert rel <= tol + ref.HALF_STEP[out.dtype], (a, rel, tol)


@pytest.mark.parametrize("name,T,K,N", EACH)
def test_every_kernel_keeps_infinities_in_their_row(name, T, K, N):
    note(f"linear nonfinite {name} T={T} K={K} N={N}")
    x, codes, scales, _ = quantized(T, K, N, 1)
    clean = moe.moe_linear_w4(x, codes, scales)
    x = x.clone()
    x[0, K - 5] = float("inf")
    x[T - 1, 3] = float("nan")
    out = moe.moe_linear_w4(x, codes, scales)
    assert torch.equal(out[1:T - 1], clean[1:T - 1])
    assert not torch.isfinite(out[0]).any() and out[T - 1].isnan().all()


@pytest.mark.parametrize("name,T,K,N", EACH)
def test_every_kernel_with_large_values_and_no_weights(name, T, K, N):
    """Values near 2^100 with groups of scale 0, whose codes are -8 as well."""
    note(f"linear large values, scales of 0 {name} T={T} K={K} N={N}")
    x, codes, scales, _ = quantized(T, K, N, 2)
    x = (x.float().clamp(-3.9, 3.9) * 2.0 ** 100).to(BF)
    scales[::3, 1] = 0
    scales[5] = 0
    codes.view(N // 16, K // 128, 16, 64)[:, 1, ::3] = 0x88
    out = moe.moe_linear_w4(x, codes, scales, out_dtype=moe.MOE_OUT_F32)
    for a, b in slices(N):
        y, bound = reference(x, codes[a:b].contiguous(), scales[a:b].contiguous())
        if name.startswith("gemm"):
            s = f64(scales[a:b])
            ax = f64(x).abs().reshape(T, K // 128, 128).sum(2)
            bound = (ref.U * (K // 128 * (2 * (128 + 3) + 4) + 132) * 55
                     * (ax @ s.t().contiguous()))
        assert_within(out[:, a:b], y, bound, f"rows {a}..{b}")
    assert (out[:, 5] == 0).all()


@pytest.mark.parametrize("name,T,K,N", EACH)
def test_every_kernel_on_streams_and_in_graphs(name, T, K, N):
    """Side stream, a workspace of the caller's, a graph replayed beside eager
    calls on other inputs: equal to the first call bit for bit."""
    note(f"linear stream, workspace, graph {name} T={T} K={K} N={N}")
    x, codes, scales, bias = quantized(T, K, N, 3)
    other = quantized(T, K, N, 4)
    want = moe.moe_linear_w4(x, codes, scales, bias=bias)
    need = moe.moe_linear_w4_ws_bytes(T, N, K)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = moe.moe_linear_w4(x, codes, scales, bias=bias, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((need + 512,), 0x7F, dtype=torch.uint8, device=DEV)
    got = moe.moe_linear_w4(x, codes, scales, bias=bias, ws=ws[:max(need, 256)])
    assert torch.equal(got, want) and (ws[max(need, 256):] == 0x7F).all()
    if need:
        with pytest.raises(moe.MoeError, match="workspace"):
            moe.moe_linear_w4(x, codes, scales, ws=ws[:need - 8])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.moe_linear_w4(x, codes, scales, bias=bias)
    for _ in range(3):
        out.fill_(-3.0)
        moe.moe_linear_w4(*other[:3], bias=other[3])
        graph.replay()
        moe.moe_linear_w4(*other[:3], bias=other[3])
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_graphs_with_workspaces_at_once():
    """Two recorded calls that each need a workspace, replayed on two streams."""
    note("linear two graphs with workspaces")
    sets = [quantized(1500, 256, 8208, s) for s in (5, 6)]
    want = [moe.moe_linear_w4(*a[:3], bias=a[3]) for a in sets]
    graphs, got = [], []
    for a in sets:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            got.append(moe.moe_linear_w4(*a[:3], bias=a[3]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(8):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert torch.equal(w, o)
