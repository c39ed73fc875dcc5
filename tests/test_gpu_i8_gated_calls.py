"""GPU tests of the 8-bit linear map at its largest sizes and over the range of its
scales, and of the gated gradient's forms with workspaces of the size they need."""
import re

import pytest
import torch

import i8_gated_ref as ref
import quantized_mixture_experts_fp32_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F64 = torch.bfloat16, torch.float64


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


# --------------------------------------------- the gradient's forms and its workspace
NAMES = ("dx", "dw_gate_up", "dw_down")
SUBSETS = [[n for i, n in enumerate(NAMES) if m >> i & 1] for m in range(1, 8)]


def block(T, d, f):
    g = torch.Generator(DEV).manual_seed(T + d + f)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(x=n(T, d).to(BF16), w=(n(2 * f, d) * 2 * d ** -0.5).to(BF16),
                v=(n(d, f) * f ** -0.5).to(BF16), dout=n(T, d).to(BF16))


def call(p, source, wanted, fill, f32=False):
    """The C entry with a workspace of exactly the bytes that it asks for, filled with
    `fill`, and nothing but 0x5a behind it."""
    lib = moe.load_library()
    T, d = p["x"].shape
    f = p["v"].shape[1]
    dout = p["dout"].float() if f32 else p["dout"]
    x, sx, gu = p["x"], None, None
    if source == "saved":
        gu = moe.moe_gated_ffn(x, p["w"], p["v"], save=True)[1]
    elif source != "recompute":
        x, sx = moe.moe_quantize_i8(x)
        if source == "checkpoint saved":
            gu = moe.moe_gated_ffn(p["x"], p["w"], p["v"], save=True)[1]
    dt = torch.float32 if f32 else BF16
    shape = {"dx": (T, d), "dw_gate_up": (2 * f, d), "dw_down": (d, f)}
    out = {n: torch.full(shape[n], 7.0, dtype=BF16 if n == "dx" else dt, device=DEV)
           for n in wanted}
    at = [out[n].data_ptr() if n in out else None for n in NAMES]

    def run(ws, size):
        a = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        return lib.moe_gated_ffn_bwd(dout.data_ptr(), int(f32), a(x), a(sx), a(gu), a(p["w"]),
                                     a(p["v"]), T, d, f, *at, int(f32), ws.data_ptr(), size,
                                     torch.cuda.current_stream().cuda_stream)

    assert run(dout, 0) == moe.MOE_ERR_WORKSPACE  # (nothing is enqueued)
    need = int(re.search(rb"< (\d+) bytes", lib.moe_last_error())[1])
    assert need <= moe.moe_gated_ffn_bwd_ws_bytes(T, d, f, int(f32), sx is not None,
                                                  gu is not None)
    room = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device=DEV)
    room[:need] = fill
    assert run(room, need) == moe.MOE_OK
    assert (room[need:] == 0x5A).all()
    return out


@pytest.mark.parametrize("source", ["saved", "recompute", "checkpoint", "checkpoint saved"])
@pytest.mark.parametrize("T,d,f", [(1, 264, 136), (40, 328, 40), (75, 40, 1744), (700, 520, 264),
                                   (1477, 8, 8), (3236, 664, 1920)])
def test_any_outputs_and_an_exact_workspace(T, d, f, source):
    """Each set of outputs, with a workspace of the needed size that held NaN or zeros:
    the bytes behind it stay, and what it held is not read."""
    print(f"gradient T={T} d={d} f={f} {source}", flush=True)
    p = block(T, d, f)
    x, rounded, gu = p["x"].to(F64), False, None
    if source.startswith("checkpoint"):
        x, rounded = ref.restore(*moe.moe_quantize_i8(p["x"])), True
    if source.endswith("saved"):
        gu = moe.moe_gated_ffn(p["x"], p["w"], p["v"], save=True)[1].to(F64)
    for f32 in (False, True):
        want, bounds = ref.gated_ffn_bwd(p["dout"].to(F64), x, p["w"].to(F64), p["v"].to(F64), gu,
                                         False, rounded, f32)
        for wanted in SUBSETS:
            got = call(p, source, wanted, 255, f32)
            again = call(p, source, wanted, 0, f32)
            for n, y in got.items():
                ref.check(f"{n} of {wanted}", y, want[NAMES.index(n)], bounds[NAMES.index(n)])
                assert torch.equal(y, again[n])


@pytest.mark.parametrize("T,d,f", [(40, 328, 40), (700, 520, 264), (1200, 1024, 512)])
def test_checkpoint_gradient_on_a_stream_and_in_graphs(T, d, f):
    """From codes: on a side stream, and recorded twice with one workspace and replayed
    with other rows and eager calls in between; every result equals the eager one."""
    print(f"checkpoint graphs T={T} d={d} f={f}", flush=True)
    p = block(T, d, f)
    codes, scales = moe.moe_quantize_i8(p["x"])
    ws = torch.empty(moe.moe_gated_ffn_bwd_ws_bytes(T, d, f, 0, True), dtype=torch.uint8,
                     device=DEV)

    def run(**kw):
        return moe.moe_gated_ffn_bwd(p["dout"], codes, p["w"], p["v"], x_scales=scales, **kw)

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(ws=ws)
        graphs.append((g, out))
    for turn in range(3):
        c, s = moe.moe_quantize_i8(p["x"].float() * 1.7 ** turn)
        codes.copy_(c.roll(turn, 0))
        scales.copy_(s.roll(turn, 0))
        want = run()
        for g, out in graphs:
            for t in out:
                t.fill_(7)
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
