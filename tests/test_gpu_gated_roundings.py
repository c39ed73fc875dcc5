"""Every kernel of the gated block on data that shows what a worst-case bound does not:
a lost term, a sum in fewer bits, a rounding that the calls do not state.  GPU."""
import pytest
import torch

import gated_roundings as gr
import quantized_mixture_experts_fp32_amd as moe
from i8_gated_sizes import GATED, JOINT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F64 = torch.bfloat16, torch.float64
F32 = moe.MOE_OUT_F32
NAMES = ("dx", "dw_gate_up", "dw_down")
SIZES = {**GATED, **JOINT}


def random_inputs(T, d, f):
    g = torch.Generator(DEV).manual_seed(T + d + f)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(x=n(T, d).to(BF16), w=(n(2 * f, d) * 2 * d ** -0.5).to(BF16),
                v=(n(d, f) * f ** -0.5).to(BF16), dout=n(T, d).to(BF16))


def gradients(p, gate_up=None, only=None, dout=None, **kw):
    """{name: gradient}, the weights' in fp32; only: that one by itself."""
    x, w, v = kw.pop("x", p["x"]), p["w"], p["v"]
    dout = p["dout"] if dout is None else dout
    if only is None:
        return moe.moe_gated_ffn_bwd(dout, x, w, v, gate_up=gate_up, dw_dtype=F32, **kw)._asdict()
    T, d, f = *x.shape, v.shape[1]
    dt = BF16 if only == "dx" else torch.float32
    out = torch.full({"dx": (T, d), "dw_gate_up": (2 * f, d), "dw_down": (d, f)}[only], 7.0,
                     dtype=dt, device=DEV)
    ws = torch.empty(moe.moe_gated_ffn_bwd_ws_bytes(T, d, f, 0, False, True), dtype=torch.uint8,
                     device=DEV)
    rc = moe.load_library().moe_gated_ffn_bwd(
        dout.data_ptr(), 0, x.data_ptr(), None, gate_up.data_ptr(), w.data_ptr(), v.data_ptr(), T,
        d, f, *[out.data_ptr() if n == only else None for n in NAMES], F32, ws.data_ptr(),
        ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == moe.MOE_OK
    return {only: out}


def calls(product, p, kept):
    """The gradient calls that reach a kernel of `product`'s: (gate_up, gradients)."""
    if product == "recompute":
        return [(None, gradients(p))]
    if product == "gradients":
        return [(kept, gradients(p, kept))]
    return [(kept, gradients(p, kept, only=n)) for n in NAMES if product in ("dh", n)]


@pytest.mark.parametrize("product", SIZES)
def test_exact_data(product):
    """Results of exact data are one value each."""
    for name, (T, d, f) in SIZES[product].items():
        print(f"exact {product} {name} T={T} d={d} f={f}", flush=True)
        p = gr.exact_inputs(T, d, f, device=DEV)
        want = gr.exact_results(p)
        out, kept = moe.moe_gated_ffn(p["x"], p["w"], p["v"], out_dtype=F32, save=True)
        assert torch.equal(out.to(F64), want["out"]) and torch.equal(kept.to(F64), want["gate_up"])
        if product in ("gate_up", "down"):
            continue
        for _, got in calls(product, p, kept):
            for n, y in got.items():
                e = want[n].float().to(y.dtype)
                assert torch.equal(y, e), (n, (y != e).sum().item())


@pytest.mark.parametrize("product", SIZES)
def test_errors_are_the_stated_roundings(product):
    for name, (T, d, f) in SIZES[product].items():
        print(f"roundings {product} {name} T={T} d={d} f={f}", flush=True)
        p = random_inputs(T, d, f)
        q = {k: m.to(F64) for k, m in p.items()}
        out, kept = moe.moe_gated_ffn(p["x"], p["w"], p["v"], out_dtype=F32, save=True)
        gr.check("out", out, gr.out_of(q["x"], q["w"], q["v"], True))
        if product in ("gate_up", "down"):
            continue
        for gate_up, got in calls(product, p, kept):
            want = gr.gradients_of(q["dout"], q["x"], q["w"], q["v"],
                                   None if gate_up is None else gate_up.to(F64), True)
            for n, y in got.items():
                gr.check(n, y, want[n])


# checkpoint calls by the kernel that forms gate and up again
CHECKPOINTS = {**JOINT["recompute"],
               "apart 128x128": (7374, 2016, 264), "apart 128x128 k2": (7647, 5912, 136),
               "apart 160x256": (5047, 752, 776), "apart 192x256": (3236, 664, 1920),
               "apart 256x256": (1167, 600, 5048), "apart 64x128": (391, 2736, 4136),
               "apart 64x64": (4717, 1376, 416)}


@pytest.mark.parametrize("T,d,f", [(1, 264, 136), (40, 264, 136), (700, 520, 264),
                                   (2600, 1024, 512)])
def test_fp32_dout(T, d, f):
    """Rounded to bf16 once, as the call states, and to nothing less."""
    print(f"fp32 dout T={T} d={d} f={f}", flush=True)
    p = gr.exact_inputs(T, d, f, device=DEV)
    want = gr.exact_results(p)
    for n, y in gradients(p, dout=p["dout"].float()).items():
        assert torch.equal(y, want[n].float().to(y.dtype)), n
    p = random_inputs(T, d, f)
    dout = p["dout"].float() * 1.001
    want = gr.gradients_of(dout.to(BF16).to(F64), *(p[k].to(F64) for k in "xwv"), None, True)
    for n, y in gradients(p, dout=dout).items():
        gr.check(n, y, want[n])


@pytest.mark.parametrize("name", CHECKPOINTS)
def test_checkpoints(name):
    """Gate and up are of the restored rows themselves, whose scales differ from group
    to group; only what dw_gate_up multiplies is rounded to bf16."""
    T, d, f = CHECKPOINTS[name]
    print(f"checkpoint {name} T={T} d={d} f={f}", flush=True)
    p = gr.exact_inputs(T, d, f, device=DEV)
    want = gr.exact_results(p)
    ones = torch.ones(T, -(-d // 128), device=DEV)
    for n, y in gradients(p, x=p["x"].to(torch.int8), x_scales=ones).items():
        assert torch.equal(y, want[n].float().to(y.dtype)), n
    p = random_inputs(T, d, f)
    g = torch.Generator(DEV).manual_seed(T)
    size = torch.exp2(2 * torch.randn(T, -(-d // 128), generator=g, device=DEV))
    x = p["x"].float() * size.repeat_interleave(128, 1)[:, :d] / 4
    codes, scales = moe.moe_quantize_i8(x)
    restored = codes.to(F64) * scales.to(F64).repeat_interleave(128, 1)[:, :d]
    rounded = moe.moe_dequantize_i8(codes, scales).to(F64)
    want = gr.gradients_of(*(t.to(F64) for t in (p["dout"], restored, p["w"], p["v"])), None, True,
                           rounded)
    for n, y in gradients(p, x=codes, x_scales=scales).items():
        gr.check(n, y, want[n])


@pytest.mark.parametrize("T,d,f", [(3, 392, 16), (70, 648, 72), (600, 1160, 136),
                                   (4000, 264, 520)])
def test_checkpoint_rows_of_any_scale(T, d, f):
    """Groups of zeros, of 2^-100 and of 2^60 beside each other, and one that is not
    finite: sums go from unit to unit without loss, and a row that is not finite
    touches its own row of dx alone."""
    print(f"checkpoint rows T={T} d={d} f={f}", flush=True)
    p = random_inputs(T, d, f)
    G = -(-d // 128)
    g = torch.Generator(DEV).manual_seed(T)
    at = torch.randint(0, 4, (T, G), generator=g, device=DEV)
    at[:, 0] = 1
    size = torch.tensor([0.0, 1.0, 2.0 ** -100, 2.0 ** 60], device=DEV)[at]
    x = p["x"].float() * size.repeat_interleave(128, 1)[:, :d]
    w = p["w"].clone()
    big = (at == 3).any(0).repeat_interleave(128)[:d]
    w[:, big] = (w[:, big].float() * 2.0 ** -62).to(BF16)
    codes, scales = moe.moe_quantize_i8(x)
    p["w"] = w
    restored = codes.to(F64) * scales.to(F64).repeat_interleave(128, 1)[:, :d]
    rounded = moe.moe_dequantize_i8(codes, scales).to(F64)
    want = gr.gradients_of(*(t.to(F64) for t in (p["dout"], restored, w, p["v"])), None, True,
                           rounded)
    clean = gradients(p, x=codes, x_scales=scales)
    for n, y in clean.items():
        gr.check(n, y, want[n])
    scales[T // 2, G - 1] = float("nan")
    codes[T // 2, 128 * (G - 1):] = 0
    got = gradients(p, x=codes, x_scales=scales)["dx"]
    keep = torch.arange(T, device=DEV) != T // 2
    assert torch.isnan(got[T // 2]).all() and torch.equal(got[keep], clean["dx"][keep])
