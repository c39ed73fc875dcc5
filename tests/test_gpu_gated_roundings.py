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


@pytest.mark.parametrize("T,d,f", [(40, 264, 136), (700, 520, 264), (2600, 1024, 512)])
def test_fp32_dout_and_checkpoints(T, d, f):
    """Both are rounded to bf16 once, as the calls state, and to nothing less."""
    print(f"sources T={T} d={d} f={f}", flush=True)
    p = gr.exact_inputs(T, d, f, device=DEV)
    want = gr.exact_results(p)
    codes = p["x"].to(torch.int8)
    scales = torch.ones(T, -(-d // 128), device=DEV)
    got = gradients(p, x=codes, x_scales=scales, dout=p["dout"].float())
    for n, y in got.items():
        assert torch.equal(y, want[n].float().to(y.dtype)), n
    p = random_inputs(T, d, f)
    dout = p["dout"].float() * 1.001
    codes, scales = moe.moe_quantize_i8(p["x"])
    x = moe.moe_dequantize_i8(codes, scales)  # bf16
    got = gradients(p, x=codes, x_scales=scales, dout=dout)
    want = gr.gradients_of(dout.to(BF16).to(F64), x.to(F64), p["w"].to(F64), p["v"].to(F64), None,
                           True)
    for n, y in got.items():
        gr.check(n, y, want[n])
