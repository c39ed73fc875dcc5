"""Each kernel that the gated block's products and the 8-bit linear map choose
from, at a size that reaches it, and calls that overlap.  GPU."""
import pytest
import torch

import i8_gated_ref as ref
import quantized_mixture_experts_fp32_amd as moe
from i8_gated_sizes import GATED, JOINT, LINEAR

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F64 = torch.bfloat16, torch.float64


def block(T, d, f, seed=0):
    g = torch.Generator(DEV).manual_seed(seed + T + d + f)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(x=n(T, d).to(BF16), w=(n(2 * f, d) * 2 * d ** -0.5).to(BF16),
                v=(n(d, f) * f ** -0.5).to(BF16), dout=n(T, d).to(BF16))


def linear(T, N, K, seed=0):
    g = torch.Generator(DEV).manual_seed(seed + T + N + K)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF16)
    w = torch.randn(N, K, generator=g, device=DEV)
    return (x, *moe.moe_quantize_i8(w, group=0), torch.randn(N, generator=g, device=DEV))


def one_gradient(p, kept, name):
    """One output of the gradient's C entry, by itself."""
    lib = moe.load_library()
    T, d = p["x"].shape
    f = p["v"].shape[1]
    shape = {"dx": (T, d), "dw_gate_up": (2 * f, d), "dw_down": (d, f)}
    out = torch.full(shape[name], 7.0, dtype=BF16, device=DEV)
    ws = torch.empty(lib.moe_gated_ffn_bwd_ws_bytes(T, d, f, 0, 0, 1), dtype=torch.uint8,
                     device=DEV)
    at = [out.data_ptr() if n == name else None for n in shape]
    rc = lib.moe_gated_ffn_bwd(p["dout"].data_ptr(), 0, p["x"].data_ptr(), None, kept.data_ptr(),
                               p["w"].data_ptr(), p["v"].data_ptr(), T, d, f, *at, 0,
                               ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == moe.MOE_OK
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("product,name", [(p, n) for p in GATED for n in GATED[p]])
def test_kernel_of_the_block(product, name):
    T, d, f = GATED[product][name]
    print(f"gated {product} {name} T={T} d={d} f={f}", flush=True)
    assert moe.moe_gated_ffn_kernel(product, T, d, f) == name
    p = block(T, d, f)
    q = {n: t.to(F64) for n, t in p.items()}
    want, bound, gu, egu = ref.gated_ffn(q["x"], q["w"], q["v"])
    out, kept = moe.moe_gated_ffn(p["x"], p["w"], p["v"], save=True)
    ref.check("out", out, want, bound)
    ref.check("gate_up", kept, gu, egu)
    if product in ("gate_up", "down"):
        return
    grads, bounds = ref.gated_ffn_bwd(q["dout"], q["x"], q["w"], q["v"], kept.to(F64))
    names = ("dx", "dw_gate_up", "dw_down")
    for n, b, e in zip(names, grads, bounds):
        if product in ("dh", n):
            got = one_gradient(p, kept, n)
            ref.check(n, got, b, e)
            assert torch.equal(got, one_gradient(p, kept, n))


@pytest.mark.parametrize("part,name", [(p, n) for p in JOINT for n in JOINT[p]])
def test_products_of_one_launch(part, name):
    T, d, f = JOINT[part][name]
    print(f"gated {part} {name} T={T} d={d} f={f}", flush=True)
    got = moe.moe_gated_ffn_kernel("dx" if part == "gradients" else "dh", T, d, f, all=True)
    assert got == name or (name == "apart" and not got.startswith(("joint", "fused")))
    p = block(T, d, f)
    q = {n: t.to(F64) for n, t in p.items()}
    kept = moe.moe_gated_ffn(p["x"], p["w"], p["v"], save=True)[1]
    kw = dict(gate_up=kept) if part == "gradients" else {}
    got = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], **kw)
    want, bounds = ref.gated_ffn_bwd(q["dout"], q["x"], q["w"], q["v"],
                                     kept.to(F64) if kw else None)
    for n, a, b, e in zip(got._fields, got, want, bounds):
        ref.check(n, a, b, e)
    again = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    part = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], need_dx=False, **kw)
    for n, a, b, e in zip(got._fields[1:], part[1:], want[1:], bounds[1:]):
        ref.check(n, a, b, e)
    if kw:
        n = "dw_down"
        ref.check(n, one_gradient(p, kept, n), want[2], bounds[2])


@pytest.mark.parametrize("name", LINEAR)
def test_kernel_of_the_linear_map(name):
    T, N, K = LINEAR[name]
    print(f"linear_i8 {name} T={T} N={N} K={K}", flush=True)
    assert moe.moe_linear_i8_kernel(T, N, K) == name
    x, codes, scales, bias = linear(T, N, K)
    xq, xs = moe.moe_quantize_i8(x, group=0)
    want, e = ref.linear_i8(xq, xs, codes, scales, bias)
    for code, f32 in ((moe.MOE_OUT_F32, True), (moe.MOE_OUT_BF16, False)):
        got = moe.moe_linear_i8(x, codes, scales, bias, out_dtype=code)
        ref.check("out", got, want, ref.stored(want, e, f32))
        assert torch.equal(got, moe.moe_linear_i8(xq, codes, scales, bias, x_scales=xs,
                                                  out_dtype=code))


@pytest.mark.parametrize("K", [16, 1024, 9216, 131056])
@pytest.mark.parametrize("T", [1, 7, 8, 9, 15, 16, 17])
def test_few_tokens_and_long_rows(T, K):
    """Borders of the kernel for few tokens, whose rows come to the block a piece
    at a time where they are long; an N that leaves a block half empty."""
    N = 40
    print(f"linear_i8 T={T} N={N} K={K}", flush=True)
    x, codes, scales, bias = linear(T, N, K)
    xq, xs = moe.moe_quantize_i8(x, group=0)
    want, e = ref.linear_i8(xq, xs, codes, scales, bias)
    got = moe.moe_linear_i8(x, codes, scales, bias, out_dtype=moe.MOE_OUT_F32)
    ref.check("out", got, want, ref.stored(want, e, True))


@pytest.mark.parametrize("d,f", [(65536, 24), (24, 65536)])
@pytest.mark.parametrize("T", [1, 8, 16, 17, 70])
def test_longest_rows_of_the_block(T, d, f):
    print(f"gated T={T} d={d} f={f}", flush=True)
    p = block(T, d, f)
    q = {n: t.to(F64) for n, t in p.items()}
    want, bound, gu, egu = ref.gated_ffn(q["x"], q["w"], q["v"])
    out, kept = moe.moe_gated_ffn(p["x"], p["w"], p["v"], save=True)
    ref.check("out", out, want, bound)
    ref.check("gate_up", kept, gu, egu)
    got = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], gate_up=kept)
    grads, bounds = ref.gated_ffn_bwd(q["dout"], q["x"], q["w"], q["v"], kept.to(F64))
    for n, a, b, e in zip(got._fields, got, grads, bounds):
        ref.check(n, a, b, e)


def test_two_calls_at_once():
    """The same operators on two streams at once, with workspaces of their own,
    give what they give alone."""
    sizes = [(300, 1024, 512), (2501, 1024, 1032)]
    work, alone = [], []
    for i, (T, d, f) in enumerate(sizes):
        p, l = block(T, d, f, i), linear(T, f, d, i)
        work.append((p, l))

    def run(p, l, stream=None):
        out, kept = moe.moe_gated_ffn(p["x"], p["w"], p["v"], save=True, stream=stream)
        g = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], gate_up=kept, stream=stream)
        r = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], stream=stream)
        return [out, kept, *g, *r, moe.moe_linear_i8(*l, stream=stream)]

    for p, l in work:
        alone.append([t.clone() for t in run(p, l)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [[], []]
    for turn in range(3):
        for i, (p, l) in enumerate(work):
            got[i].append(run(p, l, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, alone[i]))


def test_two_graphs_of_one_workspace():
    """Two captured calls that share a workspace, replayed in turn: nothing is
    carried from one to the next."""
    p1, p2 = block(300, 1024, 512), block(70, 2048, 264, 5)
    need = max(moe.moe_gated_ffn_bwd_ws_bytes(300, 1024, 512),
               moe.moe_gated_ffn_bwd_ws_bytes(70, 2048, 264))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def run(p):
        return moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], ws=ws)

    want = [[t.clone() for t in run(p)] for p in (p1, p2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in (p1, p2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(p))
        graphs.append(g)
    for turn in range(3):
        for i in (0, 1, 1, 0):
            for t in outs[i]:
                t.fill_(7)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
