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


@pytest.mark.parametrize("source", ["saved", "recompute", "checkpoint"])
def test_offsets_beyond_32_bits(source):
    """More than 2^31 values of x, h, gate_up and their gradients: only the last
    rows hold anything, so an offset that wrapped would leave them wrong or the
    others not zero."""
    T, d, f, n = (1 << 21) + 77, 1032, 1032, 96
    print(f"gated T={T} d={d} f={f} {source}", flush=True)
    tail = block(n, d, f)
    full = lambda t: torch.zeros(T, d, dtype=BF16, device=DEV).index_copy_(  # noqa: E731
        0, torch.arange(T - n, T, device=DEV), t)
    x, dout, w, v = full(tail["x"]), full(tail["dout"]), tail["w"], tail["v"]
    q = {k: t.to(F64) for k, t in tail.items()}
    out, kept = moe.moe_gated_ffn(x, w, v, save=True)
    want, bound, gu, egu = ref.gated_ffn(q["x"], q["w"], q["v"])
    ref.check("out", out[-n:], want, bound)
    ref.check("gate_up", kept[-n:], gu, egu)
    assert not out[:-n].any() and not kept[:-n].any()
    del out
    kw, x64, gu64 = {}, q["x"], None
    if source == "saved":
        kw["gate_up"], gu64 = kept, kept[-n:].to(F64)
    else:
        del kept
    if source == "checkpoint":
        x, kw["x_scales"] = moe.moe_quantize_i8(x)
        x64 = ref.restore(x[-n:], kw["x_scales"][-n:])
    got = moe.moe_gated_ffn_bwd(dout, x, w, v, **kw)
    want, bounds = ref.gated_ffn_bwd(q["dout"], x64, q["w"], q["v"], gu64,
                                     x_rounded=source == "checkpoint")
    # (the weights' sums run over all tokens: as many more roundings, of zeros)
    for name, a, b, e in zip(got._fields, got, want, bounds):
        ref.check(name, a[-n:] if name == "dx" else a, b, e)
    assert not got.dx[:-n].any()


def test_linear_offsets_beyond_32_bits():
    T, N, K, n = (1 << 20) + 33, 2056, 64, 70
    print(f"linear_i8 T={T} N={N} K={K}", flush=True)
    tail, codes, scales, _ = linear(n, N, K)
    x = torch.zeros(T, K, dtype=BF16, device=DEV)
    x[-n:] = tail
    xq, xs = moe.moe_quantize_i8(tail, group=0)
    want, e = ref.linear_i8(xq, xs, codes, scales, None)
    got = moe.moe_linear_i8(x, codes, scales, out_dtype=moe.MOE_OUT_F32)
    ref.check("out", got[-n:], want, ref.stored(want, e, True))
    assert not got[:-n].any()


@pytest.mark.parametrize("T", [3, 40])
def test_weights_beyond_32_bits(T):
    """The largest weights that the call takes, zeros but for the first and last
    features."""
    d = f = 65536
    print(f"gated T={T} d={d} f={f}", flush=True)
    g = torch.Generator(DEV).manual_seed(T)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    live = torch.cat((torch.arange(0, 8, device=DEV), torch.arange(f - 8, f, device=DEV)))
    both = torch.cat((live, f + live))  # rows of w_gate_up
    w = torch.zeros(2 * f, d, dtype=BF16, device=DEV)
    w[both] = n(32, d) * 2 * d ** -0.5
    v = torch.zeros(d, f, dtype=BF16, device=DEV)
    v[live] = n(16, f)
    x, dout = n(T, d), n(T, d)
    out, kept = moe.moe_gated_ffn(x, w, v, save=True)
    # the features that hold something, as a block of 16 features and 16 outputs
    xs, ws = x.to(F64), w[both].to(F64)
    vs = v[live][:, live].to(F64)
    want, bound, gu, egu = ref.gated_ffn(xs, ws, vs)
    ref.check("gate_up", kept[:, both], gu, egu)
    ref.check("out", out[:, live], want, bound)
    rest = torch.ones(d, dtype=torch.bool, device=DEV)
    rest[live] = False
    assert not out[:, rest].any() and not kept[:, :f][:, rest].any()
    got = moe.moe_gated_ffn_bwd(dout, x, w, v, gate_up=kept)
    # dout meets v's live rows only; dh of a feature that holds nothing gives no dx
    # and, as its g and u are 0, no weight gradient
    ds = dout[:, live].to(F64)
    grads, bounds = ref.gated_ffn_bwd(ds, xs, ws, vs, kept[:, both].to(F64))
    ref.check("dx", got.dx, grads[0], bounds[0])
    ref.check("dw_gate_up", got.dw_gate_up[both], grads[1], bounds[1])
    assert not got.dw_gate_up[8:f - 8].any() and not got.dw_gate_up[f + 8:2 * f - 8].any()
    ref.check("dw_down", got.dw_down[live][:, live], grads[2], bounds[2])
    assert not got.dw_down[:, rest].any()
