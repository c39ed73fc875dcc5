"""GPU tests of the gated feed-forward block, its gradient, and the run of them
with 8-bit checkpoints, against 64-bit definitions with derived bounds."""
import pytest
import torch

import i8_gated_ref as ref
import quantized_mixture_experts_fp32_amd as moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F64 = torch.bfloat16, torch.float64


def make(T, d, f, seed=0):
    g = torch.Generator().manual_seed(seed + T + d + f)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=n(T, d).to(BF16), w=(n(2 * f, d) * 2 * d ** -0.5).to(BF16),
                v=(n(d, f) * f ** -0.5).to(BF16), dout=n(T, d).to(BF16))


def behind(t, fill=float("nan")):
    """t on the GPU with `fill` in the memory after it."""
    room = torch.full((t.numel() + 65536,), fill, dtype=t.dtype, device=DEV)
    v = room[:t.numel()].view(t.shape)
    v.copy_(t)
    return v


def guarded(shape, dtype):
    """An output with room behind it, and what tells whether that was written."""
    n = 1
    for s in shape:
        n *= s
    room = torch.full((n + 4096,), 7.0, dtype=dtype, device=DEV)
    return room[:n].view(shape), lambda: bool((room[n:] == 7.0).all())


SIZES = [(1, 8, 8), (1, 2048, 1024), (2, 64, 24), (3, 136, 264), (16, 256, 128), (17, 520, 72),
         (33, 1032, 520), (64, 512, 256), (65, 256, 1032), (100, 2048, 512), (131, 264, 136),
         (300, 128, 640), (515, 1024, 264), (1030, 520, 512), (2304, 1536, 768)]


@pytest.mark.parametrize("T,d,f", SIZES)
def test_forward(T, d, f):
    print(f"gated_ffn T={T} d={d} f={f}", flush=True)
    p = make(T, d, f)
    q = {n: t.to(DEV).to(F64) for n, t in p.items()}
    for f32 in (False, True):
        want, bound, gu, egu = ref.gated_ffn(q["x"], q["w"], q["v"], f32)
        out, clean = guarded((T, d), torch.float32 if f32 else BF16)
        kept, clean_gu = guarded((T, 2 * f), BF16)
        code = moe.MOE_OUT_F32 if f32 else moe.MOE_OUT_BF16
        x, w, v = behind(p["x"]), behind(p["w"]), behind(p["v"])
        got, saved = moe.moe_gated_ffn(x, w, v, out=out, out_dtype=code, gate_up=kept)
        assert saved is kept and clean() and clean_gu()
        ref.check("out", got, want, bound)
        ref.check("gate_up", saved, gu, egu)
        again, none = moe.moe_gated_ffn(x, w, v, out_dtype=code)
        assert none is None and torch.equal(again, got)


@pytest.mark.parametrize("source", ["saved", "recompute", "checkpoint"])
@pytest.mark.parametrize("T,d,f", SIZES)
def test_gradient(T, d, f, source):
    print(f"gated_ffn_bwd T={T} d={d} f={f} {source}", flush=True)
    p = make(T, d, f)
    do_f32, dw_f32 = T % 2 == 0, d % 16 == 8
    dout = p["dout"].float() * 1.001 if do_f32 else p["dout"]
    x, w, v, kw = behind(p["x"]), behind(p["w"]), behind(p["v"]), {}
    x64, gu64 = x.to(F64), None
    if source == "saved":
        kw["gate_up"] = behind(moe.moe_gated_ffn(x, w, v, save=True)[1])
        gu64 = kw["gate_up"].to(F64)
    elif source == "checkpoint":
        x, kw["x_scales"] = moe.moe_quantize_i8(x)
        x64 = ref.restore(x, kw["x_scales"])
    code = moe.MOE_OUT_F32 if dw_f32 else moe.MOE_OUT_BF16
    dt = torch.float32 if dw_f32 else BF16
    dx, c1 = guarded((T, d), BF16)
    dw, c2 = guarded((2 * f, d), dt)
    dv, c3 = guarded((d, f), dt)
    got = moe.moe_gated_ffn_bwd(behind(dout), x, w, v, dw_dtype=code, dx=dx, dw_gate_up=dw,
                                dw_down=dv, **kw)
    assert c1() and c2() and c3()
    want, bounds = ref.gated_ffn_bwd(dout.to(DEV).to(F64), x64, w.to(F64), v.to(F64), gu64, do_f32,
                                     source == "checkpoint", dw_f32)
    for name, a, b, e in zip(got._fields, got, want, bounds):
        ref.check(name, a, b, e)
    part = moe.moe_gated_ffn_bwd(behind(dout), x, w, v, dw_dtype=code, need_dw=False, **kw)
    # (what is asked for chooses the kernels, so the order of the sums may differ; the
    # bounds hold for any order)
    assert part.dw_gate_up is None and part.dw_down is None
    ref.check("dx alone", part.dx, want[0], bounds[0])
    part = moe.moe_gated_ffn_bwd(behind(dout), x, w, v, dw_dtype=code, need_dx=False, **kw)
    assert part.dx is None
    ref.check("dw_gate_up alone", part.dw_gate_up, want[1], bounds[1])
    ref.check("dw_down alone", part.dw_down, want[2], bounds[2])


def test_no_tokens():
    p = make(4, 64, 24)
    w, v = p["w"].to(DEV), p["v"].to(DEV)
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    out, gu = moe.moe_gated_ffn(x, w, v, save=True)
    assert out.shape == (0, 64) and gu.shape == (0, 48)
    g = moe.moe_gated_ffn_bwd(x, x, w, v)
    assert g.dx.shape == (0, 64) and (g.dw_gate_up == 0).all() and (g.dw_down == 0).all()


@pytest.mark.parametrize("T", [3, 40, 200])
def test_rows_do_not_meet(T):
    """A token that is not finite touches its own rows of out, dx and gate_up
    alone."""
    d, f = 264, 136
    print(f"gated_ffn rows T={T}", flush=True)
    p = {n: t.to(DEV) for n, t in make(T, d, f).items()}
    clean, gu = moe.moe_gated_ffn(p["x"], p["w"], p["v"], save=True)
    dx = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"], need_dw=False).dx
    bad = p["x"].clone()
    bad[T // 2, 5] = float("nan")
    bad[T // 3, 5] = float("inf")
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[T // 2] = keep[T // 3] = False
    got, gu2 = moe.moe_gated_ffn(bad, p["w"], p["v"], save=True)
    assert torch.isnan(got[T // 2]).all()
    assert torch.equal(got[keep], clean[keep]) and torch.equal(gu2[keep], gu[keep])
    dx2 = moe.moe_gated_ffn_bwd(p["dout"], bad, p["w"], p["v"], need_dw=False).dx
    assert torch.isnan(dx2[T // 2]).all() and torch.equal(dx2[keep], dx[keep])


def test_far_gates():
    """Gates of +-60 to +-2000: silu is g or 0, its slope 1 or 0, nothing
    overflows into the result."""
    T, d, f = 24, 16, 32
    x = torch.zeros(T, d)
    x[:, 0] = torch.tensor([60., -60, 88, -88, 89, -89, 104, -104, 300, -300, 2000, -2000] * 2)
    x[:, 1] = torch.linspace(-2, 2, T)
    w = torch.zeros(2 * f, d)
    w[:f, 0] = 1.0
    w[f:, 1] = 1.0
    p = dict(x=x.to(BF16).to(DEV), w=w.to(BF16).to(DEV),
             v=make(T, d, f)["v"].to(DEV), dout=make(T, d, f)["dout"].to(DEV))
    q = {n: t.to(F64) for n, t in p.items()}
    out, _ = moe.moe_gated_ffn(p["x"], p["w"], p["v"])
    want, bound, _, _ = ref.gated_ffn(q["x"], q["w"], q["v"])
    ref.check("out", out, want, bound + 1e-36)
    got = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"])
    want, bounds = ref.gated_ffn_bwd(q["dout"], q["x"], q["w"], q["v"])
    for name, a, b, e in zip(got._fields, got, want, bounds):
        ref.check(name, a, b, e + 1e-30)


@pytest.mark.parametrize("T", [5, 96])
def test_gradient_against_differences(T):
    """<dout, out(p + e z) - out(p - e z)> / 2e against <grad, z> along random
    directions z, for x and both weights, with the 64-bit block."""
    d, f = 64, 48
    p = {n: t.to(DEV) for n, t in make(T, d, f).items()}
    q = {n: t.to(F64) for n, t in p.items()}
    got = moe.moe_gated_ffn_bwd(p["dout"], p["x"], p["w"], p["v"])
    _, bounds = ref.gated_ffn_bwd(q["dout"], q["x"], q["w"], q["v"])
    g = torch.Generator().manual_seed(T)

    def loss(x, w, v):
        gu = x @ w.t()
        return ((ref.silu(gu[:, :f]) * gu[:, f:]) @ v.t() * q["dout"]).sum()

    for i, n in enumerate("xwv"):
        z = torch.randn(q[n].shape, generator=g, dtype=F64).to(DEV)
        e = 1e-5
        args = [q["x"], q["w"], q["v"]]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + e * z, args[i] - e * z
        slope = (loss(*up) - loss(*down)) / (2 * e)
        mine = (got[i].to(F64) * z).sum()
        # third derivative over 6 e^2, and noise of 1e-16 of the loss' terms over e
        slack = (bounds[i] * z.abs()).sum() + 1e-6 * slope.abs() + 1e-6
        assert (mine - slope).abs() <= slack, (n, mine.item(), slope.item())


def train_step(block, residual, gain, dout):
    out, kept = block.forward_block(residual, gain, eps=1e-5)
    return (out, *block.backward_block(dout, kept, gain, eps=1e-5))


def step_inputs(T, d, f, dtype, seed=0):
    p = {n: t.to(DEV) for n, t in make(T, d, f, seed).items()}
    g = torch.Generator().manual_seed(seed)
    residual = (torch.randn(T, d, generator=g) * 2).to(dtype).to(DEV)
    gain = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    dout = torch.randn(T, d, generator=g).to(dtype).to(DEV)
    return moe.GatedFfn(p["w"], p["v"]), residual, gain, dout


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("T,d,f", [(1, 256, 128), (37, 520, 264), (300, 1024, 512)])
def test_block_with_checkpoint(T, d, f, dtype):
    """Norm, block, residual, and the gradient from an 8-bit checkpoint of the
    residual: against automatic differentiation in 64 bits at the restored
    residual.  Bounds on norms: n, g, u, dg, du, h, dx and the results are each
    rounded to bf16 once, and each of these roundings reaches a result through
    at most a factor 2 (norm, gate and residual): 16 of them."""
    print(f"block T={T} d={d} f={f} {dtype}", flush=True)
    block, residual, gain, dout = step_inputs(T, d, f, dtype)
    out, dres, dgain, dw, dv = train_step(block, residual, gain, dout)
    codes, scales = moe.moe_quantize_i8(residual)

    def forward(r, gn, w, v):
        n = r * (r.pow(2).mean(1, keepdim=True) + 1e-5).rsqrt() * gn
        gu = n @ w.t()
        return r + (ref.silu(gu[:, :f]) * gu[:, f:]) @ v.t()

    w, v = block.w_gate_up.to(F64), block.w_down.to(F64)
    want = forward(residual.to(F64), gain.to(F64), w, v)
    tol = 16 * 2 ** -8
    assert (out.to(F64) - want).norm() <= tol * want.norm()
    leaves = [t.clone().requires_grad_() for t in (ref.restore(codes, scales), gain.to(F64), w, v)]
    (forward(*leaves) * dout.to(F64)).sum().backward()
    assert dres.dtype == dtype and dgain.dtype == torch.float32
    for a, leaf in zip((dres, dgain, dw, dv), leaves):
        assert (a.to(F64) - leaf.grad).norm() <= tol * leaf.grad.norm()


def test_step_on_another_stream_and_in_a_graph():
    """A whole step: on a side stream, and recorded and replayed with other
    inputs and eager work between the replays; every result equals the eager
    one bit for bit.  Two graphs at once keep to their own workspaces."""
    T, d, f = 150, 512, 256
    block, residual, gain, dout = step_inputs(T, d, f, BF16)
    want = train_step(block, residual, gain, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, kept = block.forward_block(residual, gain, eps=1e-5, stream=side)
    got = (out, *block.backward_block(dout, kept, gain, eps=1e-5, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    graphs, results, inputs = [], [], []
    for seed in (1, 2):
        ins = step_inputs(T, d, f, BF16, seed)
        train_step(*ins)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = train_step(*ins)
        graphs.append(g)
        results.append(res)
        inputs.append(ins)
    for turn in range(3):
        for (block, residual, gain, dout), g in zip(inputs, graphs):
            residual.mul_(0.5 if turn else 1.0)
            g.replay()
        wants = [train_step(*ins) for ins in inputs]
        for res, want in zip(results, wants):
            assert all(torch.equal(a, b) for a, b in zip(res, want)), turn
        torch.cuda.synchronize()


def test_linear_i8_in_a_graph():
    T, N, K = 40, 520, 1024
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, K, generator=g).to(BF16).to(DEV)
    codes, scales = moe.moe_quantize_i8(torch.randn(N, K, generator=g).to(DEV), group=0)
    moe.moe_linear_i8(x, codes, scales)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.moe_linear_i8(x, codes, scales)
    for turn in range(3):
        x.add_(0.25)
        graph.replay()
        assert torch.equal(out, moe.moe_linear_i8(x, codes, scales)), turn
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_shared_expert_beside_the_routed_ones(dtype):
    """MoeLayer.forward_block(shared=...) equals the same block with the shared
    expert's output given as `add`."""
    T, d, f, E, k = 20, 256, 128, 8, 2
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    guc, gus = moe.moe_quantize_w4(n(E, 2 * f, d) * d ** -0.5)
    dnc, dns = moe.moe_quantize_w4(n(E, d, f) * f ** -0.5)
    layer = moe.MoeLayer((n(E, d) * d ** -0.5).to(BF16), None, k, f, guc, gus, dnc, dns)
    block, residual, gain, _ = step_inputs(T, d, f, dtype)
    x = moe.moe_rmsnorm(residual, gain, eps=1e-5)
    code = moe.MOE_OUT_F32 if dtype == torch.float32 else moe.MOE_OUT_BF16
    want = layer.forward_block(residual, gain, eps=1e-5, add=block.forward(x, out_dtype=code))[0]
    got = layer.forward_block(residual, gain, eps=1e-5, shared=block)[0]
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer.forward_block(residual, gain, eps=1e-5, shared=block, stream=side)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
