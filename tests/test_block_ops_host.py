"""CPU tests of the operators around the routed experts: the 64-bit
definitions the GPU tests compare with against automatic differentiation and
differences, and the argument checks of the C ABI and of the binding (every
call here is refused before any HIP call)."""
import ctypes
import os

import pytest
import torch

import block_ref as ref
import quantized_mixture_experts_fp32_amd as moe
from layer_data import w4_untile

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
NULL = None
INV, UNS, WSP, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE,
                     moe.MOE_OK)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from quantized_mixture_experts_fp32_amd import build
        build.build()
    return moe.load_library()


# ------------------------------------------------------------- the definitions
def case(gate, post, add, k=3, T=5, d=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    pos = torch.randperm(T * k, generator=g).to(torch.int32)
    pos[2], pos[T * k - 1] = -1, T * k + 3
    p = dict(res=n(T, d), y=n(T * k, d), w=torch.softmax(n(T, k), 1))
    p["add"] = n(T, d) if add else None
    p["post"] = 1 + 0.3 * n(d) if post else None
    p["gate"] = {"none": torch.ones(1, 1, dtype=torch.float64), "token": n(T, 1),
                 "channel": n(1, d)}[gate]
    return p, pos, n(T, d)


@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("add", [True, False])
def test_block_gradient_definition(gate, post, add):
    """The closed-form gradients equal automatic differentiation's, and both
    agree with central differences (h = 1e-6: 1e-10 of noise over h)."""
    p, pos, dout = case(gate, post, add)
    leaves = {n: t.clone().requires_grad_() for n, t in p.items() if t is not None}
    full = {n: leaves.get(n) for n in p}

    def forward(q):
        return ref.combine_residual(q["res"], q["y"], pos, q["w"], q["add"], q["post"], q["gate"],
                                    0.6, 1e-3, None)[0]

    (forward(full) * dout).sum().backward()
    r = ref.combine_residual_bwd(dout, p["y"], pos, p["w"], p["add"], p["post"], p["gate"], 1e-3)
    T, k = p["w"].shape
    live = (pos >= 0) & (pos < T * k)
    dy = torch.zeros_like(p["y"])
    dy[pos[live].long()] = r["dy"][0].reshape(T * k, -1)[live]
    mine = dict(res=0.6 * dout, y=dy, w=r["dw"][0], add=r["do"][0], post=r["dpost"][0])
    mine["gate"] = {"none": None, "token": r["dgate_t"][0][:, None],
                    "channel": r["dgate_c"][0][None]}[gate]
    g = torch.Generator().manual_seed(4)
    for name, leaf in leaves.items():
        if mine[name] is None:
            continue
        assert torch.allclose(leaf.grad, mine[name], rtol=1e-11, atol=1e-12), name
        v = torch.randn(leaf.shape, generator=g, dtype=torch.float64)
        h = 1e-6
        plus, minus = dict(p), dict(p)
        plus[name], minus[name] = p[name] + h * v, p[name] - h * v
        num = float(((forward(plus) - forward(minus)) * dout).sum()) / (2 * h)
        assert abs(num - float((leaf.grad * v).sum())) <= 1e-7 * (1 + abs(num)), name


def test_norm_gradient_definition():
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, gain, dout, dres = n(4, 24).requires_grad_(), n(24).requires_grad_(), n(4, 24), n(4, 24)
    ((ref.rmsnorm(x, gain, 1e-4) * dout).sum() + (x * dres).sum()).backward()
    dx, _, dgain, _ = ref.rmsnorm_bwd(dout, x.detach(), gain.detach(), dres, 1e-4)
    assert torch.allclose(dx, x.grad, rtol=1e-11) and torch.allclose(dgain, gain.grad, rtol=1e-11)
    assert torch.autograd.gradcheck(lambda a, b: ref.rmsnorm(a, b, 1e-4), (x, gain))


def test_linear_definition_unpacks_the_tiled_codes():
    import numpy as np
    N, K = 32, 384
    g = torch.Generator().manual_seed(2)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.rand(N, K // 128, generator=g).to(torch.float16)
    W = ref.dequantize_w4(codes, scales.view(torch.int16))
    rm = w4_untile(codes.numpy().reshape(-1), N, K)
    q = np.stack([rm & 15, rm >> 4], -1).reshape(N, K).astype(np.int64)
    q = np.where(q > 7, q - 16, q)
    want = q * np.repeat(scales.double().numpy(), 128, 1)
    assert np.array_equal(W.numpy(), want)


# ---------------------------------------------------------------- C ABI refusals
def test_linear_refusals(lib):
    def f(x=FAKE, T=4, N=32, K=256, group=128, c=FAKE, s=FAKE, b=NULL, out=FAKE, dt=0, ws=FAKE,
          wsb=1 << 40):
        return lib.moe_linear_w4(x, T, N, K, group, c, s, b, out, dt, ws, wsb, NULL)
    assert f(K=200) == UNS and f(N=24) == UNS and f(group=64) == UNS
    assert f(T=-1) == INV and f(N=0) == INV and f(K=0) == INV and f(dt=2) == INV
    assert f(T=1 << 30, K=1 << 20) == UNS and f(T=1 << 30, N=1 << 20) == UNS
    assert f(T=1 << 17, K=1 << 17) == UNS and f(T=1 << 17, N=1 << 17) == UNS  # 2^34
    assert f(T=1 << 23, K=128, N=16) == UNS and f(T=1, K=128, N=1 << 28) == UNS
    for name in ("x", "c", "s", "out"):
        assert f(**{name: NULL}) == INV
    for name in ("x", "c", "out"):
        assert f(**{name: ODD}) == INV
    assert f(b=ODD) == INV and f(s=ODD) == INV
    assert f(T=0, x=NULL, c=NULL, s=NULL, out=NULL, ws=NULL, wsb=0) == OK
    for T, N, K in ((4, 32, 256), (1, 2048, 2048), (64, 4096, 4096), (2000, 4096, 4096)):
        need = lib.moe_linear_w4_ws_bytes(T, N, K)
        if need:
            assert f(T=T, N=N, K=K, wsb=need - 1) == WSP and f(T=T, N=N, K=K, ws=NULL) == WSP
            assert f(T=T, N=N, K=K, ws=ctypes.c_void_p(0x10010)) == INV
    assert lib.moe_linear_w4_ws_bytes(-1, 16, 128) == 0
    for N, K in ((16, 128), (50304, 4096), (4096, 14336)):
        assert lib.moe_linear_w4_ws_bytes(0, N, K) == 0
        assert all(lib.moe_linear_w4_ws_bytes(T, N, K) == 0 for T in range(65))
    for T, N, K in ((1, 1, 1), (100, 8, 100), ((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1)):
        lib.moe_linear_w4_ws_bytes(T, N, K)     # refused sizes are priced all the same


def test_norm_refusals(lib):
    def f(x=FAKE, xd=0, g=FAKE, T=4, d=64, eps=1e-6, out=FAKE, od=0):
        return lib.moe_rmsnorm(x, xd, g, T, d, eps, out, od, NULL)
    assert f(d=60) == UNS and f(d=8200) == UNS and f(d=0) == INV and f(T=-1) == INV
    assert f(T=1 << 23) == UNS
    assert f(xd=2) == INV and f(od=-1) == INV
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert f(eps=eps) == INV
    assert f(x=NULL) == INV and f(out=NULL) == INV
    assert f(x=ODD) == INV and f(out=ODD) == INV and f(g=ODD) == INV
    assert f(T=0, x=NULL, out=NULL) == OK

    def b(do=FAKE, dd=0, x=FAKE, xd=0, g=FAKE, dres=NULL, T=4, d=64, eps=1e-6, dx=FAKE, dg=FAKE,
          ws=FAKE, wsb=1 << 30):
        return lib.moe_rmsnorm_bwd(do, dd, x, xd, g, dres, T, d, eps, dx, dg, ws, wsb, NULL)
    need = lib.moe_rmsnorm_bwd_ws_bytes(4, 64)
    assert need >= 64 * 4
    assert b(wsb=need - 1) == WSP and b(ws=NULL) == WSP and b(ws=ODD) == INV
    assert b(do=NULL) == INV and b(x=NULL) == INV and b(dx=NULL) == INV
    assert b(dres=ODD) == INV and b(dg=ODD) == INV and b(dd=3) == INV and b(d=12) == UNS
    assert b(eps=0.0) == INV
    assert b(T=0, do=NULL, x=NULL, dx=NULL, dg=NULL, ws=NULL, wsb=0) == OK


def test_block_refusals(lib):
    def f(res=FAKE, dt=0, y=FAKE, pos=FAKE, w=FAKE, k=2, add=NULL, post=NULL, gate=NULL, mode=0,
          scale=1.0, eps=1e-6, ng=NULL, T=4, d=64, out=FAKE, nxt=NULL):
        return lib.moe_combine_residual(res, dt, y, pos, w, k, add, post, gate, mode, scale, eps,
                                        ng, T, d, out, nxt, NULL)
    assert f(d=12) == UNS and f(d=8200) == UNS and f(k=17) == UNS and f(k=-1) == INV
    assert f(T=1 << 30, k=2) == UNS
    assert f(dt=2) == INV and f(eps=0.0) == INV and f(scale=float("nan")) == INV
    assert f(scale=float("inf")) == INV
    assert f(mode=3) == INV and f(mode=1) == INV and f(mode=2) == INV and f(gate=FAKE) == INV
    assert f(y=NULL) == INV and f(pos=NULL) == INV and f(w=NULL) == INV
    assert f(k=0) == INV                               # pairs with k = 0
    assert f(k=0, y=NULL, pos=NULL, w=NULL) == INV     # neither pairs nor add
    assert f(res=NULL) == INV and f(out=NULL) == INV and f(ng=FAKE) == INV
    for name in ("res", "y", "add", "post", "out", "nxt"):
        assert f(**{name: ODD}) == INV, name
    assert f(ng=ODD, nxt=FAKE) == INV
    assert f(gate=ctypes.c_void_p(0x10004), mode=2) == INV
    assert f(T=0, res=NULL, y=NULL, pos=NULL, w=NULL, out=NULL) == OK

    def b(do=FAKE, dt=0, y=FAKE, pos=FAKE, w=FAKE, k=2, add=NULL, post=NULL, gate=NULL, mode=0,
          scale=1.0, eps=1e-6, T=4, d=64, dy=FAKE, dyd=0, dw=FAKE, dadd=NULL, dres=NULL,
          dpost=NULL, dgate=NULL, ws=NULL, wsb=0):
        return lib.moe_combine_residual_bwd(do, dt, y, pos, w, k, add, post, gate, mode, scale,
                                            eps, T, d, dy, dyd, dw, dadd, dres, dpost, dgate, ws,
                                            wsb, NULL)
    need = lib.moe_combine_residual_bwd_ws_bytes(4, 64)
    assert b(post=FAKE, dpost=FAKE) == WSP
    assert b(post=FAKE, dpost=FAKE, ws=FAKE, wsb=need - 1) == WSP
    assert b(gate=FAKE, mode=2, dgate=FAKE) == WSP
    assert b(dpost=FAKE, ws=FAKE, wsb=1 << 30) == INV      # no post norm
    assert b(dgate=FAKE) == INV and b(dadd=FAKE) == INV    # no gate, no add
    assert b(k=0, y=NULL, pos=NULL, w=NULL, add=FAKE) == INV
    assert b(do=NULL) == INV and b(dyd=5) == INV and b(dt=5) == INV
    assert b(dy=ODD) == INV and b(dres=ODD) == INV and b(dw=ODD) == INV
    assert b(T=0, do=NULL, y=NULL, pos=NULL, w=NULL) == OK


def test_sort_refusals(lib):
    def f(x=FAKE, dt=0, pos=FAKE, w=NULL, T=4, k=2, d=64, xs=FAKE):
        return lib.moe_dispatch(x, dt, pos, w, T, k, d, xs, NULL)
    assert f(k=0) == INV and f(k=17) == UNS and f(d=20) == UNS and f(dt=2) == INV
    assert f(T=-1) == INV and f(d=8200) == UNS
    assert f(x=NULL) == INV and f(pos=NULL) == INV and f(xs=NULL) == INV
    assert f(x=ODD) == INV and f(xs=ODD) == INV and f(w=ODD) == INV
    assert f(T=0, x=NULL, pos=NULL, xs=NULL) == OK

    def b(g=FAKE, dt=0, x=NULL, pos=FAKE, w=NULL, T=4, k=2, d=64, dx=FAKE, dw=NULL):
        return lib.moe_dispatch_bwd(g, dt, x, pos, w, T, k, d, dx, dw, NULL)
    assert b(dw=FAKE) == INV and b(dw=FAKE, x=FAKE) == INV and b(dw=FAKE, w=FAKE) == INV
    assert b(g=NULL) == INV and b(dx=NULL) == INV and b(pos=NULL) == INV and b(dx=ODD) == INV
    assert b(k=0) == INV and b(d=4) == UNS
    assert b(T=0, g=NULL, pos=NULL, dx=NULL) == OK

    def c(do=FAKE, dd=0, y=FAKE, pos=FAKE, w=FAKE, T=4, k=2, d=64, dy=FAKE, dyd=0, dw=FAKE):
        return lib.moe_combine_bwd(do, dd, y, pos, w, T, k, d, dy, dyd, dw, NULL)
    assert c(do=NULL) == INV and c(y=NULL) == INV and c(w=NULL) == INV and c(pos=NULL) == INV
    assert c(dd=2) == INV and c(dyd=2) == INV and c(dy=ODD) == INV and c(k=17) == UNS
    assert c(dy=NULL, dw=NULL) == OK and c(T=0, do=NULL) == OK


# --------------------------------------------------------------- binding refusals
def test_binding_refusals():
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    x, gain = z(4, 64), z(64)
    pos, w, y = z(8, dtype=torch.int32), z(4, 2), z(8, 64)

    def refused(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    refused("a tensor is needed", moe.moe_rmsnorm, None)
    refused("x must be", moe.moe_rmsnorm, gain)
    refused("expected a GPU", moe.moe_rmsnorm, x, gain)
    refused("float64", moe.moe_rmsnorm, x.double())
    refused("contiguous", moe.moe_rmsnorm, z(64, 4).t())
    for shape in ((2 ** 32 + 5, 8), (1, 2 ** 32 + 8)):  # an int of 32 bits would wrap
        refused("below 2", moe.moe_rmsnorm, torch.empty(shape, device="meta"))
    refused("dout must be", moe.moe_rmsnorm_bwd, gain, x)
    refused("expected a GPU", moe.moe_rmsnorm_bwd, x, x, gain)
    refused("x must be", moe.moe_linear_w4, gain, z(16, 32, dtype=torch.uint8), z(16, 1))
    refused("float32", moe.moe_linear_w4, x, z(16, 32, dtype=torch.uint8), z(16, 1))
    refused("expected a GPU", moe.moe_linear_w4, z(4, 128, dtype=torch.bfloat16),
            z(16, 64, dtype=torch.uint8), z(16, 1, dtype=torch.int16))
    refused("must be", moe.moe_combine_residual, gain)
    refused("expected a GPU", moe.moe_combine_residual, x, y, pos, w)
    refused("expected a GPU", moe.moe_combine_residual_bwd, x, y, pos, w)
    refused("expected a GPU", moe.moe_dispatch, x, pos, 2)
    refused("must be", moe.moe_dispatch_bwd, z(7, 64), pos, 2)
    refused("must be", moe.moe_dispatch_bwd, y, pos, 0)
    refused("must be", moe.moe_combine_bwd, x, y, pos, gain)


def test_block_layer_refusals():
    """forward_block checks the residual before it allocates or launches: the
    router reads its weights by the residual's width."""
    wr = torch.zeros(8, 128)
    layer = moe.MoeLayer(wr, None, 2, 128, None, None, None, None)
    for bad in (torch.zeros(4, 256), torch.zeros(4, 64), torch.zeros(128)):
        with pytest.raises(ValueError, match="expected .T..128."):
            layer.forward_block(bad)
    with pytest.raises(ValueError, match="residual is on meta"):
        layer.forward_block(torch.empty(4, 128, device="meta"))
    with pytest.raises(ValueError, match="expected a GPU"):
        layer.forward_block(torch.zeros(4, 128))
