"""CPU tests of the 8-bit rows, the 8-bit linear map and the gated block: the
definitions that the GPU tests compare with, and the refusals of the C ABI and
of the binding (every call here is refused before any HIP call)."""
import ctypes
import inspect
import os

import numpy as np
import pytest
import torch

import i8_gated_ref as ref
import quantized_mixture_experts_fp32_amd as moe
from i8_gated_sizes import GATED, JOINT, LINEAR

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
NULL = None
INV, UNS, WSP, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE,
                     moe.MOE_OK)
F64 = torch.float64


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from quantized_mixture_experts_fp32_amd import build
        build.build()
    return moe.load_library()


# ------------------------------------------------------------- the definitions
@pytest.mark.parametrize("kept", [True, False])
def test_gated_gradient_definition(kept):
    """The closed form equals automatic differentiation's."""
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    T, d, f = 5, 16, 24
    x, w, v, dout = n(T, d), n(2 * f, d), n(d, f), n(T, d)
    leaves = [t.clone().requires_grad_() for t in (x, w, v)]
    gu = leaves[0] @ leaves[1].t()
    ((ref.silu(gu[:, :f]) * gu[:, f:]) @ leaves[2].t() * dout).sum().backward()
    got, bounds = ref.gated_ffn_bwd(dout, x, w, v, gu.detach() if kept else None)
    for a, leaf, e in zip(got, leaves, bounds):
        assert torch.allclose(a, leaf.grad, rtol=1e-11, atol=1e-11) and (e >= 0).all()


def test_quantize_definition():
    """Restored values are within half a step, the largest value of a group is
    +-127 steps, and the codes use the whole range."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 300)) * 10.0 ** rng.uniform(-20, 20, (40, 1))).astype(np.float32)
    for group in (128, 0):
        codes, scales = ref.quantize(x, group)
        back = ref.restore(torch.from_numpy(codes), torch.from_numpy(scales)).numpy()
        s = scales[:, None] if group == 0 else np.repeat(scales, 128, 1)[:, :300]
        # half a step, and three roundings of 2^-24 each on values up to 127 steps
        assert (np.abs(back - x) <= s * (0.5 + 3 * 127 * 2.0 ** -24)).all()
        assert np.abs(codes).max() == 127
        top = [np.abs(codes[:, i:i + (group or 300)]).max(1) for i in range(0, 300, group or 300)]
        assert (np.stack(top) == 127).all()


# ---------------------------------------------------------- refusals, C ABI
def test_rows_refusals(lib):
    def q(x=FAKE, dt=0, T=4, K=256, group=128, c=FAKE, s=FAKE):
        return lib.moe_quantize_i8(x, dt, T, K, group, c, s, NULL)

    def r(c=FAKE, s=FAKE, T=4, K=256, group=128, out=FAKE, dt=0):
        return lib.moe_dequantize_i8(c, s, T, K, group, out, dt, NULL)

    for fn in (q, r):
        assert fn(T=-1) == INV and fn(K=0) == INV and fn(dt=2) == INV
        assert fn(K=100) == UNS and fn(K=1 << 20) == UNS and fn(T=1 << 23) == UNS
        assert fn(T=1 << 20, K=1 << 14) == UNS
        assert fn(group=64) == UNS and fn(group=-1) == UNS
        assert fn(c=NULL) == INV and fn(s=NULL) == INV and fn(c=ODD) == INV and fn(s=ODD) == INV
        assert fn(T=0, c=NULL, s=NULL) == OK
    assert q(x=NULL) == INV and q(x=ODD) == INV and r(out=NULL) == INV and r(out=ODD) == INV


def test_norm_refusals(lib):
    def n(c=FAKE, s=FAKE, g=NULL, T=4, d=256, eps=1e-5, out=FAKE, dt=0):
        return lib.moe_rmsnorm_i8(c, s, g, T, d, eps, out, dt, NULL)

    def b(do=FAKE, dt=0, c=FAKE, s=FAKE, g=NULL, dres=NULL, T=4, d=256, eps=1e-5, dx=FAKE, xdt=0,
          dg=NULL, ws=NULL, wsb=0):
        return lib.moe_rmsnorm_bwd_i8(do, dt, c, s, g, dres, T, d, eps, dx, xdt, dg, ws, wsb, NULL)

    for fn in (n, b):
        assert fn(T=-1) == INV and fn(d=100) == UNS and fn(d=8200) == UNS and fn(T=1 << 23) == UNS
        assert fn(eps=0.0) == INV and fn(eps=float("nan")) == INV and fn(dt=3) == INV
        assert fn(c=NULL) == INV and fn(s=NULL) == INV and fn(c=ODD) == INV and fn(s=ODD) == INV
        assert fn(g=ODD) == INV and fn(T=0, c=NULL, s=NULL) == OK
    assert n(out=NULL) == INV and n(out=ODD) == INV
    assert b(do=NULL) == INV and b(dx=NULL) == INV and b(dres=ODD) == INV and b(xdt=2) == INV
    need = lib.moe_rmsnorm_bwd_ws_bytes(4, 256)
    assert b(g=FAKE, dg=FAKE, ws=FAKE, wsb=need - 1) == WSP
    assert b(g=FAKE, dg=FAKE, ws=ctypes.c_void_p(0x10008), wsb=need) == INV


def test_linear_refusals(lib):
    def f(x=FAKE, sx=NULL, T=4, N=64, K=256, c=FAKE, s=FAKE, b=NULL, out=FAKE, dt=0, ws=FAKE,
          wsb=1 << 40):
        return lib.moe_linear_i8(x, sx, T, N, K, c, s, b, out, dt, ws, wsb, NULL)

    assert f(T=-1) == INV and f(N=0) == INV and f(K=0) == INV and f(dt=7) == INV
    assert f(K=24) == UNS and f(N=12) == UNS and f(K=1 << 17) == UNS
    assert f(T=1 << 23) == UNS and f(N=1 << 28) == UNS
    assert f(T=1 << 22, K=1 << 12) == UNS and f(T=1 << 22, N=1 << 12) == UNS
    for name in ("x", "c", "s", "out"):
        assert f(**{name: NULL}) == INV and f(**{name: ODD}) == INV
    assert f(sx=ODD) == INV and f(b=ODD) == INV
    need = lib.moe_linear_i8_ws_bytes(400, 64, 256, 0)
    assert need >= 400 * 256 + 1600 and lib.moe_linear_i8_ws_bytes(0, 64, 256, 0) == 0
    assert lib.moe_linear_i8_ws_bytes(400, 64, 24, 0) == 0
    assert f(T=400, wsb=need - 1) == WSP and f(T=400, ws=NULL) == WSP
    assert f(T=400, ws=ctypes.c_void_p(0x10010)) == INV
    assert f(T=0, x=NULL, c=NULL, s=NULL, out=NULL, ws=NULL, wsb=0) == OK


def test_gated_refusals(lib):
    def f(x=FAKE, w=FAKE, v=FAKE, T=4, d=256, f=128, out=FAKE, dt=0, gu=NULL, ws=FAKE,
          wsb=1 << 40):
        return lib.moe_gated_ffn(x, w, v, T, d, f, out, dt, gu, ws, wsb, NULL)

    def b(do=FAKE, dt=0, x=FAKE, sx=NULL, gu=NULL, w=FAKE, v=FAKE, T=4, d=256, f=128, dx=FAKE,
          dw=FAKE, dv=FAKE, wdt=0, ws=FAKE, wsb=1 << 40):
        return lib.moe_gated_ffn_bwd(do, dt, x, sx, gu, w, v, T, d, f, dx, dw, dv, wdt, ws, wsb,
                                     NULL)

    for fn in (f, b):
        assert fn(T=-1) == INV and fn(d=0) == INV and fn(f=-8) == INV and fn(dt=2) == INV
        assert fn(d=100) == UNS and fn(f=100) == UNS and fn(d=65544) == UNS and fn(f=65544) == UNS
        assert fn(T=1 << 23) == UNS and fn(T=1 << 22, d=4096) == UNS and fn(T=1 << 22, f=2048) == UNS
        for name in ("x", "w", "v"):
            assert fn(**{name: NULL}) == INV and fn(**{name: ODD}) == INV
        assert fn(gu=ODD) == INV and fn(ws=NULL) == WSP and fn(ws=ctypes.c_void_p(0x10010)) == INV
    assert f(out=NULL) == INV and f(out=ODD) == INV
    assert b(do=NULL) == INV and b(sx=ODD) == INV and b(wdt=2) == INV
    for name in ("dx", "dw", "dv"):
        assert b(**{name: ODD}) == INV
    need = lib.moe_gated_ffn_ws_bytes(4, 256, 128)
    assert need >= 4 * 128 * 2 and f(wsb=need - 1) == WSP
    assert lib.moe_gated_ffn_ws_bytes(0, 256, 128) == 0 == lib.moe_gated_ffn_ws_bytes(4, 100, 128)
    for args in ((0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        n = lib.moe_gated_ffn_bwd_ws_bytes(4, 256, 128, *args)
        kw = dict(dt=args[0], sx=FAKE if args[1] else NULL, gu=FAKE if args[2] else NULL)
        assert n > 0 and b(wsb=n - 1, **kw) == WSP
    assert f(T=0, x=NULL, w=NULL, v=NULL, out=NULL, ws=NULL, wsb=0) == OK
    assert b(T=0, do=NULL, x=NULL, w=NULL, v=NULL, dw=NULL, dv=NULL, ws=NULL, wsb=0) == OK
    assert b(dx=NULL, dw=NULL, dv=NULL, do=NULL) == OK  # nothing wanted


# ---------------------------------------------------------- refusals, binding
CALLS = ("moe_quantize_i8", "moe_dequantize_i8", "moe_linear_i8", "moe_gated_ffn",
         "moe_gated_ffn_bwd")
BF = torch.bfloat16


def inputs(name, **change):
    T, d, f = 4, 128, 16
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    i8, f32 = torch.int8, torch.float32
    p = {
        "moe_quantize_i8": dict(x=z(T, d)),
        "moe_dequantize_i8": dict(codes=z(T, d, dt=i8), scales=z(T, 1, dt=f32)),
        "moe_linear_i8": dict(x=z(T, d), codes=z(f, d, dt=i8), scales=z(f, dt=f32)),
        "moe_gated_ffn": dict(x=z(T, d), w_gate_up=z(2 * f, d), w_down=z(d, f)),
        "moe_gated_ffn_bwd": dict(dout=z(T, d), x=z(T, d), w_gate_up=z(2 * f, d), w_down=z(d, f)),
    }[name]
    return {**p, **change}


@pytest.mark.parametrize("name", CALLS)
def test_binding_names_and_device(name):
    call = getattr(moe, name)
    sig = inspect.signature(call)
    lead = next(iter(sig.parameters))
    assert sig.parameters["stream"].kind is inspect.Parameter.KEYWORD_ONLY
    with pytest.raises(ValueError, match="expected a GPU"):
        call(**inputs(name))
    with pytest.raises(TypeError, match=f"'{lead}'"):
        call()
    with pytest.raises(ValueError, match="a tensor is needed"):
        call(**inputs(name, **{lead: None}))


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU: gets past the device check of a
    call that is refused for something else."""
    is_cuda = True

    def get_device(self):
        return 0


def gpu(t):
    return t.as_subclass(OnGpu)


@pytest.mark.parametrize("name,bad,what", [
    ("moe_quantize_i8", dict(x=torch.zeros(4, 128, dtype=torch.float16)), "float16"),
    ("moe_quantize_i8", dict(x=torch.zeros(128, dtype=BF)), r"\[T\]\[K\]"),
    ("moe_quantize_i8", dict(x=torch.zeros(128, 4, dtype=BF).t()), "contiguous"),
    ("moe_dequantize_i8", dict(codes=torch.zeros(4, 128, dtype=torch.uint8)), "uint8"),
    ("moe_dequantize_i8", dict(codes=torch.zeros(4, 136, dtype=torch.int8)), "shape"),
    ("moe_linear_i8", dict(x=torch.zeros(4, 128)), "float32"),
    ("moe_linear_i8", dict(x=torch.zeros(4, 120, dtype=BF)), "shape"),
    ("moe_gated_ffn", dict(x=torch.zeros(4, 128)), "float32"),
    ("moe_gated_ffn", dict(x=torch.zeros(4, 120, dtype=BF)), "shape"),
    ("moe_gated_ffn_bwd", dict(dout=torch.zeros(4, 120, dtype=BF)), "shape"),
    ("moe_gated_ffn_bwd", dict(dout=torch.zeros(4, 128, dtype=torch.float16)), "float16"),
])
def test_binding_refuses(name, bad, what):
    args = {n: gpu(t) for n, t in inputs(name, **bad).items()}
    with pytest.raises(ValueError, match=what), torch.no_grad():
        inspect.unwrap(getattr(moe, name))(**args)


def test_layer_refuses_two_adds():
    layer = moe.MoeLayer.__new__(moe.MoeLayer)
    layer.d, layer.wr = 128, torch.zeros(8, 128)
    with pytest.raises(ValueError, match="shared and add"):
        layer.forward_block(torch.zeros(4, 128), add=torch.zeros(4, 128), shared=object())


# ------------------------------------------------------------ the kernels' names
@pytest.mark.parametrize("product,name", [(p, n) for p in GATED for n in GATED[p]])
def test_kernel_of_the_block(lib, product, name):
    assert moe.moe_gated_ffn_kernel(product, *GATED[product][name]) == name


@pytest.mark.parametrize("name", LINEAR)
def test_kernel_of_the_linear_map(lib, name):
    assert moe.moe_linear_i8_kernel(*LINEAR[name]) == name


def test_no_other_kernel_is_chosen(lib):
    """Over many sizes, every choice is one that a GPU test reaches."""
    rng = np.random.default_rng(5)
    for T, d, f in np.exp2(rng.uniform(0, [14, 13, 13], (3000, 3))).astype(int).tolist():
        d, f = -(-d // 8) * 8, -(-f // 8) * 8
        for p in GATED:
            assert moe.moe_gated_ffn_kernel(p, T, d, f) in GATED[p], (p, T, d, f)
        for p, joint in (("dx", "gradients"), ("dh", "recompute")):
            name = moe.moe_gated_ffn_kernel(p, T, d, f, all=True)
            assert name in JOINT[joint] or not name.startswith(("joint", "fused")), (
                p, T, d, f)
        assert moe.moe_linear_i8_kernel(T, 4 * d, 2 * f) in LINEAR, (T, d, f)


def test_no_kernel(lib):
    assert moe.moe_linear_i8_kernel(0, 64, 64) == "" == moe.moe_linear_i8_kernel(4, 64, 8)
    assert moe.moe_gated_ffn_kernel("dx", 0, 64, 64) == ""
    assert moe.moe_gated_ffn_kernel("dx", 4, 64, 12) == ""
    assert lib.moe_gated_ffn_kernel(6, 4, 64, 64, 0) == b""
    assert lib.moe_gated_ffn_kernel(-1, 4, 64, 64, 1) == b""
    with pytest.raises(ValueError, match="none of"):
        moe.moe_gated_ffn_kernel("up", 4, 64, 64)
