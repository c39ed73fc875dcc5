"""The operators around the routed experts on the GPU against their 64-bit
definitions (block_ref): the 4-bit linear map, the norms before and after a
block, the token sort and its gradient; strided and dropped rows, guards
around outputs, streams, graphs, repeatability, and all of them together."""
import numpy as np
import pytest
import torch

import block_ref as ref
import quantized_mixture_experts_fp32_amd as moe
from block_ref import assert_within, f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def note(msg):
    print(msg, flush=True)


def gen(seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=F32):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV)

    normal.g = g
    return normal


def guarded(shape, dtype, fill=-7.0):
    """A dense tensor between two guard rows, and a check that they kept."""
    n = int(np.prod(shape))
    buf = torch.full((n + 512,), fill, dtype=dtype, device=DEV)
    view = buf[256:256 + n].view(shape)

    def kept():
        torch.cuda.synchronize()
        assert (buf[:256] == fill).all() and (buf[256 + n:] == fill).all()

    return view, kept


def grouping(seed, T, k, E, drop=0.0, pad=0):
    """pair_pos of a routed batch with dropped pairs at -1 (or past the end)."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), int)
    live = rng.random((T, k)) >= drop
    if pad:
        live[T - pad:] = False
    flat, keep = ids.reshape(-1), live.reshape(-1)
    pos = np.where(rng.random(T * k) < 0.5, -1, T * k + 5).astype(np.int32)
    order = [p for p in np.argsort(flat, kind="stable") if keep[p]]
    pos[order] = np.arange(len(order))
    return torch.from_numpy(pos).to(DEV)


# ----------------------------------------------------------------- linear map
LINEAR = [(1, 128, 16), (1, 2048, 2048), (2, 384, 48), (5, 4096, 272), (16, 1024, 1040),
          (17, 640, 528), (31, 1152, 64), (33, 2048, 272), (48, 4096, 512), (64, 2560, 4112),
          (65, 512, 272), (127, 1024, 48), (130, 384, 2064), (300, 1152, 528), (1000, 512, 784),
          (515, 2048, 4096), (1, 14336, 400), (3, 16512, 64), (70, 16512, 32), (2050, 256, 16),
          # few tokens, more row tiles: two and three a block, streamed (one and
          # several chunks of K)
          (3, 1024, 4128), (2, 1152, 4112), (5, 1152, 8208), (4, 1152, 20496), (9, 2176, 20496),
          (2, 8320, 20496),
          # token passes: six tiles a block, streamed
          (40, 640, 10256), (70, 1152, 12304), (70, 2176, 12304), (40, 4352, 24592),
          # GEMM tiles of 64, 96 and 128 tokens, N ending inside a feature block
          (1500, 640, 4112), (2501, 640, 2064), (1500, 256, 8208),
          # tiles of 32, 48 and 64 tokens by two to six row tiles
          (2501, 1408, 64), (64, 640, 976), (387, 640, 976), (33, 640, 13696), (97, 2304, 6224),
          (191, 4224, 4112),
          # few tokens streamed over one and several chunks of K, token passes
          (3, 3200, 26608), (16, 4224, 24912), (17, 1664, 50480), (17, 2176, 49216),
          (45, 2176, 49232), (19, 5248, 25712),
          # the GEMM for short K
          (2501, 128, 6160), (97, 256, 61664), (3001, 256, 3856)]


def linear_inputs(T, K, N, seed=0):
    normal = gen(1000 * seed + T + K + N)
    x = normal(T, K, dtype=BF)
    codes, scales = moe.moe_quantize_w4((normal(1, N, K) / K ** 0.5).contiguous())
    return x, codes[0], scales[0], normal(N)


@pytest.mark.parametrize("out_dtype", [moe.MOE_OUT_BF16, moe.MOE_OUT_F32])
@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear(T, K, N, out_dtype):
    note(f"linear T={T} K={K} N={N} out={out_dtype}")
    x, codes, scales, bias = linear_inputs(T, K, N)
    bias = bias if N % 32 else None
    out, kept = guarded((T, N), F32 if out_dtype == moe.MOE_OUT_F32 else BF)
    got = moe.moe_linear_w4(x, codes, scales, bias=bias, out=out, out_dtype=out_dtype)
    assert got is out
    kept()
    y, bound = ref.linear(x, codes, scales, bias)
    assert_within(out, y, bound, "linear")
    # in rms: about 256 roundings at |partial| ~ 1500 sigma against a group
    # sum of ~ 335 sigma give 2.5e-6; four times that, and the store
    rel = float((f64(out) - y).norm() / y.norm())
    assert rel <= 1e-5 + ref.HALF_STEP[out.dtype], rel


def test_linear_many_row_tiles():
    """More row tiles than a block's totals hold for a K of several chunks; the
    rows of the first, some middle and the last tiles against the definition."""
    T, K, N = 2, 4224, 131152
    note(f"linear T={T} K={K} N={N}")
    normal = gen(17)
    x = normal(T, K, dtype=BF)
    codes = torch.randint(0, 256, (N, K // 2), generator=normal.g, dtype=torch.uint8).to(DEV)
    scales = (torch.rand(N, K // 128, generator=normal.g) * 0.01).to(torch.float16).to(DEV)
    bias = normal(N)
    out = moe.moe_linear_w4(x, codes, scales, bias=bias, out_dtype=moe.MOE_OUT_F32)
    for a, b in ((0, 64), (4080, 4144), (65520, 65600), (N - 80, N)):
        y, bound = ref.linear(x, codes[a:b], scales[a:b].contiguous(), bias[a:b])
        assert_within(out[:, a:b], y, bound, f"rows {a}..{b}")


def test_linear_accepts_bits_and_leading_axis():
    note("linear: bf16 bits, [1][N][K/2] codes, fp16 scales")
    x, codes, scales, _ = linear_inputs(7, 512, 96)
    a = moe.moe_linear_w4(x, codes, scales)
    b = moe.moe_linear_w4(x.view(torch.int16), codes[None], scales[None].view(torch.float16))
    assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 20, 200])
def test_linear_zero_scales_and_large_values(T):
    """A group whose scale is 0 contributes nothing whatever its codes (the
    -8 a quantizer never writes among them), and values near 2^100 stay exact
    up to fp32's relative error."""
    note(f"linear zero scales T={T}")
    x, codes, scales, _ = linear_inputs(T, 768, 64, seed=3)
    scales = scales.clone()
    scales[::3, 1] = 0
    scales[5] = 0
    codes = codes.clone()
    codes.view(4, 6, 16, 64)[:, 1, ::3] = 0x88
    x = (x.float() * 2.0 ** 100).to(BF)
    out = moe.moe_linear_w4(x, codes, scales, out_dtype=moe.MOE_OUT_F32)
    y, bound = ref.linear(x, codes, scales)
    assert_within(out, y, bound, "linear")
    assert (out[:, 5] == 0).all()


@pytest.mark.parametrize("T", [3, 40, 300])
def test_linear_nonfinite_row_stays_in_its_row(T):
    note(f"linear nonfinite row T={T}")
    x, codes, scales, _ = linear_inputs(T, 512, 80, seed=4)
    clean = moe.moe_linear_w4(x, codes, scales)
    x = x.clone()
    x[1, 17] = float("inf")
    x[T - 1, 3] = float("nan")
    out = moe.moe_linear_w4(x, codes, scales)
    rest = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(out[rest], clean[rest])
    assert not torch.isfinite(out[1]).any() and out[T - 1].isnan().all()


# ---------------------------------------------------------------------- norms
NORM = [(1, 8), (3, 24), (5, 128), (2, 1000), (4, 2048), (3, 2056), (2, 4096), (1, 6152),
        (1030, 264), (515, 2048), (7, 8192), (2100, 1024), (300, 2600), (270, 5000)]


@pytest.mark.parametrize("dtype,out_dtype", [(BF, 0), (BF, 1), (F32, 0), (F32, 1)])
@pytest.mark.parametrize("T,d", NORM)
def test_rmsnorm(T, d, dtype, out_dtype):
    note(f"rmsnorm T={T} d={d} {dtype} out={out_dtype}")
    normal = gen(T + d)
    x = (normal(T, d) * 3).to(dtype)
    x[T // 2] = 0                       # an empty row: rstd = eps^(-1/2)
    gain = 1 + 0.3 * normal(d) if d % 16 else None
    out, kept = guarded((T, d), F32 if out_dtype else BF)
    moe.moe_rmsnorm(x, gain, eps=EPS, out=out, out_dtype=out_dtype)
    kept()
    y = ref.rmsnorm(f64(x), f64(gain), EPS)
    assert_within(out, y, ref.C * ref.U * y.abs(), "rmsnorm")
    assert (out[T // 2] == 0).all()


@pytest.mark.parametrize("ddtype,dtype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,d", NORM)
def test_rmsnorm_bwd(T, d, ddtype, dtype):
    note(f"rmsnorm_bwd T={T} d={d} {ddtype} {dtype}")
    normal = gen(7 * T + d)
    x, dout = (normal(T, d) * 3).to(dtype), normal(T, d, dtype=ddtype)
    x[T // 2] = 0
    gain = 1 + 0.3 * normal(d) if d % 16 or T > 600 else None
    dres = normal(T, d, dtype=dtype) if T != 4 else None
    dx, kept = guarded((T, d), dtype)
    _, dgain = moe.moe_rmsnorm_bwd(dout, x, gain, eps=EPS, dres=dres, dx=dx)
    kept()
    rdx, edx, rdg, edg = ref.rmsnorm_bwd(f64(dout), f64(x), f64(gain), f64(dres), EPS)
    assert_within(dx, rdx, edx, "dx")
    assert (dgain is None) == (gain is None)
    if gain is not None:
        assert_within(dgain, rdg, edg, "dgain")
    if dres is not None:                # in place
        again, dg2 = moe.moe_rmsnorm_bwd(dout, x, gain, eps=EPS, dres=dres, dx=dres)
        assert again is dres and torch.equal(dres, dx)
        assert dg2 is None or torch.equal(dg2, dgain)


# -------------------------------------------------------------- end of a block
# (T, d, k, E, dtype, gate, post, next, add, share of dropped pairs, padding)
BLOCK = [(1, 2048, 8, 64, BF, "token", True, True, False, 0.0, 0),
         (1, 8, 1, 2, F32, "none", True, True, False, 0.0, 0),
         (5, 256, 2, 8, F32, "channel", True, True, True, 0.3, 1),
         (33, 1000, 3, 8, BF, "none", False, True, False, 0.2, 2),
         (17, 2056, 8, 60, BF, "channel", True, False, True, 0.1, 0),
         (9, 4096, 16, 32, F32, "token", True, True, True, 0.2, 3),
         (3, 8192, 11, 16, BF, "channel", True, True, False, 0.0, 1),
         (40, 512, 0, 1, BF, "token", True, True, True, 0.0, 0),
         (6, 6152, 0, 1, F32, "none", False, False, True, 0.0, 0),
         (700, 264, 6, 64, BF, "channel", True, True, False, 0.0, 77),
         (1100, 1024, 8, 64, F32, "token", False, True, True, 0.05, 5),
         (530, 2048, 4, 8, BF, "channel", False, False, False, 0.0, 0),
         (300, 2600, 8, 16, BF, "channel", True, True, False, 0.1, 7),
         (270, 5000, 7, 16, F32, "none", True, True, True, 0.0, 0),
         (260, 4360, 12, 16, BF, "token", True, False, False, 0.1, 0)]


class BlockCase:
    def __init__(self, T, d, k, E, dtype, gate, post, nxt, add, drop, pad, seed=0):
        normal = gen(T + 3 * d + 7 * k + seed)
        self.T, self.d, self.k, self.dtype, self.scale = T, d, k, dtype, 0.75
        self.res = (normal(T, d) * 2).to(dtype)
        self.y = normal(T * k, d) if k else None
        self.pos = grouping(T + k, T, k, E, drop, pad) if k else None
        self.w = torch.softmax(normal(T, k), 1) if k else None
        if k:
            # what dropped pairs and unowned rows hold is never read
            dead = ~((self.pos >= 0) & (self.pos < T * k))
            self.w.view(-1)[dead] = float("nan")
            owned = torch.zeros(T * k, dtype=torch.bool, device=DEV)
            owned[self.pos[~dead].long()] = True
            self.y[~owned] = float("nan")
            self.owned = owned
        self.add = normal(T, d).to(dtype) if add else None
        self.post = 1 + 0.3 * normal(d) if post else None
        self.nxt = 1 + 0.3 * normal(d) if nxt else None
        self.gate_mode = {"none": 0, "token": 1, "channel": 2}[gate]
        self.gate = {"none": None, "token": torch.sigmoid(normal(T)),
                     "channel": normal(d)}[gate]
        if gate == "token" and T > 4:
            self.gate[3] = 0.0
        self.dout = normal(T, d).to(dtype)

    def kw(self):
        return dict(add=self.add, post_gain=self.post, gate=self.gate, gate_mode=self.gate_mode,
                    res_scale=self.scale, eps=EPS)

    def gate64(self):
        if self.gate is None:
            return torch.ones(1, 1, dtype=torch.float64, device=DEV)
        g = f64(self.gate)
        return g[:, None] if self.gate_mode == moe.MOE_GATE_TOKEN else g[None]

    def refs(self):
        return (f64(self.y), self.pos, f64(self.w), f64(self.add), f64(self.post), self.gate64())


@pytest.mark.parametrize("case", range(len(BLOCK)))
def test_combine_residual(case):
    note(f"combine_residual {BLOCK[case]}")
    c = BlockCase(*BLOCK[case])
    out, kept = guarded((c.T, c.d), c.dtype)
    nout, nkept = guarded((c.T, c.d), BF)
    _, n = moe.moe_combine_residual(c.res, c.y, c.pos, c.w, next_gain=c.nxt, out=out,
                                    next_out=nout if c.nxt is not None else None, **c.kw())
    kept(), nkept()
    y, pos, w, add, post, gate = c.refs()
    v, ev, rn, en = ref.combine_residual(f64(c.res), y, pos, w, add, post, gate, c.scale, EPS,
                                         f64(c.nxt))
    assert_within(out, v, ev, "out")
    assert (n is None) == (c.nxt is None)
    if n is not None:
        assert_within(n, rn, en, "next")
    # in place, and the next norm without a gain
    _, n1 = moe.moe_combine_residual(c.res, c.y, c.pos, c.w, out=c.res, next_norm=True, **c.kw())
    assert torch.equal(c.res, out)
    assert_within(n1, v * ref.rstd(v, EPS),
                  ref.rstd(v, EPS) * (ev + v.abs() * (ref.C * ref.U + ev.norm(dim=1, keepdim=True)
                                                      / v.norm(dim=1, keepdim=True))), "next1")


@pytest.mark.parametrize("dy_dtype", [0, 1])
@pytest.mark.parametrize("case", range(len(BLOCK)))
def test_combine_residual_bwd(case, dy_dtype):
    note(f"combine_residual_bwd {BLOCK[case]} dy={dy_dtype}")
    c = BlockCase(*BLOCK[case])
    kept = []
    out = {}
    if c.k:
        out["dy_pairs"], k1 = guarded((c.T * c.k, c.d), F32 if dy_dtype else BF)
        out["dtopk_w"], k2 = guarded((c.T, c.k), F32)
        kept += [k1, k2]
    got = moe.moe_combine_residual_bwd(c.dout, c.y, c.pos, c.w, dy_dtype=dy_dtype, **out, **c.kw())
    for k in kept:
        k()
    y, pos, w, add, post, gate = c.refs()
    r = ref.combine_residual_bwd(f64(c.dout), y, pos, w, add, post, gate, EPS)
    if c.k:
        rows = c.pos.view(-1).long()
        live = (rows >= 0) & (rows < c.T * c.k)
        dy, edy = r["dy"]
        assert_within(got.dy_pairs[rows[live]], dy.view(-1, c.d)[live], edy.view(-1, c.d)[live],
                      "dy")
        assert (got.dy_pairs[~c.owned] == -7.0).all()
        assert_within(got.dtopk_w, *r["dw"], "dw")
        assert (got.dtopk_w.view(-1)[~live] == 0).all()
    if add is not None:
        assert_within(got.dadd, *r["do"], "dadd")
    assert_within(got.dresidual, c.scale * f64(c.dout), 0.0, "dresidual")
    if post is not None:
        assert_within(got.dpost_gain, *r["dpost"], "dpost_gain")
    if c.gate_mode:
        assert_within(got.dgate, *r["dgate_t" if c.gate_mode == 1 else "dgate_c"], "dgate")
    absent = dict(dy_pairs=c.y, dtopk_w=c.y, dadd=c.add, dpost_gain=c.post, dgate=c.gate)
    for name, given in absent.items():
        assert (getattr(got, name) is None) == (given is None), name


def test_block_gradient_against_differences():
    """Directional differences of the 64-bit forward against the kernels'
    gradients, through the end of the block and the next norm."""
    note("block gradient against differences")
    c = BlockCase(12, 328, 4, 8, F32, "channel", True, True, True, 0.2, 1, seed=9)
    normal = gen(77)
    dn = normal(c.T, c.d)
    out, _ = moe.moe_combine_residual(c.res, c.y, c.pos, c.w, next_gain=c.nxt, **c.kw())
    dv, dnext_gain = moe.moe_rmsnorm_bwd(dn, out, c.nxt, eps=EPS, dres=c.dout)
    g = moe.moe_combine_residual_bwd(dv, c.y, c.pos, c.w, **c.kw())
    live = c.owned[:, None]
    y0 = torch.where(live, c.y, torch.zeros_like(c.y))
    w0 = torch.where(torch.isnan(c.w), torch.zeros_like(c.w), c.w)
    at = dict(res=c.res, y=y0, w=w0, add=c.add, post=c.post, gate=c.gate, nxt=c.nxt)
    grads = dict(res=g.dresidual, y=torch.where(live, g.dy_pairs, torch.zeros_like(c.y)),
                 w=g.dtopk_w, add=g.dadd, post=g.dpost_gain, gate=g.dgate, nxt=dnext_gain)

    def loss(p):
        v, _, n, _ = ref.combine_residual(p["res"], p["y"], c.pos, p["w"], p["add"], p["post"],
                                          p["gate"][None], c.scale, EPS, p["nxt"])
        return float((v * f64(c.dout)).sum() + (n * f64(dn)).sum())

    base = {n: f64(t) for n, t in at.items()}
    for name in base:
        v = f64(normal(*base[name].shape))
        h = 1e-5 * float(base[name].norm() / v.norm())
        plus, minus = dict(base), dict(base)
        plus[name], minus[name] = base[name] + h * v, base[name] - h * v
        num = (loss(plus) - loss(minus)) / (2 * h)
        ana = f64(grads[name]) * v
        # fp32 gradients: C U of the terms' magnitudes and some (the fp32 `out`
        # that the norm's gradient starts from); differences: h^2 and 1e-16 / h
        assert abs(num - float(ana.sum())) <= 1e-5 * float(ana.abs().sum()) + 1e-4, name


@pytest.mark.parametrize("post", [False, True])
def test_dropped_pairs_of_an_infinite_token(post):
    """A dropped pair has the weight gradient 0 whatever its token's row holds."""
    note(f"dropped pairs of an infinite token, post {post}")
    normal = gen(5)
    T, d, k = 3, 264, 3
    pos = torch.tensor([0, -1, 1, 9, 2, 3, 4, 5, -1], dtype=torch.int32, device=DEV)
    dropped = torch.tensor([[0, 1, 0], [1, 0, 0], [0, 0, 1]], dtype=torch.bool, device=DEV)
    y, w = normal(T * k, d), torch.softmax(normal(T, k), 1)
    x, dxs = normal(T, d), normal(T * k, d)
    x[:, 17] = float("inf")
    gain = 1 + 0.3 * normal(d) if post else None
    dw = moe.moe_combine_residual_bwd(x, y, pos, w, post_gain=gain, eps=EPS).dtopk_w
    assert (dw[dropped] == 0).all() and not torch.isfinite(dw[~dropped]).any()
    for dw in (moe.moe_dispatch_bwd(dxs, pos, k, x=x, topk_w=w)[1],
               moe.moe_combine_bwd(x, y, pos, w)[1]):
        assert (dw[dropped] == 0).all() and torch.isinf(dw[~dropped]).all()


def test_block_gradient_without_norm_does_not_square_the_output():
    """Without a norm the gradient of o is gate * dout and no <o, y_j> enters:
    rows of 1e25, whose squares have no fp32, leave it finite."""
    note("block gradient without norm, large rows")
    c = BlockCase(5, 264, 3, 8, F32, "token", False, False, True, 0.2, 0)
    c.y *= 1e25
    g = moe.moe_combine_residual_bwd(c.dout, c.y, c.pos, c.w, **c.kw())
    r = ref.combine_residual_bwd(f64(c.dout), *c.refs(), EPS)
    assert_within(g.dadd, *r["do"], "dadd")
    assert_within(g.dtopk_w, *r["dw"], "dtopk_w")
    assert_within(g.dgate, *r["dgate_t"], "dgate")


# ------------------------------------------------------------------ token sort
# (T, d, k, E, dtype, share of dropped pairs, padding)
SORT = [(1, 8, 1, 1, BF, 0.0, 0), (1, 2048, 8, 64, F32, 0.0, 0), (3, 24, 2, 4, F32, 0.4, 1),
        (33, 1000, 3, 8, BF, 0.3, 2), (19, 4104, 16, 32, BF, 0.1, 0), (7, 8192, 8, 60, F32, 0.2, 2),
        (1030, 264, 6, 64, BF, 0.0, 31), (515, 2048, 8, 64, F32, 0.0, 0)]


def sort_inputs(case):
    T, d, k, E, dtype, drop, pad = SORT[case]
    normal = gen(T + d + k)
    pos = grouping(T + k, T, k, E, drop, pad)
    live = (pos >= 0) & (pos < T * k)
    owned = torch.zeros(T * k, dtype=torch.bool, device=DEV)
    owned[pos[live].long()] = True
    w = torch.softmax(normal(T, k), 1)
    w.view(-1)[~live] = float("nan")
    return T, d, k, dtype, normal, pos, live, owned, w


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("case", range(len(SORT)))
def test_dispatch(case, weighted):
    note(f"dispatch {SORT[case]} weighted={weighted}")
    T, d, k, dtype, normal, pos, live, owned, w = sort_inputs(case)
    x = normal(T, d, dtype=dtype)
    out, kept = guarded((T * k, d), dtype)
    moe.moe_dispatch(x, pos, k, topk_w=w if weighted else None, out=out)
    kept()
    rows = f64(x).repeat_interleave(k, 0)
    if weighted:
        rows = rows * f64(w).view(-1, 1)
    got = out[pos[live].long()]
    assert_within(got, rows[live], 0.0, "xs")
    if not weighted:
        assert torch.equal(got, x.repeat_interleave(k, 0)[live])
    assert (out[~owned] == -7.0).all()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("case", range(len(SORT)))
def test_dispatch_bwd(case, weighted):
    note(f"dispatch_bwd {SORT[case]} weighted={weighted}")
    T, d, k, dtype, normal, pos, live, owned, w = sort_inputs(case)
    x, dxs = normal(T, d, dtype=dtype), normal(T * k, d, dtype=dtype)
    dxs[~owned] = float("nan")
    dx, kept = guarded((T, d), dtype)
    _, dw = moe.moe_dispatch_bwd(dxs, pos, k, x=x if weighted else None,
                                 topk_w=w if weighted else None, dx=dx)
    kept()
    rows, lv = ref.pair_rows(f64(dxs), pos, T, k)
    f = torch.where(lv, f64(w) if weighted else torch.ones_like(f64(w)), 0.0)[..., None]
    assert_within(dx, (rows * f).sum(1), 20 * ref.U * (rows * f).abs().sum(1), "dx")
    assert (dw is None) == (not weighted)
    if weighted:
        t = rows * f64(x)[:, None]
        assert_within(dw, t.sum(2), ref.C * ref.U * t.abs().sum(2), "dw")
        only, none = moe.moe_dispatch_bwd(dxs, pos, k, topk_w=w)
        assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("ddtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(SORT)))
def test_combine_bwd(case, ddtype):
    note(f"combine_bwd {SORT[case]} {ddtype}")
    T, d, k, dtype, normal, pos, live, owned, w = sort_inputs(case)
    dout, y = normal(T, d, dtype=ddtype), normal(T * k, d)
    y[~owned] = float("nan")
    dy, kept = guarded((T * k, d), dtype)
    _, dw = moe.moe_combine_bwd(dout, y, pos, w, dy_pairs=dy,
                                dy_dtype=moe.MOE_OUT_F32 if dtype == F32 else moe.MOE_OUT_BF16)
    kept()
    rows, lv = ref.pair_rows(f64(y), pos, T, k)
    t = rows * f64(dout)[:, None]
    assert_within(dw, t.sum(2), ref.C * ref.U * t.abs().sum(2), "dw")
    assert (dw.view(-1)[~live] == 0).all()
    rdy = (f64(dout)[:, None] * torch.where(lv, f64(w), 0.0)[..., None]).view(T * k, d)
    assert_within(dy[pos[live].long()], rdy[live], 0.0, "dy")
    assert (dy[~owned] == -7.0).all()


def test_sort_and_back_is_the_layer_grouping():
    """dispatch with moe_permute's grouping, then the framework's combine: the
    weighted sum of k copies is the token itself (weights sum to 1)."""
    note("sort and back")
    T, d, k, E = 203, 512, 4, 16
    normal = gen(5)
    ids = torch.stack([torch.randperm(E, generator=normal.g)[:k] for _ in range(T)])
    off, sp, pos = moe.moe_permute(ids.to(torch.int32).to(DEV), E)
    x, w = normal(T, d), torch.softmax(normal(T, k), 1)
    xs = moe.moe_dispatch(x, pos, k)
    assert torch.equal(xs, x[(sp // k).long()])
    back = moe.moe_combine(xs, pos, w, out_dtype=moe.MOE_OUT_F32)
    want = f64(x) * f64(w).sum(1, keepdim=True)
    assert_within(back, want, 20 * ref.U * f64(x).abs(), "back")


def test_offsets_past_32_bits():
    """Grouped rows past 4 GiB: the last token's rows of every call."""
    note("offsets past 32 bits")
    T, k, d = 20000, 8, 8192
    normal = gen(31)
    pos = torch.arange(T * k, dtype=torch.int32, device=DEV)
    last = slice((T - 1) * k, T * k)
    y = torch.zeros(T * k, d, device=DEV)           # 5.2 GB
    x, w = torch.zeros(T, d, device=DEV), torch.softmax(normal(T, k), 1)
    x[-1], y[last] = normal(d), normal(k, d)
    y64, w64, x64 = f64(y[last]), f64(w[-1]), f64(x[-1])
    out, _ = moe.moe_combine_residual(x, y, pos, w)
    assert_within(out[-1:], (x64 + (w64[:, None] * y64).sum(0))[None],
                  20 * ref.U * (x64.abs() + (w64[:, None] * y64.abs()).sum(0))[None], "combine")
    dy, dw = moe.moe_combine_bwd(x, y, pos, w)
    assert_within(dy[last], w64[:, None] * x64, 0.0, "dy")
    assert_within(dw[-1], (y64 * x64).sum(1), ref.C * ref.U * (y64 * x64).abs().sum(1), "dw")
    del dy
    xs = moe.moe_dispatch(x, pos, k, topk_w=w)
    assert_within(xs[last], w64[:, None] * x64, 0.0, "xs")
    xs[last] = y[last]
    dx, dw = moe.moe_dispatch_bwd(xs, pos, k, x=x, topk_w=w)
    assert_within(dx[-1], (w64[:, None] * y64).sum(0),
                  20 * ref.U * (w64[:, None] * y64.abs()).sum(0), "dx")
    del xs
    g = moe.moe_combine_residual_bwd(x, y, pos, w)
    assert_within(g.dy_pairs[last], w64[:, None] * x64, 0.0, "block dy")


# --------------------------------------------------- zero tokens, repeatability
def test_zero_tokens():
    note("zero tokens")
    d, k = 64, 2
    z = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    gain = torch.ones(d, device=DEV)
    pos = z(0, dtype=torch.int32)
    assert moe.moe_linear_w4(z(0, 128, dtype=BF), z(16, 64, dtype=torch.uint8),
                             z(16, 1, dtype=torch.int16)).shape == (0, 16)
    assert moe.moe_rmsnorm(z(0, d)).shape == (0, d)
    _, dg = moe.moe_rmsnorm_bwd(z(0, d), z(0, d), gain)
    assert (dg == 0).all()
    out, nxt = moe.moe_combine_residual(z(0, d), z(0, d), pos, z(0, k), next_gain=gain)
    assert out.shape == nxt.shape == (0, d)
    g = moe.moe_combine_residual_bwd(z(0, d), z(0, d), pos, z(0, k), post_gain=gain, gate=gain,
                                     gate_mode=moe.MOE_GATE_CHANNEL)
    assert (g.dpost_gain == 0).all() and (g.dgate == 0).all() and g.dy_pairs.shape == (0, d)
    assert moe.moe_dispatch(z(0, d), pos, k).shape == (0, d)
    assert moe.moe_dispatch_bwd(z(0, d), pos, k)[0].shape == (0, d)
    dy, dw = moe.moe_combine_bwd(z(0, d), z(0, d), pos, z(0, k))
    assert dy.shape == (0, d) and dw.shape == (0, k)
    torch.cuda.synchronize()


class Chain:
    """The operators as a decoder layer uses them, training step included."""

    def __init__(self, T, seed=0):
        d, k, E, N = 512, 4, 8, 512
        normal = gen(40 + T + seed)
        self.k = k
        self.res = normal(T, d, dtype=BF)
        self.wc, self.ws = moe.moe_quantize_w4((normal(1, N, d) / d ** 0.5).contiguous())
        self.gains = [1 + 0.2 * normal(d) for _ in range(3)]
        ids = torch.stack([torch.randperm(E, generator=normal.g)[:k] for _ in range(T)])
        self.ids = ids.to(torch.int32).to(DEV)
        self.E = E
        self.w = torch.softmax(normal(T, k), 1)
        self.gate = torch.sigmoid(normal(T))

    def step(self, stream=None):
        s = dict(stream=stream) if stream is not None else {}
        a = moe.moe_rmsnorm(self.res, self.gains[0], **s)
        o = moe.moe_linear_w4(a, self.wc, self.ws, **s)
        mid, xn = moe.moe_combine_residual(self.res, add=o, next_gain=self.gains[1], **s)
        _, _, pos = moe.moe_permute(self.ids, self.E, **s)
        xs = moe.moe_dispatch(xn, pos, self.k, **s)
        y = moe.moe_linear_w4(xs, self.wc, self.ws, out_dtype=moe.MOE_OUT_F32, **s)
        kw = dict(post_gain=self.gains[2], gate=self.gate, gate_mode=moe.MOE_GATE_TOKEN, **s)
        out, _ = moe.moe_combine_residual(mid, y, pos, self.w, **kw)
        g = moe.moe_combine_residual_bwd(out, y, pos, self.w, dy_dtype=moe.MOE_OUT_BF16, **kw)
        dxn, dw2 = moe.moe_dispatch_bwd(g.dy_pairs, pos, self.k, x=xn, topk_w=self.w, **s)
        dmid, dgain = moe.moe_rmsnorm_bwd(dxn, mid, self.gains[1], dres=g.dresidual, **s)
        dy, dw3 = moe.moe_combine_bwd(dmid, y, pos, self.w, **s)
        return [out, y, xs, g.dtopk_w, g.dpost_gain, g.dgate, dxn, dw2, dmid, dgain, dy, dw3]


@pytest.mark.parametrize("T", [1, 16, 150])
def test_chain_repeats_and_runs_on_a_stream(T):
    note(f"chain T={T}: repeat, side stream")
    c = Chain(T)
    first = c.step()
    for a, b in zip(first, c.step()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(2048, 2048, device=DEV)
    for _ in range(4):
        busy = busy @ busy * 1e-3       # the default stream has work of its own
    second = c.step(stream=side)
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 16, 150])
def test_chain_captured_and_replayed(T):
    note(f"chain T={T}: graph")
    c = Chain(T)
    want = c.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.step()
    for r in range(3):
        for t in got:
            t.fill_(-3.0)
        c.res.copy_(c.res.float() * (1 + r) if r else c.res)
        want = c.step()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(want, got)):
            assert torch.equal(a, b), (r, i)


def test_two_graphs_do_not_share_workspaces():
    note("two graphs, replayed in turn and on two streams")
    cs = [Chain(90, seed=s) for s in (1, 2)]
    want = [c.step() for c in cs]
    graphs, got = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            got.append(c.step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        for a, b in zip(w, o):
            assert torch.equal(a, b)


def test_block_around_the_quantized_layer():
    """norm -> router, grouping and int4 experts -> combine, norm, gate and
    residual: equal to the layer's own combine followed by the 64-bit rest."""
    note("block around the quantized layer")
    T, d, E, k, f = 37, 512, 8, 2, 256
    normal = gen(11)
    res = normal(T, d, dtype=BF)
    gains = [1 + 0.2 * normal(d) for _ in range(3)]
    wr = (normal(E, d) / d ** 0.5).to(BF)
    gu = moe.moe_quantize_w4((normal(E, 2 * f, d) / d ** 0.5).contiguous())
    dn = moe.moe_quantize_w4((normal(E, d, f) / f ** 0.5).contiguous())
    layer = moe.MoeLayer(wr, None, k, f, *gu, *dn)
    x = moe.moe_rmsnorm(res, gains[0], eps=EPS)
    o = layer.forward(x, out_dtype=moe.MOE_OUT_F32)
    out, nxt = moe.moe_combine_residual(res, layer.y_pairs, layer.pair_pos, layer.topk_w,
                                        post_gain=gains[1], res_scale=0.5, eps=EPS,
                                        next_gain=gains[2])
    o64 = ref.block_output(f64(layer.y_pairs), layer.pair_pos, f64(layer.topk_w), None, T, d)
    assert_within(o, o64, 8 * ref.U * o64.abs().max(), "combine")
    one = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    v, ev, rn, en = ref.combine_residual(f64(res), f64(layer.y_pairs), layer.pair_pos,
                                         f64(layer.topk_w), None, f64(gains[1]), one, 0.5, EPS,
                                         f64(gains[2]))
    assert_within(out, v, ev, "out")
    assert_within(nxt, rn, en, "next")

    # the layer's own method makes the same calls
    got = layer.forward_block(res, gains[0], post_gain=gains[1], res_scale=0.5, eps=EPS,
                              next_gain=gains[2])
    assert torch.equal(got[0], out) and torch.equal(got[1], nxt)
    plain, none = layer.forward_block(res, gains[0], eps=EPS)
    assert none is None
    assert_within(plain, f64(res) + f64(o), 8 * ref.U * o64.abs().max(), "plain block")


@pytest.mark.parametrize("T", [1, 37])
def test_block_layer_on_a_stream_and_captured(T):
    """forward_block with bf16 and fp32 residuals, in place, on a side stream
    and replayed from a graph, equals the eager call."""
    note(f"forward_block T={T}: stream, graph")
    d, E, k, f = 512, 8, 2, 256
    normal = gen(60 + T)
    wr = (normal(E, d) / d ** 0.5).to(BF)
    gu = moe.moe_quantize_w4((normal(E, 2 * f, d) / d ** 0.5).contiguous())
    dn = moe.moe_quantize_w4((normal(E, d, f) / f ** 0.5).contiguous())
    layer = moe.MoeLayer(wr, None, k, f, *gu, *dn)
    gain, nxt, gate = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d), normal(d)
    kw = dict(gate=gate, gate_mode=moe.MOE_GATE_CHANNEL, post_gain=gain, next_gain=nxt, eps=EPS)
    for dtype in (BF, F32):
        res = normal(T, d, dtype=dtype)
        want = layer.forward_block(res, gain, **kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = layer.forward_block(res, gain, stream=side, **kw)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        graph, buf = torch.cuda.CUDAGraph(), res.clone()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out, nout = layer.forward_block(buf, gain, out=buf, **kw)
        assert out is buf
        for _ in range(3):
            buf.copy_(res)
            graph.replay()
            torch.cuda.synchronize()
            again = layer.forward_block(res, gain, **kw)
            torch.cuda.synchronize()
            assert torch.equal(buf, want[0]) and torch.equal(nout, want[1])
            assert torch.equal(again[0], want[0])


def test_gpu_argument_checks():
    """Refusals that need a device: a CPU tensor among GPU ones, a stream of
    the wrong kind of device is refused by shape checks before any launch."""
    note("argument checks")
    x = torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError, match="gain is on cpu"):
        moe.moe_rmsnorm(x, torch.ones(64))
    with pytest.raises(ValueError, match="not contiguous"):
        moe.moe_rmsnorm(torch.zeros(64, 4, device=DEV).t())
    with pytest.raises(ValueError, match="below 2"):   # an int of 32 bits would wrap
        moe.moe_dispatch(x, torch.zeros(8, dtype=torch.int32, device=DEV), 2 ** 32 + 2)
    with pytest.raises(moe.MoeError, match="misaligned"):
        moe.moe_rmsnorm(torch.zeros(4 * 64 + 1, device=DEV)[1:].view(4, 64))
    with pytest.raises(moe.MoeError, match="multiple of 8"):
        moe.moe_rmsnorm(torch.zeros(4, 60, device=DEV))
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_rmsnorm_bwd(x, x, torch.ones(64, device=DEV),
                            ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(moe.MoeError, match="MOE_ERR_UNSUPPORTED"):
        moe.moe_linear_w4(torch.zeros(2, 128, dtype=BF, device=DEV),
                          torch.zeros(24, 64, dtype=torch.uint8, device=DEV),
                          torch.zeros(24, 1, dtype=torch.int16, device=DEV))
