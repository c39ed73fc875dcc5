"""What the gated block's roundings leave of it, for tests that an elementwise worst
case (i8_gated_ref) is too wide for.

Roundings as random.  The calls state where they round to bf16: h, dg and du between
the products, the results where they are bf16 (x and dout are taken as the call has
rounded them).  Each of these roundings is taken as independent and even over its
step, so that its variance is step^2 / 12, and a result's variance is the sum of
theirs.  fp32 sums of n products add n (2^-23)^2 of the products' squares: the matrix
cores' own order and rounding, a whole step for each term.  The mean of error^2 /
variance over a result is then 1; its spread follows from how many independent
roundings it rests on: for a result E Z with independent E [r][n] of variances s^2
and any Z [n][m], row r has pr = (sum s^2)^2 / sum s^4 of them and m values, of which
pr m / (pr + m) are independent.  A right result is within 8 standard deviations.

Exact data.  Small whole numbers, gates of 24 to 40 (silu(g) = g and its slope 1 in
fp32) and ups in steps of 1/32, so that every product and every partial sum in any
order is exact in fp32: results are one value each, whatever the kernel."""
import torch

from i8_gated_ref import silu

F64, BF16 = torch.float64, torch.bfloat16


def t_(m):
    return m.t().contiguous()


# --------------------------------------------------------- roundings as random
def rounding(v):
    """Variance of rounding v to bf16: v in [2^(e-1), 2^e) has steps of 2^(e-8)."""
    e = torch.frexp(v.abs()).exponent.to(F64)
    return torch.where(v == 0, 0.0, torch.exp2(2 * (e - 8)) / 12)


def sums(a, b):
    """Variance of the fp32 sums of a [M][n] times b [n][N]."""
    return a.shape[1] * 2.0 ** -46 * (a * a) @ (b * b)


def independent(var, m):
    """How many independent values rest on roundings of these variances, [r][n], when
    each row of them meets a matrix of m columns."""
    pr = var.sum(1) ** 2 / (var * var).sum(1).clamp_min(1e-300)
    return (pr * m / (pr + m).clamp_min(1)).sum().item()


def excess(got, want, var):
    """Mean of error^2 / variance."""
    off = (got.to(F64) - want) ** 2
    assert torch.isfinite(off).all()
    return (off / var.clamp_min(1e-300)).mean().item()


def limit(n):
    return 1 + 8 * (2 / n) ** 0.5


def pre(x, w):
    f = w.shape[0] // 2
    gu, e = x @ t_(w), sums(x, t_(w))
    return gu[:, :f], gu[:, f:], e[:, :f], e[:, f:]


def out_of(x, w, v, f32):
    """(out, variance, independent values) of the block, all fp64."""
    g, u, eg, eu = pre(x, w)
    h = silu(g) * u
    var = rounding(h)
    n = independent(var, v.shape[0])
    var = var + (1.1 * u) ** 2 * eg + silu(g) ** 2 * eu
    y = h @ t_(v)
    e = var @ t_(v * v) + sums(h, t_(v))
    return y, e if f32 else e + rounding(y), n


def gradients_of(dout, x, w, v, gate_up, dw_f32, x_rounded=None):
    """{name: (gradient, variance, independent values)}, all fp64.  x_rounded: what
    dw_gate_up multiplies in x's place (a checkpoint's rows, rounded to bf16)."""
    T, d = x.shape
    f = v.shape[1]
    if gate_up is None:
        g, u, eg, eu = pre(x, w)
    else:
        g, u = gate_up[:, :f], gate_up[:, f:]
        eg = eu = torch.zeros_like(g)
    s = torch.sigmoid(g)
    a, da = g * s, s * (1 + g * (1 - s))
    dh, edh = dout @ v, sums(dout, v)
    h, dgu = a * u, torch.cat((dh * u * da, dh * a), 1)
    rounded, vh = rounding(dgu), rounding(h)
    more = torch.cat(((u * da) ** 2 * edh + (dh * da) ** 2 * eu + (0.5 * dh * u) ** 2 * eg,
                      a * a * edh + (1.1 * dh) ** 2 * eg), 1)
    var = rounded + more
    eh = vh + (1.1 * u) ** 2 * eg + a * a * eu
    x = x if x_rounded is None else x_rounded
    dx, dw, dv = dgu @ w, t_(dgu) @ x, t_(dout) @ h
    edx = var @ (w * w) + sums(dgu, w) + rounding(dx)
    edw = t_(var) @ (x * x) + sums(t_(dgu), x)
    edv = t_(dout * dout) @ eh + sums(t_(dout), h)
    if not dw_f32:
        edw, edv = edw + rounding(dw), edv + rounding(dv)
    return {"dx": (dx, edx, independent(rounded, d)),
            "dw_gate_up": (dw, edw, independent(t_(rounded), d)),
            "dw_down": (dv, edv, independent(t_(vh), d))}


def check(name, got, model):
    """A result's errors are those of its roundings."""
    want, var, n = model
    r = excess(got, want, var)
    assert r <= limit(n), f"{name}: errors^2 {r:.3f} of the roundings', limit {limit(n):.3f}"


# ------------------------------------------------------------------- exact data
def exact_inputs(T, d, f, seed=0, device="cpu"):
    """x, w, v, dout (bf16): whole numbers, w's up rows in 1/32."""
    g = torch.Generator().manual_seed(seed + T + d + f)
    whole = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()  # noqa: E731
    terms = min(8, d - 1)
    x = whole(-1, 1, T, d)
    x[:, 0] = 32

    def sparse(rows, cols, n, first):  # n times +-1 a row, from column `first` on
        at = torch.randint(first, cols, (rows, n), generator=g)
        return torch.zeros(rows, cols).scatter_add_(1, at, 2 * whole(0, 1, rows, n) - 1)

    w = sparse(2 * f, d, terms, 1)
    w[:f, 0] = 1
    w[f:] /= 32
    v = t_(sparse(f, d, 3, 0))
    p = dict(x=x, w=w, v=v, dout=whole(-3, 3, T, d))
    return {k: m.to(BF16).to(device) for k, m in p.items()}


def exact_results(p):
    """{name: value} of the block and its gradient in fp64, with the stated roundings
    to bf16 between the products; every sum's terms stay below 2^24 units."""
    x, w, v, dout = (p[k].to(F64) for k in ("x", "w", "v", "dout"))
    f = v.shape[1]
    bf = lambda m: m.to(torch.float32).to(BF16).to(F64)  # noqa: E731

    def product(a, b, units):  # of units of 1 / units each
        assert ((a.abs() @ b.abs()) * units < 2 ** 24).all()
        return a @ b

    gu = product(x, t_(w), 32)
    g, u = gu[:, :f], gu[:, f:]
    assert g.min() >= 24 and g.max() <= 40
    h = bf(g * u)
    dh = product(dout, v, 1)
    dgu = bf(torch.cat((dh * u, dh * g), 1))
    units = torch.ones_like(w)  # dg in 1/32, du whole; x's first column in 32
    units[:f], units[f:, 0] = 32, 1 / 32
    units[:f, 0] = 1
    return {"gate_up": gu, "out": product(h, t_(v), 32), "dx": product(dgu, w, 32),
            "dw_gate_up": product(t_(dgu), x, units), "dw_down": product(t_(dout), h, 32)}


# ------------------------------------------------- the calls' arithmetic on the CPU
def emulated(p, kept=None, dw_f32=False, wrong=""):
    """The block and its gradient as the calls state them, in fp32 with roundings to
    bf16, from bf16 x, w, v, dout; `wrong` names a mistake to plant."""
    x, w, v, dout = (p[k].float() for k in ("x", "w", "v", "dout"))
    T, f = x.shape[0], v.shape[1]
    bf = lambda m: m.to(BF16).float()  # noqa: E731
    few = lambda m: m.to(torch.float8_e4m3fn).float()  # noqa: E731
    gu = x @ w.t()
    if kept is not None:
        gu = kept.float()
    if wrong == "bf16 pre-activations":
        gu = bf(gu)
    g, u = gu[:, :f], gu[:, f:]
    s = torch.sigmoid(g)
    a = g * s
    h = few(a * u) if wrong == "8-bit h" else bf(a * u)
    dh = dout @ v
    if wrong == "bf16 dh":
        dh = bf(dh)
    dgu = torch.cat((dh * u * (s + a * (1 - s)), dh * a), 1)
    dgu = few(dgu) if wrong == "8-bit dg and du" else bf(dgu)
    n = f - 8 if wrong == "last features dropped" else f
    live = torch.ones(2 * f)
    if n < f:
        live[n:f] = live[f + n:] = 0

    def over_tokens(m, q):
        if wrong == "last token dropped":
            m, q = m[:-1], q[:-1]
        if wrong != "bf16 sums of splits":
            return m.t() @ q
        step, y = -(-T // 8), 0
        for i in range(0, T, step):
            y = bf(y + bf(m[i:i + step].t() @ q[i:i + step]))
        return y

    dw, dv = over_tokens(dgu, x), over_tokens(dout, h)
    return {"out": bf(h[:, :n] @ v[:, :n].t()), "dx": bf((dgu * live) @ w),
            "dw_gate_up": dw if dw_f32 else bf(dw), "dw_down": dv if dw_f32 else bf(dv)}
