"""64-bit definitions of the 8-bit rows, the 8-bit linear map and the gated
feed-forward block, and how far a correct kernel may be from them.

Bounds are elementwise and first order in the roundings that the calls state:
half a step of bf16 is 2^-8 of the value; a sum of n products in fp32 is within
(n + 2) 2^-23 of the sum of their magnitudes (the matrix cores' order and
rounding inside an instruction are their own: a whole step for each term)."""
import numpy as np
import torch

F64 = torch.float64
BF = 2.0 ** -8    # half a step of bf16, relative
F32 = 2.0 ** -24  # half a step of fp32
STEP = 2.0 ** -23
TINY = np.float32(2.0 ** -119)


def quantize(x, group):
    """Codes int8 and scales fp32 of fp32 rows (numpy), group 128 or 0."""
    T, K = x.shape
    n = group or K
    G = -(-K // n)
    codes, scales = np.zeros((T, K), np.int8), np.zeros((T, G), np.float32)
    with np.errstate(all="ignore"):
        for g in range(G):
            v = x[:, n * g:n * (g + 1)].astype(np.float32)
            m = np.abs(v).max(1)
            bad = ~np.isfinite(v).all(1)
            live = ~bad & (m >= TINY)
            safe = np.where(live, m, np.float32(1))
            s = np.where(live, safe / np.float32(127), np.float32(0))
            scales[:, g] = np.where(bad, np.float32(np.nan), s)
            inv = np.where(live, np.float32(127) / safe, np.float32(0))
            q = np.rint(np.where(live[:, None], v, np.float32(0)) * inv[:, None])
            codes[:, n * g:n * (g + 1)] = q.astype(np.int8)
    return codes, scales if group else scales[:, 0]


def restore(codes, scales):
    """codes * scales in fp64 (torch)."""
    s = scales.to(F64)
    if s.dim() == 1:
        return codes.to(F64) * s[:, None]
    return codes.to(F64) * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


def linear_i8(q, sx, codes, scales, bias):
    """(value, bound before the store's rounding): four fp32 steps, each half a
    step of a value no larger than |scaled sum| + |bias|."""
    y = (q.to(F64) @ codes.to(F64).t().contiguous()) * sx.to(F64)[:, None] * scales.to(F64)
    b = torch.zeros_like(y) if bias is None else bias.to(F64)[None, :]
    return y + b, 4.01 * F32 * (y.abs() + b.abs())


def stored(y, bound, f32):
    """The bound with the store's rounding (and bf16's smallest step)."""
    return bound if f32 else bound * (1 + BF) + BF * y.abs() + 2.0 ** -133


def sum_error(n, a, b):
    """Of fp32 sums of n products: a [M][n] and b [n][N] magnitudes."""
    return (n + 2) * STEP * (a @ b)


def silu(g):
    return g * torch.sigmoid(g)


def pre_activations(x, w):
    """(gate, up) and the bounds of their fp32 sums."""
    f = w.shape[0] // 2
    gu = x @ w.t().contiguous()
    e = sum_error(x.shape[1], x.abs(), w.abs().t().contiguous())
    return gu[:, :f], gu[:, f:], e[:, :f], e[:, f:]


# silu' lies in [-0.1, 1.1], silu'' in [-0.2, 0.5].  e^-g with g taken times
# log2 e in fp32 and the hardware exp2, reciprocal and products: (|g| + 8) steps.
def act_error(g):
    return (g.abs() + 8) * STEP


def h_error(g, u, eg, eu):
    h = silu(g) * u
    e = 1.1 * u.abs() * eg + silu(g).abs() * eu + h.abs() * act_error(g)
    return h, e * (1 + BF) + BF * h.abs() + 2.0 ** -133


def gated_ffn(x, w, v, f32=False):
    """(out, bound, gate_up, its bound) for fp64 x [T][d], w [2f][d], v [d][f]."""
    g, u, eg, eu = pre_activations(x, w)
    h, eh = h_error(g, u, eg, eu)
    vt = v.t().contiguous()
    y = h @ vt
    e = eh @ vt.abs() + sum_error(v.shape[1], h.abs() + eh, vt.abs())
    gu, egu = torch.cat((g, u), 1), torch.cat((eg, eu), 1)
    return y, stored(y, e, f32), gu, stored(gu, egu, False)


def gated_ffn_bwd(dout, x, w, v, gate_up=None, dout_f32=False, x_rounded=False, dw_f32=False):
    """((dx, dw_gate_up, dw_down), their bounds).  x_rounded: the call rounds x
    to bf16 first; dout_f32: it rounds dout."""
    T, d = x.shape
    f = v.shape[1]
    ex = BF * x.abs() if x_rounded else torch.zeros_like(x)
    edo = BF * dout.abs() if dout_f32 else torch.zeros_like(dout)
    if gate_up is None:
        g, u, eg, eu = pre_activations(x, w)
        wa = w.abs().t().contiguous()
        more = ex @ wa
        eg, eu = eg + more[:, :f], eu + more[:, f:]
    else:
        g, u = gate_up[:, :f], gate_up[:, f:]
        eg = eu = torch.zeros_like(g)
    s = torch.sigmoid(g)
    a, da = g * s, s * (1 + g * (1 - s))
    dh = dout @ v
    edh = edo @ v.abs() + sum_error(d, dout.abs(), v.abs())
    dg, du = dh * u * da, dh * a
    act = act_error(g) + 4 * STEP
    edg = edh * (u * da).abs() + (dh * da).abs() * eu + 0.5 * (dh * u).abs() * eg
    # (the terms of da cancel: the roundings are of each)
    edg = edg + act * (dh * u).abs() * (s + (a * (1 - s)).abs())
    edu = edh * a.abs() + 1.1 * dh.abs() * eg + act * du.abs()
    dgu, e = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    e = e * (1 + BF) + BF * dgu.abs() + 2.0 ** -133
    h, eh = h_error(g, u, eg, eu)
    dx = dgu @ w
    edx = e @ w.abs() + sum_error(2 * f, dgu.abs() + e, w.abs())
    t = lambda m: m.t().contiguous()  # noqa: E731
    dw = t(dgu) @ x
    edw = t(e) @ (x.abs() + ex) + t(dgu).abs() @ ex + sum_error(T, t(dgu).abs() + t(e), x.abs() + ex)
    dv = t(dout) @ h
    edv = t(dout).abs() @ eh + t(edo) @ (h.abs() + eh) + sum_error(T, t(dout).abs() + t(edo),
                                                                   h.abs() + eh)
    return (dx, dw, dv), (stored(dx, edx, False), stored(dw, edw, dw_f32),
                          stored(dv, edv, dw_f32))


def check(name, got, want, bound):
    """Every element within its bound (and finite)."""
    off = (got.to(F64) - want).abs()
    assert torch.isfinite(got).all(), name
    worst = (off / bound.clamp_min(1e-300)).max().item() if off.numel() else 0.0
    assert worst <= 1.0, (name, worst)
