"""Plain 64-bit definitions of the operators around the routed experts, and
elementwise error bounds of their fp32 evaluation.

U is fp32's unit roundoff.  A sum of terms t_i whose evaluation passes m
roundings is off by at most m U sum |t_i|, a product chain of m roundings by
m U of its value; the bounds below count the roundings on the longest path of
a row (a thread's share of up to 32 values, 6 wave steps, 4 to 16 waves, and
the few products around them) as C = 128, and a column sum adds one for each
row that one of its chains passes.  Storing adds half a step of the type.
"""
import torch

U = 2.0 ** -24
C = 128
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.int16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    """The values of a tensor in fp64 (int16: bf16 bits)."""
    if t is None:
        return None
    return (t.view(torch.bfloat16) if t.dtype == torch.int16 else t).double()


def assert_within(out, ref, err, what):
    """|out - ref| <= err + half a step of out's type at |ref| + err."""
    o = f64(out)
    ref = ref.to(o.device)
    assert o.shape == ref.shape, (what, o.shape, ref.shape)
    tol = err + HALF_STEP[out.dtype] * (ref.abs() + err) + 2.0 ** -133
    bad = ~((o - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(),
                           float(((o - ref).abs() / tol).nan_to_num(float("inf")).max()))


# ---------------------------------------------------------------- linear map
def dequantize_w4(codes, scales):
    """fp64 [N][K] of the tiled int4 codes: word j of a row's group holds
    elements 8j..8j+7, the even ones in nibbles 0-3, the odd ones in 4-7."""
    N, K = codes.shape[-2], codes.shape[-1] * 2
    b = codes.reshape(N // 16, K // 128, 16, 16, 4).long()
    words = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16) | (b[..., 3] << 24)
    q = torch.stack([(words >> (4 * (e // 2 + 4 * (e % 2)))) & 15 for e in range(8)], -1)
    q = torch.where(q >= 8, q - 16, q).permute(0, 2, 1, 3, 4).reshape(N, K // 128, 128)
    s = scales.reshape(N, K // 128).view(torch.float16).double()
    return (q * s[..., None]).reshape(N, K)


def linear(x, codes, scales, bias=None):
    """(y, bound): the group sums are accumulated in fp32 over the 256 terms
    192 x and (192 + 8 q) x, |192 + 8 q| <= 248, weighted by s / 8; the K/128
    groups and the bias are then added."""
    W, x = dequantize_w4(codes, scales), f64(x)
    y = x @ W.t().contiguous()
    N, K = W.shape
    G = K // 128
    s = scales.reshape(N, G).view(torch.float16).double().abs()
    ax = x.abs().reshape(-1, G, 128).sum(2)
    bound = U * (256 + G + 4) * (440.0 / 8) * (ax @ s.t().contiguous())
    if bias is not None:
        y = y + f64(bias)
        bound = bound + U * y.abs()
    return y, bound


# --------------------------------------------------------------------- norms
def rstd(x, eps):
    return ((x * x).mean(1, keepdim=True) + eps).rsqrt()


def rmsnorm(x, gain, eps):
    y = x * rstd(x, eps)
    return y if gain is None else y * gain


def rmsnorm_bwd(dout, x, gain, dres, eps):
    """dx, dgain and their bounds."""
    g = torch.ones_like(x[:1]) if gain is None else gain
    r = rstd(x, eps)
    u, h = dout * g, x * r
    dx = r * (u - h * (u * h).mean(1, keepdim=True))
    edx = C * U * r * (u.abs() + h.abs() * (u * h).abs().mean(1, keepdim=True))
    if dres is not None:
        dx, edx = dx + dres, edx + 2 * U * dres.abs()
    dgain = (dout * h).sum(0)
    return dx, edx, dgain, (C + x.shape[0] / 64) * U * (dout * h).abs().sum(0)


# ------------------------------------------------------------- end of a block
def pair_rows(rows, pair_pos, T, k):
    """rows[pair_pos] as [T][k][d], zeros for dropped pairs, and which are live."""
    pos = pair_pos.reshape(-1).long()
    live = (pos >= 0) & (pos < T * k)
    got = torch.zeros(T * k, rows.shape[1], dtype=rows.dtype, device=rows.device)
    got[live] = rows[pos[live]]
    return got.view(T, k, -1), live.view(T, k)


def block_output(y, pos, w, add, T, d):
    o = torch.zeros(T, d, dtype=torch.float64, device=(add if y is None else y).device)
    if y is not None:
        rows, live = pair_rows(y, pos, T, w.shape[1])
        o = o + (rows * torch.where(live, w, torch.zeros_like(w))[..., None]).sum(1)
    return o if add is None else o + add


def combine_residual(res, y, pos, w, add, post, gate, scale, eps, nxt):
    """v and the next norm (gate broadcast to [T][d] or [1][1]), with bounds."""
    T, d = res.shape
    o = block_output(y, pos, w, add, T, d)
    oa = block_output(None if y is None else y.abs(), pos, None if w is None else w.abs(),
                      None if add is None else add.abs(), T, d)
    # an error e of o moves rstd by at most rstd * norm(e) / norm(o)
    a = 1 + oa.norm(dim=1, keepdim=True) / o.norm(dim=1, keepdim=True).clamp_min(1e-30)
    n, na = o, oa
    if post is not None:
        r = rstd(o, eps)
        n, na = o * r * post, oa * r * post.abs() * a
    v = scale * res + gate * n
    ev = C * U * ((scale * res).abs() + gate.abs() * na)
    if nxt is None:
        return v, ev, None, None
    r = rstd(v, eps)
    out = v * r * nxt
    eo = r * nxt.abs() * (ev + v.abs() * (C * U + ev.norm(dim=1, keepdim=True)
                                          / v.norm(dim=1, keepdim=True).clamp_min(1e-30)))
    return v, ev, out, eo


def combine_residual_bwd(dout, y, pos, w, add, post, gate, eps):
    """Per-token and per-channel gradients (dict of (value, bound)); gate is
    [T][1], [1][d] or [1][1]."""
    T, d = dout.shape
    o = block_output(y, pos, w, add, T, d)
    oa = block_output(None if y is None else y.abs(), pos, None if w is None else w.abs(),
                      None if add is None else add.abs(), T, d)
    a = 1 + oa.norm(dim=1, keepdim=True) / o.norm(dim=1, keepdim=True).clamp_min(1e-30)
    a = a.clamp_max(1e3)
    r = rstd(o, eps) if post is not None else torch.ones(T, 1, dtype=o.dtype, device=o.device)
    g = post if post is not None else torch.ones(1, d, dtype=o.dtype, device=o.device)
    u = dout * gate * g
    h, ha = o * r, oa * r
    if post is not None:
        do = r * (u - h * (u * h).mean(1, keepdim=True))
        eo = r * (u.abs() + ha * (u.abs() * ha).mean(1, keepdim=True)) * a
    else:
        do, eo = u, u.abs()
    out = dict(do=(do, C * U * eo))
    m = (C + T / 64) * U
    out["dpost"] = ((dout * gate * h).sum(0), m * (dout * gate * ha * a).abs().sum(0))
    n, na = h * g, ha * g.abs() * a
    out["dgate_t"] = ((dout * n).sum(1), C * U * (dout.abs() * na).sum(1))
    out["dgate_c"] = ((dout * n).sum(0), m * (dout.abs() * na).sum(0))
    if y is not None:
        rows, live = pair_rows(y, pos, T, w.shape[1])
        wl = torch.where(live, w, torch.zeros_like(w))
        out["dy"] = (do[:, None] * wl[..., None], (C * U * eo)[:, None] * wl.abs()[..., None])
        out["dw"] = ((rows * do[:, None]).sum(2), 2 * C * U * (rows.abs() * eo[:, None]).sum(2))
    return out
