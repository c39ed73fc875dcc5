"""Speed cases of the operators around the routed experts: the 4-bit linear
map, the norms before and after a block, and the token sort with its gradient.

Shapes follow the layers this package is built for (model width d 2048 or
4096, top-8 of 64 or 256 experts, group-128 int4 codes) and the batches they
see: one token, decode batches up to 64, prompts of thousands of tokens.

`run` computes an operator in plain torch (fp32, rounded once at the end);
with `own` true it makes the package's call.  `exact` computes the same
outputs in fp64, written apart from the plain form.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode token through a square projection: latency
        linear("linear-token", 1, 2048, 2048, "bf16", False),
        # four sequences' logits over a 50304-word vocabulary: weight bytes
        linear("linear-vocabulary", 4, 4096, 50304, "f32", False),
        # a decode batch of 64 through a fused projection with bias
        linear("linear-batch", 64, 4096, 12288, "bf16", True),
        # a ragged prompt: the product is bound by the matrix cores
        linear("linear-prompt", 2501, 4096, 4096, "bf16", False),
        # the norm in front of a block, decode
        dict(name="norm-decode", op="norm", dir="fwd", T=16, d=4096, dtype="bf16"),
        # its gradient over a training batch, with the residual path's gradient
        dict(name="norm-train", op="norm", dir="bwd", T=8191, d=4096, dtype="bf16"),
        # end of a routed block for one token: combine, post norm, token gate,
        # residual, next norm
        block("block-token", "fwd", 1, 4096, 8, 256, "bf16", "token", True, True, False, 0),
        # the same over a padded prompt with a float32 residual stream, a
        # channel gate and a shared expert's output
        block("block-prompt", "fwd", 4096, 2048, 8, 64, "f32", "channel", True, True, True, 37),
        # its gradient over a training batch
        block("block-train", "bwd", 4093, 4096, 8, 256, "bf16", "channel", True, False, False, 0),
        # tokens copied into expert order before the experts' products
        dict(name="sort-prompt", op="dispatch", dir="fwd", T=8192, d=2048, k=8, E=64,
             dtype="bf16", weighted=False, pad=100),
        # the gradient of that copy, with weights applied on the way in
        dict(name="sort-train", op="dispatch", dir="bwd", T=4095, d=2048, k=8, E=64,
             dtype="bf16", weighted=True, pad=0),
        # the gradient of the combine: expert rows and routing weights (a
        # small router-tuning batch)
        dict(name="combine-train", op="combine", dir="bwd", T=515, d=4096, k=8, E=256,
             dtype="f32", weighted=True, pad=3),
    ]


def linear(name, T, K, N, out, bias):
    return dict(name=name, op="linear", dir="fwd", T=T, K=K, N=N, dtype=out, bias=bias)


def block(name, direction, T, d, k, E, dtype, gate, post, nxt, add, pad):
    return dict(name=name, op="block", dir=direction, T=T, d=d, k=k, E=E, dtype=dtype, gate=gate,
                post=post, next=nxt, add=add, pad=pad)


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def cost(case):
    """Rough seconds of a pass: what bounds a drawn case."""
    w = work(case)
    return max(w["bytes"] / 4e12, w["flops"] / 5e14)


def draw(rng):
    most = max(cost(c) for c in listed())
    while True:
        c = candidate(rng)
        if cost(c) <= most:
            return c


def candidate(rng):
    op = rng.choice(["linear", "linear", "linear", "norm", "norm", "block", "block", "block",
                     "dispatch", "dispatch", "combine"])
    if op == "linear":
        return dict(op=op, dir="fwd", T=spread(rng, 1, 4096), K=GROUP * spread(rng, 4, 112),
                    N=16 * spread(rng, 16, 3144), dtype=rng.choice(["bf16", "f32"]),
                    bias=rng.random() < 0.5)
    T, d, dtype = spread(rng, 1, 8192), 8 * spread(rng, 32, 1024), rng.choice(["bf16", "f32"])
    if op == "norm":
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, d=d, dtype=dtype)
    k = rng.choice([2, 4, 6, 8])
    E = rng.choice([8, 64, 60, 256])
    pad = rng.choice([0, 0, T // 9])
    if op == "block":
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, d=d, k=k, E=E, dtype=dtype,
                    gate=rng.choice(["none", "token", "channel"]), post=rng.random() < 0.7,
                    next=rng.random() < 0.7, add=rng.random() < 0.4, pad=pad)
    if op == "dispatch":
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, d=d, k=k, E=E, dtype=dtype,
                    weighted=rng.random() < 0.5, pad=pad)
    return dict(op=op, dir="bwd", T=T, d=d, k=k, E=E, dtype=dtype, weighted=True, pad=pad)


def work(case):
    """Bytes (every input read once, every output written once) and flops."""
    T, e = case["T"], SIZE[case["dtype"]]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        return dict(bytes=N * K // 2 + N * K // GROUP * 2 + 2 * T * K + e * T * N
                    + (4 * N if case["bias"] else 0), flops=2 * T * N * K)
    d = case["d"]
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            return dict(bytes=T * d * (e + 2) + 4 * d, flops=4 * T * d)
        return dict(bytes=T * d * (2 + 3 * e) + 8 * d, flops=10 * T * d)
    k = case["k"]
    P = (T - case["pad"]) * k
    if case["op"] == "block":
        rows = 4 * P * d + 8 * T * k
        add = e * T * d if case["add"] else 0
        small = (4 * d if case["post"] else 0) + {"none": 0, "token": 4 * T,
                                                  "channel": 4 * d}[case["gate"]]
        if case["dir"] == "fwd":
            nxt = 2 * T * d + 4 * d if case["next"] else 0
            return dict(bytes=rows + add + small + nxt + 2 * e * T * d,
                        flops=2 * P * d + 10 * T * d)
        return dict(bytes=rows + add + 2 * small + 2 * e * T * d + (4 if e == 4 else 2) * P * d
                    + 4 * T * k + add, flops=7 * P * d + 12 * T * d)
    if case["op"] == "dispatch":
        if case["dir"] == "fwd":
            return dict(bytes=e * T * d + e * P * d + (8 if case["weighted"] else 4) * T * k,
                        flops=P * d)
        return dict(bytes=e * P * d + e * T * d + 4 * T * k
                    + (e * T * d + 8 * T * k if case["weighted"] else 0), flops=4 * P * d)
    return dict(bytes=4 * P * d + 4 * T * d + e * P * d + 12 * T * k, flops=3 * P * d)


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    T, dt = case["T"], DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        s["x"] = normal(T, K).to(torch.bfloat16)
        s["codes"], s["scales"] = quantized(normal(N, K) / math.sqrt(K))
        s["bias_"] = normal(N) if case["bias"] else None
        return s
    d = case["d"]
    if case["op"] == "norm":
        s["x"] = (normal(T, d) * 3).to(dt)
        s["gain"] = 1 + 0.2 * normal(d)
        if case["dir"] == "bwd":
            s["dout"], s["dres"] = normal(T, d).to(torch.bfloat16), normal(T, d).to(dt)
        return s
    k = case["k"]
    s["pos"] = grouping(g, T, k, case["E"], case["pad"])
    s["w"] = torch.softmax(normal(T, k), 1)
    if case["op"] == "block":
        s["y"] = normal(T * k, d)
        s["add_"] = normal(T, d).to(dt) if case["add"] else None
        s["res"] = (normal(T, d) * 3).to(dt)
        s["post_gain"] = 1 + 0.2 * normal(d) if case["post"] else None
        s["gate_"] = {"none": None, "token": torch.sigmoid(normal(T)),
                      "channel": 0.5 + 0.1 * normal(d)}[case["gate"]]
        s["next_gain"] = 1 + 0.2 * normal(d) if case["next"] else None
        s["scale"] = 0.75
        s["dout"] = normal(T, d).to(dt)
        return s
    if case["op"] == "dispatch":
        s["x"] = normal(T, d).to(dt)
        s["xs"] = torch.zeros(T * k, d, dtype=dt, device="cuda")
        s["dxs"] = normal(T * k, d).to(dt)
        return s
    s["y"] = normal(T * k, d)
    s["dout"] = normal(T, d)
    s["dy"] = torch.zeros(T * k, d, dtype=dt, device="cuda")
    return s


def quantized(w):
    """Symmetric group-128 int4 codes in the package's tiled order (16-row
    tiles, 64 bytes per row and group; in each 32-bit word the even elements
    in nibbles 0-3, the odd ones in nibbles 4-7) and their fp16 scales."""
    N, K = w.shape
    w = w.view(N, K // GROUP, GROUP)
    scales = (w.abs().amax(2) / 7).to(torch.float16)
    q = torch.round(w / scales.float().unsqueeze(2)).clamp_(-7, 7).to(torch.int32)
    q = q.view(N // 16, 16, K // GROUP, 16, 4, 2).transpose(1, 2) & 15
    shift = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device=w.device)
    words = (q.to(torch.int64) << shift).sum((4, 5))
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return (words.contiguous().view(torch.uint8).view(N, K // 2),
            scales.contiguous().view(torch.int16))


def grouping(g, T, k, E, pad):
    """pair_pos of a routed batch: pair t*k + j's row when pairs are grouped
    by expert; the last `pad` tokens are padding, their pairs dropped (-1)."""
    live = T - pad
    score = torch.rand(live, E, generator=g, device="cuda")
    ids = score.topk(min(k, E), 1).indices.reshape(-1)
    pos = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    order = torch.argsort(ids, stable=True)
    pos[order] = torch.arange(live * k, dtype=torch.int32, device="cuda")
    return pos


# ------------------------------------------------------------------- one pass
def run(s):
    if own:
        return run_own(s)
    return PLAIN[s["op"], s["dir"]](s)


def run_own(s):
    import quantized_mixture_experts_fp32_amd as moe
    out = moe.MOE_OUT_BF16 if s["dtype"] == "bf16" else moe.MOE_OUT_F32
    op, bwd = s["op"], s["dir"] == "bwd"
    if op == "linear":
        return moe.moe_linear_w4(s["x"], s["codes"], s["scales"], bias=s["bias_"], out_dtype=out)
    if op == "norm":
        if bwd:
            return moe.moe_rmsnorm_bwd(s["dout"], s["x"], s["gain"], eps=EPS, dres=s["dres"])
        return moe.moe_rmsnorm(s["x"], s["gain"], eps=EPS)
    if op == "block":
        gate = dict(gate=s["gate_"], gate_mode={"none": moe.MOE_GATE_NONE,
                                                "token": moe.MOE_GATE_TOKEN,
                                                "channel": moe.MOE_GATE_CHANNEL}[s["gate"]])
        if bwd:
            r = moe.moe_combine_residual_bwd(s["dout"], s["y"], s["pos"], s["w"], add=s["add_"],
                                             post_gain=s["post_gain"], res_scale=s["scale"],
                                             eps=EPS, dy_dtype=out, **gate)
            return dict(dy=live_rows(r.dy_pairs, s), dw=r.dtopk_w, dadd=r.dadd, dres=r.dresidual,
                        dgain=r.dpost_gain, dgate=r.dgate)
        return moe.moe_combine_residual(s["res"], s["y"], s["pos"], s["w"], add=s["add_"],
                                        post_gain=s["post_gain"], res_scale=s["scale"], eps=EPS,
                                        next_gain=s["next_gain"], **gate)
    w = s["w"] if s["weighted"] else None
    if op == "dispatch":
        if bwd:
            return moe.moe_dispatch_bwd(s["dxs"], s["pos"], s["k"], x=s["x"] if s["weighted"]
                                        else None, topk_w=w)
        return moe.moe_dispatch(s["x"], s["pos"], s["k"], topk_w=w, out=s["xs"])
    return moe.moe_combine_bwd(s["dout"], s["y"], s["pos"], w, dy_dtype=out, dy_pairs=s["dy"])


def live_rows(rows, s):
    """The rows that a pair owns: those of dropped pairs come last and hold
    whatever the buffer held."""
    return rows[:(s["T"] - s["pad"]) * s["k"]]


# ------------------------------------------------------------ the plain forms
def dequantized(codes, scales):
    N, K = codes.shape[0], codes.shape[1] * 2
    words = codes.view(torch.int32).view(N // 16, K // GROUP, 16, 16, 1)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=codes.device, dtype=torch.int32)
    q = (words >> shift) & 15
    q = (q - 16 * (q >= 8).to(torch.int32)).transpose(1, 2).reshape(N, K // GROUP, GROUP)
    return (q.float() * scales.view(torch.float16).float().unsqueeze(2)).view(N, K)


def plain_linear(s):
    y = s["x"].float() @ dequantized(s["codes"], s["scales"]).t()
    if s["bias_"] is not None:
        y = y + s["bias_"]
    return y.to(DTYPES[s["dtype"]])


def normalised(x):
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def plain_norm(s):
    return (normalised(s["x"].float()) * s["gain"]).to(torch.bfloat16)


def norm_gradient(dn, x):
    """Gradient of normalised(x) against x, for the gradient dn of its result."""
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    h = x * r
    return r * (dn - h * (dn * h).mean(1, keepdim=True)), h


def plain_norm_bwd(s):
    x, dout = s["x"].float(), s["dout"].float()
    dx, h = norm_gradient(dout * s["gain"], x)
    return (dx + s["dres"].float()).to(s["x"].dtype), (dout * h).sum(0)


def pair_rows(rows, s):
    """rows[pair_pos] as [T][k][d] in fp32, zero where a pair is dropped."""
    pos = s["pos"].long()
    got = rows.index_select(0, pos.clamp_min(0)).float()
    got = torch.where((pos >= 0).unsqueeze(1), got, torch.zeros((), device=got.device))
    return got.view(s["T"], s["k"], -1)


def scattered(values, into, s):
    """values [T][k][d] written to the rows their pairs own, others left."""
    pos = s["pos"].long()
    live = pos >= 0
    into[pos[live]] = values.reshape(pos.numel(), -1)[live].to(into.dtype)
    return into


def block_output(s):
    o = (pair_rows(s["y"], s) * s["w"].unsqueeze(2)).sum(1)
    return o + s["add_"].float() if s["add_"] is not None else o


def gate_of(s):
    g = s["gate_"]
    return 1.0 if g is None else g.unsqueeze(1) if s["gate"] == "token" else g


def plain_block(s):
    n = block_output(s)
    if s["post_gain"] is not None:
        n = normalised(n) * s["post_gain"]
    r = s["scale"] * s["res"].float() + gate_of(s) * n
    nxt = None
    if s["next_gain"] is not None:
        nxt = (normalised(r) * s["next_gain"]).to(torch.bfloat16)
    return r.to(DTYPES[s["dtype"]]), nxt


def plain_block_bwd(s):
    dt = DTYPES[s["dtype"]]
    o, dr = block_output(s), s["dout"].float()
    dn = gate_of(s) * dr
    do, n, dgain = dn, o, None
    if s["post_gain"] is not None:
        do, h = norm_gradient(dn * s["post_gain"], o)
        n, dgain = h * s["post_gain"], (dn * h).sum(0)
    dgate = {"none": None, "token": 1, "channel": 0}[s["gate"]]
    dgate = None if dgate is None else (dr * n).sum(dgate)
    dw = (pair_rows(s["y"], s) * do.unsqueeze(1)).sum(2)
    dy = torch.empty(s["T"] * s["k"], s["d"], dtype=dt, device=o.device)
    dy = scattered(s["w"].unsqueeze(2) * do.unsqueeze(1), dy, s)
    return dict(dy=live_rows(dy, s), dw=dw, dadd=do.to(dt) if s["add_"] is not None else None,
                dres=(s["scale"] * dr).to(dt), dgain=dgain, dgate=dgate)


def plain_dispatch(s):
    x = s["x"].float().unsqueeze(1).expand(-1, s["k"], -1)
    return scattered(x * s["w"].unsqueeze(2) if s["weighted"] else x, s["xs"], s)


def plain_dispatch_bwd(s):
    rows = pair_rows(s["dxs"], s)
    if not s["weighted"]:
        return rows.sum(1).to(s["dxs"].dtype), None
    return ((rows * s["w"].unsqueeze(2)).sum(1).to(s["dxs"].dtype),
            (rows * s["x"].float().unsqueeze(1)).sum(2))


def plain_combine_bwd(s):
    dout = s["dout"].float().unsqueeze(1)
    return (scattered(s["w"].unsqueeze(2) * dout, s["dy"], s), (pair_rows(s["y"], s) * dout).sum(2))


PLAIN = {("linear", "fwd"): plain_linear, ("norm", "fwd"): plain_norm,
         ("norm", "bwd"): plain_norm_bwd, ("block", "fwd"): plain_block,
         ("block", "bwd"): plain_block_bwd, ("dispatch", "fwd"): plain_dispatch,
         ("dispatch", "bwd"): plain_dispatch_bwd, ("combine", "bwd"): plain_combine_bwd}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    T = case["T"]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        # nibble n of a word (n = 2 * byte + half) holds element 2n of its
        # eight for n < 4 and 2n - 7 above
        b = s["codes"].view(N // 16, K // GROUP, 16, 16, 4)
        nib = torch.stack((b & 15, b >> 4), 5).flatten(4)
        at = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device="cuda")
        v = nib.index_select(4, at).to(torch.int8)
        v = torch.where(v > 7, v - 16, v).permute(0, 2, 1, 3, 4).reshape(N, K // GROUP, GROUP)
        W = (v.to(f64) * s["scales"].view(torch.float16).to(f64)[..., None]).reshape(N, K)
        y = torch.matmul(s["x"].to(f64), W.t().contiguous())
        return y if s["bias_"] is None else y + s["bias_"].to(f64)
    d = case["d"]
    if case["op"] == "norm":
        x, gain = s["x"].to(f64), s["gain"].to(f64)
        rms = ((x ** 2).sum(1) / d + EPS).sqrt()[:, None]
        if case["dir"] == "fwd":
            return x / rms * gain
        v = s["dout"].to(f64)
        a = ((v * gain) * x).sum(1)[:, None] / d
        return s["dres"].to(f64) + v * gain / rms - x * a / rms ** 3, (v * x / rms).sum(0)
    k = case["k"]
    pos = s["pos"].to(torch.int64).view(T, k)
    live = (pos >= 0).to(f64)
    at = torch.where(pos < 0, 0, pos)
    w = s["w"].to(f64)
    count = (T - case["pad"]) * k
    owner = torch.zeros(T * k, dtype=torch.int64, device="cuda")
    flat = pos.reshape(-1)
    owner[flat[flat >= 0]] = torch.nonzero(flat >= 0)[:, 0]
    token, rank = owner // k, owner % k
    if case["op"] == "block":
        o = torch.zeros(T, d, dtype=f64, device="cuda")
        for j in range(k):
            o += (w[:, j] * live[:, j])[:, None] * s["y"][at[:, j]].to(f64)
        if s["add_"] is not None:
            o += s["add_"].to(f64)
        gate = torch.ones(1, 1, dtype=f64, device="cuda")
        if case["gate"] != "none":
            gate = s["gate_"].to(f64)
            gate = gate[:, None] if case["gate"] == "token" else gate[None, :]
        post = s["post_gain"].to(f64) if case["post"] else 1.0
        rms = ((o ** 2).sum(1) / d + EPS).sqrt()[:, None] if case["post"] else 1.0
        if case["dir"] == "fwd":
            r = s["scale"] * s["res"].to(f64) + gate * post * o / rms
            if not case["next"]:
                return r, None
            return r, r / ((r ** 2).sum(1) / d + EPS).sqrt()[:, None] * s["next_gain"].to(f64)
        dr = s["dout"].to(f64)
        u = dr * gate * post / rms
        do = u - o * ((u * o).sum(1)[:, None] / d) / rms ** 2 if case["post"] else u
        dw = torch.stack([(do * s["y"][at[:, j]].to(f64)).sum(1) * live[:, j] for j in range(k)], 1)
        dg = dr * post * o / rms
        return dict(dy=(do * 1.0)[token[:count]] * w[token[:count], rank[:count]][:, None], dw=dw,
                    dadd=do if case["add"] else None, dres=s["scale"] * dr,
                    dgain=(dr * gate * o / rms).sum(0) if case["post"] else None,
                    dgate={"none": None, "token": dg.sum(1), "channel": dg.sum(0)}[case["gate"]])
    if case["op"] == "dispatch":
        if case["dir"] == "fwd":
            out = torch.zeros(T * k, d, dtype=f64, device="cuda")
            out[:count] = s["x"].to(f64)[token[:count]]
            if case["weighted"]:
                out[:count] *= w[token[:count], rank[:count]][:, None]
            return out
        dx = torch.zeros(T, d, dtype=f64, device="cuda")
        for j in range(k):
            f = live[:, j] * w[:, j] if case["weighted"] else live[:, j]
            dx += f[:, None] * s["dxs"][at[:, j]].to(f64)
        if not case["weighted"]:
            return dx, None
        x = s["x"].to(f64)
        return dx, torch.stack([(x * s["dxs"][at[:, j]].to(f64)).sum(1) * live[:, j]
                                for j in range(k)], 1)
    dout = s["dout"].to(f64)
    dy = torch.zeros(T * k, d, dtype=f64, device="cuda")
    dy[:count] = dout[token[:count]] * w[token[:count], rank[:count]][:, None]
    return dy, torch.stack([(dout * s["y"][at[:, j]].to(f64)).sum(1) * live[:, j]
                            for j in range(k)], 1)
