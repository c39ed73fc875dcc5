"""Speed cases of the shared expert's operators: the gated feed-forward block
with its gradient, 8-bit activation checkpoints with the backward passes that
read them, and the linear map in 8-bit integers.

Shapes follow the layers this package is built for (model width d 2048 or
4096, expert width f 1024 or 2048) and the batches they see: one token, decode
batches up to 64, prompts and training batches of thousands of tokens.

`run` computes an operator in plain torch (fp32, rounded once at the end);
with `own` true it makes the package's call.  `exact` computes the same
outputs in fp64, written apart from the plain form.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-5
TINY = 2.0 ** -119  # groups below it are stored as zeros
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the shared expert for one decode token: latency
        forward("gated-token", 1, 2048, 1024, False),
        # a decode batch: the weights' bytes
        forward("gated-decode", 16, 4096, 2048, False),
        # a ragged prompt, pre-activations kept for a training step
        forward("gated-prompt", 2501, 4096, 2048, True),
        # its gradient over a training batch, from kept pre-activations
        backward("gated-train", 4096, 4096, 2048, "saved"),
        # over a ragged batch from an 8-bit checkpoint of the block's input
        backward("gated-train-checkpoint", 4093, 2048, 1024, "checkpoint"),
        # a small tuning batch, nothing kept but the input
        backward("gated-tune", 131, 2048, 1024, "recompute"),
        # a training batch's activations into a checkpoint and back
        trip("checkpoint-train", 8192, 4096, "bf16"),
        # a few rows of a float32 stream, the last group of a row incomplete
        trip("checkpoint-few", 33, 2056, "f32"),
        # gradient of the norm in front of a block, its input from a checkpoint
        dict(name="checkpoint-norm", op="norm", T=8191, d=4096, dtype="bf16"),
        # one decode token through a square projection in 8-bit integers
        linear("i8-token", 1, 2048, 2048, "bf16", False),
        # a decode batch of 64 through a fused projection with bias
        linear("i8-batch", 64, 4096, 12288, "f32", True),
        # a ragged prompt
        linear("i8-prompt", 2501, 4096, 4096, "bf16", False),
    ]


def forward(name, T, d, f, save):
    return dict(name=name, op="gated", T=T, d=d, f=f, save=save, dtype="bf16")


def backward(name, T, d, f, source):
    return dict(name=name, op="gated_bwd", T=T, d=d, f=f, source=source, dtype="bf16")


def trip(name, T, d, dtype):
    return dict(name=name, op="trip", T=T, d=d, dtype=dtype)


def linear(name, T, K, N, dtype, bias):
    return dict(name=name, op="linear", T=T, K=K, N=N, dtype=dtype, bias=bias)


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
    op = rng.choice(["gated", "gated", "gated_bwd", "gated_bwd", "trip", "norm", "linear",
                     "linear"])
    T, dtype = spread(rng, 1, 8192), rng.choice(["bf16", "f32"])
    if op == "linear":
        return dict(op=op, T=T, K=16 * spread(rng, 16, 512), N=8 * spread(rng, 32, 6288),
                    dtype=dtype, bias=rng.random() < 0.5)
    if op in ("trip", "norm"):
        return dict(op=op, T=T, d=8 * spread(rng, 32, 1024), dtype=dtype)
    d, f = 8 * spread(rng, 32, 512), 8 * spread(rng, 16, 512)
    if op == "gated":
        return dict(op=op, T=T, d=d, f=f, save=rng.random() < 0.4, dtype="bf16")
    return dict(op=op, T=T, d=d, f=f, source=rng.choice(["saved", "recompute", "checkpoint"]),
                dtype="bf16")


def checkpoint_bytes(T, d):
    return T * d + 4 * T * -(-d // GROUP)


def work(case):
    """Bytes (every input read once, every output written once) and flops."""
    T, e = case["T"], SIZE[case["dtype"]]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        return dict(bytes=N * K + 4 * N + 2 * T * K + e * T * N + (4 * N if case["bias"] else 0),
                    flops=2 * T * N * K)
    d = case["d"]
    if case["op"] == "trip":  # the checkpoint is written, and read again
        return dict(bytes=2 * e * T * d + 2 * checkpoint_bytes(T, d), flops=4 * T * d)
    if case["op"] == "norm":
        return dict(bytes=checkpoint_bytes(T, d) + T * d * (2 + 2 * e) + 8 * d,
                    flops=11 * T * d)
    f = case["f"]
    if case["op"] == "gated":
        return dict(bytes=6 * d * f + 4 * T * d + (4 * T * f if case["save"] else 0),
                    flops=6 * T * d * f)
    kept = {"saved": 2 * T * d + 4 * T * f, "recompute": 2 * T * d,
            "checkpoint": checkpoint_bytes(T, d)}[case["source"]]
    return dict(bytes=12 * d * f + 4 * T * d + kept,
                flops=(12 if case["source"] == "saved" else 16) * T * d * f)


# ----------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def outlying(*shape):
        """Activations: some channels stand out."""
        return normal(*shape) * (1 + 9 * (torch.rand(shape[-1], generator=g, device="cuda")
                                          < 0.01).float())

    T, dt = case["T"], DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        s["x"] = outlying(T, K).to(torch.bfloat16)
        s["codes"], s["scales"] = quantized(normal(N, K) / math.sqrt(K), K)
        s["bias_"] = normal(N) if case["bias"] else None
        return s
    d = case["d"]
    if case["op"] == "trip":
        s["x"] = (outlying(T, d) * 3).to(dt)
        return s
    if case["op"] == "norm":
        s["codes"], s["scales"] = quantized((outlying(T, d) * 3).to(dt).float(), GROUP)
        s["gain"] = 1 + 0.2 * normal(d)
        s["dout"], s["dres"] = normal(T, d).to(torch.bfloat16), normal(T, d).to(dt)
        return s
    f = case["f"]
    s["x"] = normal(T, d).to(torch.bfloat16)
    s["w_gate_up"] = (normal(2 * f, d) / math.sqrt(d)).to(torch.bfloat16)
    s["w_down"] = (normal(d, f) / math.sqrt(f)).to(torch.bfloat16)
    if case["op"] == "gated_bwd":
        s["dout"] = normal(T, d).to(torch.bfloat16)
        if case["source"] == "saved":
            s["gate_up"] = (s["x"].float() @ s["w_gate_up"].float().t()).to(torch.bfloat16)
        elif case["source"] == "checkpoint":
            s["codes"], s["scales"] = quantized(s.pop("x").float(), GROUP)
    return s


def quantized(x, group):
    """Codes int8 [T][d] and scales fp32 [T][groups] ([T] for one group) of
    groups of `group` values of each row: scale max|x| / 127, code x times
    127 / max|x|, rounded to the nearest (ties to even)."""
    T, d = x.shape
    n = -(-d // group)
    v = torch.nn.functional.pad(x, (0, n * group - d)).view(T, n, group)
    top = v.abs().amax(2)
    top = torch.where(top < TINY, torch.zeros_like(top), top)
    c127 = torch.full_like(top, 127.0)
    scales = top / c127
    inv = torch.where(top > 0, c127 / top, torch.zeros_like(top))
    codes = torch.round(v * inv.unsqueeze(2)).to(torch.int8)
    codes = codes.view(T, n * group)[:, :d].contiguous()
    return codes, (scales.view(T) if group == d else scales.contiguous())


# ------------------------------------------------------------------- one pass
def run(s):
    if own:
        return run_own(s)
    return PLAIN[s["op"]](s)


def run_own(s):
    import quantized_mixture_experts_fp32_amd as moe
    out = moe.MOE_OUT_BF16 if s["dtype"] == "bf16" else moe.MOE_OUT_F32
    if s["op"] == "linear":
        return moe.moe_linear_i8(s["x"], s["codes"], s["scales"], bias=s["bias_"], out_dtype=out)
    if s["op"] == "trip":
        codes, scales = moe.moe_quantize_i8(s["x"])
        return moe.moe_dequantize_i8(codes, scales, out_dtype=out), scales
    if s["op"] == "norm":
        return moe.moe_rmsnorm_bwd(s["dout"], s["codes"], s["gain"], eps=EPS, dres=s["dres"],
                                   x_scales=s["scales"], dx_dtype=out)
    if s["op"] == "gated":
        return moe.moe_gated_ffn(s["x"], s["w_gate_up"], s["w_down"], save=s["save"])
    if s["source"] == "checkpoint":
        x = dict(x=s["codes"], x_scales=s["scales"])
    else:
        x = dict(x=s["x"], gate_up=s.get("gate_up"))
    r = moe.moe_gated_ffn_bwd(s["dout"], w_gate_up=s["w_gate_up"], w_down=s["w_down"], **x)
    return r.dx, r.dw_gate_up, r.dw_down


# ------------------------------------------------------------ the plain forms
def restored(codes, scales):
    if scales.dim() == 1:
        return codes.float() * scales.unsqueeze(1)
    return codes.float() * scales.repeat_interleave(GROUP, 1)[:, :codes.shape[1]]


def plain_linear(s):
    codes, scales = quantized(s["x"].float(), s["K"])
    y = (codes.float() @ s["codes"].float().t()) * (scales.unsqueeze(1) * s["scales"])
    if s["bias_"] is not None:
        y = y + s["bias_"]
    return y.to(DTYPES[s["dtype"]])


def plain_trip(s):
    codes, scales = quantized(s["x"].float(), GROUP)
    return restored(codes, scales).to(DTYPES[s["dtype"]]), scales


def plain_norm(s):
    x, dout = restored(s["codes"], s["scales"]), s["dout"].float()
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    h, u = x * r, dout * s["gain"]
    dx = s["dres"].float() + r * (u - h * (u * h).mean(1, keepdim=True))
    return dx.to(DTYPES[s["dtype"]]), (dout * h).sum(0)


def plain_gated(s):
    f = s["f"]
    gu = s["x"].float() @ s["w_gate_up"].float().t()
    g, u = gu[:, :f], gu[:, f:]
    y = (g * torch.sigmoid(g) * u) @ s["w_down"].float().t()
    return y.to(torch.bfloat16), gu.to(torch.bfloat16) if s["save"] else None


def plain_gated_bwd(s):
    f = s["f"]
    x = restored(s["codes"], s["scales"]) if s["source"] == "checkpoint" else s["x"].float()
    w, dout = s["w_gate_up"].float(), s["dout"].float()
    gu = s["gate_up"].float() if s["source"] == "saved" else x @ w.t()
    g, u = gu[:, :f], gu[:, f:]
    sig = torch.sigmoid(g)
    dh = dout @ s["w_down"].float()
    dgu = torch.cat((dh * u * sig * (1 + g * (1 - sig)), dh * g * sig), 1)
    bf = torch.bfloat16
    return (dgu @ w).to(bf), (dgu.t() @ x).to(bf), (dout.t() @ (g * sig * u)).to(bf)


PLAIN = {"linear": plain_linear, "trip": plain_trip, "norm": plain_norm, "gated": plain_gated,
         "gated_bwd": plain_gated_bwd}


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    T = case["T"]

    def by_groups(v, group):
        """Codes (as fp64) and scales of the rows of v, group after group;
        the codes are defined in fp32, their products are exact in fp64."""
        q, sc = torch.empty_like(v), []
        for i in range(0, v.shape[1], group):
            part = v[:, i:i + group]
            m = part.abs().max(1).values
            live = m >= TINY
            inv = torch.where(live, 127.0 / m, 0.0).to(torch.float32).to(f64)
            q[:, i:i + group] = torch.round((part * inv[:, None]).to(torch.float32)).to(f64)
            sc.append(torch.where(live, m / 127.0, 0.0))
        return q, torch.stack(sc, 1)

    def weighted(q, sc):
        v = q.to(f64).clone()
        for i in range(sc.shape[1]):
            v[:, GROUP * i:GROUP * (i + 1)] *= sc[:, i:i + 1].to(f64)
        return v

    if case["op"] == "linear":
        q, sc = by_groups(s["x"].to(f64), case["K"])
        y = torch.matmul(q, s["codes"].to(f64).t().contiguous())
        y = y * sc * s["scales"].to(f64)[None, :]
        return y if s["bias_"] is None else y + s["bias_"].to(f64)
    if case["op"] == "trip":
        q, sc = by_groups(s["x"].to(f64), GROUP)
        return weighted(q, sc), sc
    if case["op"] == "norm":
        d = case["d"]
        x, gain, v = weighted(s["codes"], s["scales"]), s["gain"].to(f64), s["dout"].to(f64)
        rms = ((x ** 2).sum(1) / d + EPS).sqrt()[:, None]
        a = ((v * gain) * x).sum(1)[:, None] / d
        return s["dres"].to(f64) + v * gain / rms - x * a / rms ** 3, (v * x / rms).sum(0)
    d, f = case["d"], case["f"]
    W, D = s["w_gate_up"].to(f64), s["w_down"].to(f64)
    x = weighted(s["codes"], s["scales"]) if "codes" in s else s["x"].to(f64)
    if "gate_up" in s:
        gate, up = s["gate_up"].to(f64).split(f, 1)
    else:
        gate = torch.matmul(x, W[:f].t().contiguous())
        up = torch.matmul(x, W[f:].t().contiguous())
    e = torch.exp(-gate)
    act = gate / (1 + e)
    if case["op"] == "gated":
        y = torch.matmul(act * up, D.t().contiguous())
        return y, torch.cat((gate, up), 1) if case["save"] else None
    dy = s["dout"].to(f64)
    dh = torch.matmul(dy, D)
    d_up = dh * act
    d_gate = dh * up * (1 / (1 + e) + gate * e / (1 + e) ** 2)
    dx = torch.matmul(d_gate, W[:f].contiguous()) + torch.matmul(d_up, W[f:].contiguous())
    dW = torch.cat((torch.matmul(d_gate.t().contiguous(), x),
                    torch.matmul(d_up.t().contiguous(), x)), 0)
    return dx, dW, torch.matmul(dy.t().contiguous(), act * up)
