"""The experts' prefill kernels at counts that leave lane groups, token blocks
and whole tiles without rows, element by element against 64 bits."""
import pytest
import torch

import block_ref as ref
import quantized_mixture_experts_fp32_amd as moe
from block_ref import f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def product(x, ex, codes, scales):
    """x W'^T for values x known up to ex, and the bound of its evaluation in
    one running total: per group 128 products and 3 parts of the offset's sum,
    each counted twice (an MFMA may cut its products at the largest), 4 for the
    step to the group's unit; the group sums' own 128; terms up to 440 / 8 |s x|."""
    y, _ = ref.linear(x, codes, scales)
    N, G = codes.shape[-2], x.shape[1] // 128
    s = scales.reshape(N, G).view(torch.float16).double().abs()
    ax = (x.abs() + ex).reshape(-1, G, 128).sum(2)
    W = ref.dequantize_w4(codes, scales).abs()
    roundings = G * (2 * (128 + 3) + 4) + 132
    return y, (ref.U * roundings * 55 * (ax @ s.t().contiguous())
               + ex @ W.t().contiguous())


@pytest.mark.parametrize("counts", [(1, 4, 33, 36, 97, 0, 128, 129), (5, 31, 32, 64, 65, 3, 2, 127),
                                    (0, 0, 1, 0, 0, 0, 0, 161)])
def test_ragged_experts(counts):
    print(f"ragged experts {counts}", flush=True)
    E, d, f, T = len(counts), 256, 384, sum(counts)
    g = torch.Generator().manual_seed(sum(counts) + counts[1])
    normal = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    gu = moe.moe_quantize_w4((normal(E, 2 * f, d) / d ** 0.5).contiguous())
    dn = moe.moe_quantize_w4((normal(E, d, f) / f ** 0.5).contiguous())
    x = normal(T, d).to(torch.bfloat16)
    offsets = torch.tensor([0, *counts]).cumsum(0).to(torch.int32).to(DEV)
    order = torch.randperm(T, generator=g).to(torch.int32).to(DEV)
    y = torch.full((T + 8, d), -7.0, device=DEV)
    moe.moe_expert_ffn_wq(x, offsets, order, 1, f, *gu, *dn, y_pairs=y[:T],
                          path=moe.MOE_PATH_PREFILL)
    torch.cuda.synchronize()
    assert (y[T:] == -7.0).all()
    at = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        xe = f64(x)[order[at:at + n].long()]
        both, err = product(xe, torch.zeros_like(xe), gu[0][e], gu[1][e])
        (a, b), (ea, eb) = both.split(f, 1), err.split(f, 1)
        silu = a * torch.sigmoid(a)
        h = silu * b
        # |silu'| < 1.1; h is rounded to bf16, 8 more fp32 steps for silu
        eh = 1.1 * ea * (b.abs() + eb) + (silu.abs() + 1.1 * ea) * eb
        eh = eh + (h.abs() + eh) * (2.0 ** -8 + 8 * ref.U)
        want, bound = product(h, eh, dn[0][e], dn[1][e])
        off = (f64(y[at:at + n]) - want).abs()
        assert (off <= bound).all(), (e, n, float((off / bound).max()))
        at += n
