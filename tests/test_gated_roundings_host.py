"""CPU tests of the checks in gated_roundings: they take the arithmetic that the calls
of the gated block state, and refuse mistakes and roundings beside it."""
import pytest
import torch

import gated_roundings as gr

BF16, F64 = torch.bfloat16, torch.float64
SIZES = [(640, 136, 264), (1477, 40, 72), (130, 264, 520)]


def random_inputs(T, d, f, seed=0):
    g = torch.Generator().manual_seed(seed + T + d + f)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=n(T, d).to(BF16), w=(n(2 * f, d) * 2 * d ** -0.5).to(BF16),
                v=(n(d, f) * f ** -0.5).to(BF16), dout=n(T, d).to(BF16))


def models(p, kept, dw_f32):
    q = {k: m.to(F64) for k, m in p.items()}
    return {"out": gr.out_of(q["x"], q["w"], q["v"], False),
            **gr.gradients_of(q["dout"], q["x"], q["w"], q["v"],
                              None if kept is None else kept.to(F64), dw_f32)}


def refused(p, kept, dw_f32, wrong):
    """The results that the check of random roundings refuses."""
    want, bad = models(p, kept, dw_f32), []
    for name, got in gr.emulated(p, kept, dw_f32, wrong).items():
        try:
            gr.check(name, got, want[name])
        except AssertionError:
            bad.append(name)
    return bad


def kept_of(p):
    return (p["x"].float() @ p["w"].float().t()).to(BF16)


@pytest.mark.parametrize("T,d,f", SIZES)
@pytest.mark.parametrize("dw_f32", [False, True])
@pytest.mark.parametrize("kept", [False, True])
def test_the_stated_arithmetic_is_taken(T, d, f, dw_f32, kept):
    for seed in range(4):
        p = random_inputs(T, d, f, seed)
        k = kept_of(p) if kept else None
        if kept:  # (out is of the unrounded pre-activations)
            want = models(p, k, dw_f32)
            got = gr.emulated(p, k, dw_f32)
            for name in ("dx", "dw_gate_up", "dw_down"):
                gr.check(name, got[name], want[name])
        else:
            assert refused(p, k, dw_f32, "") == []


GRADS = {"dx", "dw_gate_up", "dw_down"}


@pytest.mark.parametrize("T,d,f", SIZES)
@pytest.mark.parametrize("dw_f32", [False, True])
@pytest.mark.parametrize("wrong,seen", [
    ("bf16 pre-activations", GRADS | {"out"}),
    ("bf16 dh", {"dx", "dw_gate_up"}),
    ("8-bit h", {"out", "dw_down"}),
    ("8-bit dg and du", {"dx", "dw_gate_up"}),
    ("last features dropped", {"out", "dx"}),
    ("last token dropped", {"dw_gate_up", "dw_down"}),
    ("bf16 sums of splits", {"dw_gate_up", "dw_down"}),
])
def test_mistakes_are_refused(T, d, f, dw_f32, wrong, seen):
    assert set(refused(random_inputs(T, d, f), None, dw_f32, wrong)) == seen


@pytest.mark.parametrize("T,d,f", SIZES)
def test_a_checkpoint_rounded_throughout_is_refused(T, d, f):
    """Rows that are not bf16's, rounded before the pre-activations too."""
    p = random_inputs(T, d, f)
    g = torch.Generator().manual_seed(T)
    rows = p["x"].to(F64) * (1 + torch.rand(T, d, generator=g, dtype=F64))
    p["x"] = rows.to(BF16)
    want = gr.gradients_of(*(t.to(F64) for t in (p["dout"], rows, p["w"], p["v"])), None, True,
                           p["x"].to(F64))
    got = gr.emulated(p, dw_f32=True)
    for name in GRADS:
        with pytest.raises(AssertionError, match=name):
            gr.check(name, got[name], want[name])


@pytest.mark.parametrize("T,d,f", SIZES + [(1, 8, 8), (5, 16, 8)])
def test_exact_data(T, d, f):
    """The stated arithmetic gives the exact results, whatever the order of a sum."""
    p = gr.exact_inputs(T, d, f)
    want, kept = gr.exact_results(p), kept_of(p)
    assert torch.equal(kept.to(F64), want["gate_up"])
    for k in (None, kept):
        for f32 in (False, True):
            got = gr.emulated(p, k, f32)
            for name in ("out", "dx", "dw_gate_up", "dw_down"):
                y = want[name].float()
                assert torch.equal(got[name], y if f32 and name[:2] == "dw" else
                                   y.to(BF16).float()), name


@pytest.mark.parametrize("wrong,seen", [
    ("last token dropped", ("dw_gate_up", "dw_down")),
    ("bf16 sums of splits", ("dw_gate_up", "dw_down")),
    ("last features dropped", ("out", "dx")),
])
def test_exact_data_shows_mistakes(wrong, seen):
    for T, d, f in [(640, 136, 264), (4118, 232, 72), (7214, 8, 320)]:
        p = gr.exact_inputs(T, d, f)
        want, got = gr.exact_results(p), gr.emulated(p, dw_f32=True, wrong=wrong)
        for name in seen:
            assert not torch.equal(got[name].to(F64), want[name]), (name, T)
