"""The buffers that a layer keeps between steps: one set per batch size and
stream, from that stream's memory, and a set of its own for every recorded
step.  On the CPU the rule is checked with the stream stood in for; on the GPU
steps change batch size and stream, and graphs replay beside eager steps.  The
calls that create results and workspaces take them from their stream too."""
import contextlib
import inspect

import pytest
import torch

import quantized_mixture_experts_fp32_amd as moe

DEV = "cuda:0"
NAMES = ("topk_idx", "topk_w", "offsets", "sorted_pair", "pair_pos", "ws_rp", "ws_ffn",
         "ws_layer", "y_pairs")


# ------------------------------------------------------------------ the rule
@pytest.fixture
def stream(monkeypatch):
    """Stands in for the stream: [handle, whether it records a graph]."""
    now = [7, False]
    monkeypatch.setattr(moe, "_launch_stream", lambda: tuple(now))
    return now


def host_layer():
    return moe.MoeLayer(torch.zeros(8, 128), None, 2, 128, None, None, None, None)


def held(layer, T):
    layer._buffers(T, layer.wr)
    assert layer.topk_w.shape == (T, 2) and layer.y_pairs.shape == (2 * T, 128)
    return [getattr(layer, n) for n in NAMES]


def same(a, b):
    return [x is y for x, y in zip(a, b)]


def test_buffers_stay_while_batch_and_stream_do(stream):
    layer = host_layer()
    first = held(layer, 4)
    assert all(same(first, held(layer, 4)))
    assert not any(same(first, held(layer, 5)))
    four = held(layer, 4)
    stream[0] = 8
    side = held(layer, 4)
    assert not any(same(four, side)) and all(same(side, held(layer, 4)))


def test_recorded_steps_have_buffers_of_their_own(stream):
    layer = host_layer()
    eager = held(layer, 4)
    stream[1] = True
    graphs = [held(layer, 4) for _ in range(2)]
    stream[1] = False
    after = held(layer, 4)
    sets = [eager, *graphs, after]
    for i, a in enumerate(sets):
        for b in sets[i + 1:]:
            assert not any(same(a, b))
    assert all(same(after, held(layer, 4)))


def test_buffers_are_made_again_after_a_failed_allocation(stream, monkeypatch):
    layer = host_layer()
    held(layer, 4)
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda *a, **kw: (_ for _ in ()).throw(MemoryError()))
        with pytest.raises(MemoryError):
            layer._buffers(5, layer.wr)
    held(layer, 5)
    held(layer, 4)


class AnyCall:
    """Stands in for the library: every call succeeds, sizes are 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("_bytes") else 0


Z = torch.zeros
CALLS = {
    "moe_route": (Z(4, 128), Z(8, 128), None, 2),
    "moe_permute": (Z(4, 2, dtype=torch.int32), 8),
    "moe_route_permute": (Z(4, 128), Z(8, 128), None, 2),
    "moe_expert_ffn_wq": (Z(4, 128), Z(9), Z(8), 2, 128, None, None, None, None),
    "moe_combine": (Z(8, 128), Z(8), Z(4, 2)),
    "moe_bp_distortion": (Z(8, 8), None, None, None, 128, 128),
    "moe_allocate_bits": (Z(8, 8), Z(8), 128, 128, 2, 8, 1000),
    "moe_quantize_w4": (Z(1, 16, 128),),
    "moe_quantize_bitplane8": (Z(1, 16, 128),),
    "moe_retile_w4": (Z(1, 16, 64), 16, 128),
    "moe_retile_bitplane8": (Z(1, 8, 16, 16), 16, 128),
}


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_creates_is_the_given_streams(name, monkeypatch):
    """Results and workspaces are allocated while the given stream is current,
    whether it is given by name or by position."""
    class Stream:
        cuda_stream, device = 1234, torch.device("cuda:0")

    side, now, made = Stream(), [], []

    @contextlib.contextmanager
    def launch_on(stream, values):
        now.append(stream)
        yield
        now.pop()

    empty = torch.empty

    def watched(*args, **kw):
        made.append(list(now))
        return empty(*args, **kw)

    monkeypatch.setattr(moe, "load_library", AnyCall)
    monkeypatch.setattr(moe, "_launch_on", launch_on)
    monkeypatch.setattr(torch, "empty", watched)
    call = getattr(moe, name)
    call(*CALLS[name], stream=side)
    assert made and all(m == [side] for m in made), made
    made.clear()
    names = list(inspect.signature(call).parameters)
    rest = [inspect.signature(call).parameters[n].default for n in names[len(CALLS[name]):-1]]
    call(*CALLS[name], *rest, side)
    assert made and all(m == [side] for m in made), made


# ------------------------------------------------------------------ on the GPU
def note(msg):
    print(msg, flush=True)


class Layer:
    def __init__(self, seed, d=512, E=8, k=2, f=256):
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, dtype=torch.float32):
            return torch.randn(*shape, generator=g).to(dtype).to(DEV)

        self.normal, self.d = normal, d
        gu = moe.moe_quantize_w4((normal(E, 2 * f, d) / d ** 0.5).contiguous())
        dn = moe.moe_quantize_w4((normal(E, d, f) / f ** 0.5).contiguous())
        wr = (normal(E, d) / d ** 0.5).to(torch.bfloat16)
        self.make = lambda: moe.MoeLayer(wr, None, k, f, *gu, *dn)
        self.gain = 1 + 0.2 * normal(d)
        self.kw = dict(gain=self.gain, post_gain=self.gain, next_gain=self.gain, eps=1e-5)

    def rows(self, T):
        return self.normal(T, self.d, dtype=torch.bfloat16)


def churn(products=6):
    """Takes, writes and drops memory of the current stream's while it has
    work in flight: whatever else used that memory would be overwritten."""
    busy = torch.ones(1024, 1024, device=DEV)
    for _ in range(products):
        busy = busy @ busy * 1e-3
        for n in (64, 4096, 1 << 17, 1 << 20):
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0x7F)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["block", "forward", "steps", "bind"])
def test_side_stream_with_changing_batches(call):
    """Prompt and token steps in turn on a side stream, while the default
    stream takes and writes memory: equal to the same steps in order."""
    note(f"side stream, changing batches: {call}")
    L = Layer(1)
    sizes = [37, 1, 150, 1, 37, 8]
    res = [L.rows(T) for T in sizes]

    def step(layer, r, stream=None):
        if call == "block":
            return layer.forward_block(r, stream=stream, **L.kw)
        if call == "forward":
            return (layer.forward(r, stream=stream),)
        if call == "steps":
            return (layer.forward_steps(r, stream=stream),)
        with torch.cuda.stream(stream):  # (None: the current one)
            out = torch.empty_like(r)
        return (layer.bind(r, out, stream=stream)(),)

    layer = L.make()
    want = [step(layer, r) for r in res]
    torch.cuda.synchronize()
    layer, side = L.make(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for r in res:
        churn()
        got.append(step(layer, r, side))
        churn()
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        for a, b in zip(w, o):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("warm", [False, True])
def test_graph_replays_beside_steps_of_other_batches(warm):
    """A captured token step replays while eager steps of the same layer
    change the batch size and what they dropped is written over."""
    note(f"graph beside other batches, warm {warm}")
    L = Layer(2)
    token, prompt = L.rows(1), L.rows(150)
    layer = L.make()
    if warm:
        layer.forward_block(token, **L.kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.forward_block(token, **L.kw)
    other = L.make()
    want = [other.forward_block(r, **L.kw) for r in (token, prompt)]
    for _ in range(3):
        eager = layer.forward_block(prompt, **L.kw)
        again = layer.forward_block(token, **L.kw)
        churn()
        for t in got:
            t.fill_(-3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(got, again, want[0]):
            assert torch.equal(a, c) and torch.equal(b, c)
        for a, b in zip(eager, want[1]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_bound_step_and_captured_step_outlive_a_change_of_batch():
    note("bound and captured steps after a change of batch")
    L = Layer(3)
    token, prompt = L.rows(4), L.rows(150)
    layer = L.make()
    want = L.make().forward(token)
    outs = [torch.empty_like(token) for _ in range(2)]
    bound = layer.bind(token, outs[0])
    graph = layer.capture(token, outs[1])
    for _ in range(3):
        layer.forward(prompt)
        churn()
        for o in outs:
            o.fill_(-3.0)
        torch.cuda.synchronize()
        bound()
        graph.replay()
        churn()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.gpu
def test_two_graphs_of_one_layer_on_two_streams():
    """Two recorded steps of one layer replayed at once do not meet."""
    note("two graphs of one layer on two streams")
    L = Layer(4)
    xs = [L.rows(37) for _ in range(2)]
    layer = L.make()
    want = [L.make().forward_block(x, **L.kw) for x in xs]
    graphs, got = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            got.append(layer.forward_block(x, **L.kw))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(8):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            for a, b in zip(w, o):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_block_on_two_streams_in_turn():
    """One layer on two streams without any order between them."""
    note("one layer on two streams in turn")
    L = Layer(5)
    xs = [L.rows(150) for _ in range(2)]
    want = [L.make().forward_block(x, **L.kw) for x in xs]
    layer, streams = L.make(), [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for x, s in zip(xs, streams):
            got.append(layer.forward_block(x, stream=s, **L.kw))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        for a, b in zip(want[i % 2], o):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_calls_on_a_side_stream_keep_their_own_memory():
    """Grouping and combine on a side stream with workspaces of their own,
    while the default stream takes and writes memory."""
    note("calls on a side stream")
    T, d, k, E = 150, 512, 4, 8
    g = torch.Generator().manual_seed(6)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    ids = ids.to(torch.int32).to(DEV)
    y = torch.randn(T * k, d, generator=g).to(DEV)
    w = torch.softmax(torch.randn(T, k, generator=g), 1).to(DEV)

    def step(stream=None):
        off, sp, pos = moe.moe_permute(ids, E, stream=stream)
        churn(1)
        return off, sp, pos, moe.moe_combine(y, pos, w, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        churn()
        got = step(side)
        churn()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
