"""The layers around the head on streams of their own: tensors dropped as soon as a call
returns, calls that run at the same time, and two captured graphs replayed at the same time.
"""

import pytest

from _util import ensure_built

pytestmark = pytest.mark.gpu

BUSY = 4_000_000  # cycles, some milliseconds


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


def calls(arcs, seed=1):
    """name -> (make(): fresh inputs, call(inputs, stream): tuple of outputs)"""
    import torch
    from workloads import make_params
    N, V, D = 40, 3001, 264

    def normal(*shape, k=0, t=torch.bfloat16):
        return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(10 * seed + k), device="cuda").to(t)

    def layer(n=N):
        return [normal(n, D), normal(V, D, k=1) / 16, normal(V, k=2), normal(n, V, k=3), normal(n, V, k=4)]

    def odd():
        return [t[:, 1:].contiguous() if t.dim() == 2 and t.shape[1] == D else t for t in layer()]

    def rows():
        ids = torch.randint(0, V, (N * 50,), generator=torch.Generator("cuda").manual_seed(seed), device="cuda", dtype=torch.int32)
        return [normal(N, V), arcs.params_to_device(make_params(N, temperature=0.9, presence=0.5, repetition=1.2)), ids,
                torch.arange(N + 1, device="cuda") * 50, ids.flip(0).contiguous(), normal(N * 50, k=5, t=torch.float32),
                torch.randint(-2**31, 2**31 - 1, (N, (V + 31) // 32), device="cuda", dtype=torch.int32,
                              generator=torch.Generator("cuda").manual_seed(seed))]

    def forward(x, s):
        return arcs.linear(x[0], x[1], bias=x[2], activation="silu", residual=x[3], want_pre=True, stream=s)

    def adjust(x, s):
        return (arcs.adjust_logits(x[0], x[1], hist_ids=x[2], hist_offsets=x[3], bias_ids=x[4], bias_values=x[5],
                                   bias_offsets=x[3], mask=x[6], stream=s),)

    def clip(x, s):
        outs = [torch.empty_like(t) for t in x]
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        norm = arcs.clip_gradients(arcs.TensorList(x, outs=outs), 3.0, stream=s)
        return (norm, *outs)

    return {
        "linear_few": (lambda: layer(9), forward),
        "linear": (layer, forward),
        "linear_odd": (odd, forward),
        "linear_backward": (layer, lambda x, s: arcs.linear_backward(x[0], x[1], x[4], pre=x[3], activation="gelu", want_bias=True, stream=s)),
        "adjust_logits": (rows, adjust),
        "clip_gradients": (lambda: [normal(70000, t=torch.float32), normal(5, k=1), normal(33333, k=2)], clip),
    }


NAMES = ("linear_few", "linear", "linear_odd", "linear_backward", "adjust_logits", "clip_gradients")


def same(got, want):
    import torch
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_inputs_dropped_after_the_call(arcs, name):
    """The stream is kept busy first; what the caller's stream allocates and fills meanwhile is
    not the dropped tensors' memory."""
    import torch
    make, call = calls(arcs)[name]
    want = [t.clone() for t in call(make(), None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    x = make()
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in x] + [1 << 20, 1 << 22]
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out = call(x, side)
    del x
    junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    side.synchronize()
    same(out, want)
    del junk


@pytest.mark.parametrize("name", NAMES)
def test_calls_at_the_same_time(arcs, name):
    """Two streams, other inputs on each, several calls in flight."""
    import torch
    both = [calls(arcs, seed)[name] for seed in (1, 2)]
    x = [make() for make, _ in both]
    want = [[t.clone() for t in call(v, None)] for (_, call), v in zip(both, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, (_, call) in enumerate(both):
            got[i].append(call(x[i], streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            same(out, want[i])


@pytest.mark.parametrize("name", ["linear", "linear_backward", "adjust_logits"])
def test_two_graphs_at_the_same_time(arcs, name):
    """Each graph has its own workspace in its own pool; both are replayed over and over beside
    each other and beside eager calls."""
    import torch
    both = [calls(arcs, seed)[name] for seed in (1, 2)]
    x = [make() for make, _ in both]
    want = [[t.clone() for t in call(v, None)] for (_, call), v in zip(both, x)]
    torch.cuda.synchronize()
    graphs, held = [], []
    for (_, call), v in zip(both, x):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(call(v, None))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for outs in held:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = both[0][1](x[0], None)
        torch.cuda.synchronize()
        same(eager, want[0])
        for outs, ref in zip(held, want):
            same(outs, ref)


def test_a_stream_is_told_of_every_tensor(arcs, monkeypatch):
    """record_stream is called for inputs and outputs on the given stream, and for nothing when no
    stream is given."""
    import torch
    for name in ("linear", "linear_backward", "adjust_logits"):
        make, call = calls(arcs)[name]
        x = make()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with monkeypatch.context() as m:
            seen = []
            m.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append((t.data_ptr(), s.cuda_stream)))
            call(x, None)
            assert not seen
            out = call(x, side)
            side.synchronize()
        used = x if name != "linear" else x[:4]
        used = [t for i, t in enumerate(used) if not (name == "linear_backward" and i == 2)]
        here = torch.cuda.current_stream().cuda_stream
        assert {(t.data_ptr(), side.cuda_stream) for t in [*used, *out]} <= set(seen)
        assert {(t.data_ptr(), here) for t in out} <= set(seen)


def test_a_stream_of_another_device_is_refused(arcs):
    import torch
    if torch.cuda.device_count() < 2:
        class Elsewhere:
            device = torch.device("cuda", 1)
            cuda_stream = 0
        stream = Elsewhere()
    else:
        stream = torch.cuda.Stream(device=1)
    make, call = calls(arcs)["linear"]
    with pytest.raises(ValueError):
        call(make(), stream)
    make, call = calls(arcs)["adjust_logits"]
    with pytest.raises(ValueError):
        call(make(), stream)


def test_views_and_broadcasts(arcs):
    """Strides that the documentation allows, and those it does not."""
    import torch
    g = torch.Generator("cuda").manual_seed(5)
    h, w = torch.randn(30, 64, generator=g, device="cuda"), torch.randn(50, 64, generator=g, device="cuda")
    want = arcs.linear(h, w)
    # every second row of a larger buffer
    wide = torch.full((60, 64), float("nan"), device="cuda")
    wide[::2] = h
    same([arcs.linear(wide[::2], w)], [want])
    for bad in (h.t(), h[:, ::2], h[:1].expand(30, 64), h.double(), h.cpu(), h[0]):
        with pytest.raises((ValueError, TypeError, arcs.ArcsError)):
            arcs.linear(bad, w)
    with pytest.raises((ValueError, arcs.ArcsError)):
        arcs.linear(h, w, bias=torch.zeros(1, device="cuda").expand(50))
    with pytest.raises(arcs.ArcsError):
        arcs.linear_backward(h, w, torch.ones(1, 50, device="cuda").expand(30, 50))
    with pytest.raises(ValueError):
        arcs.linear(h, w, activation="tanh")
    sq = torch.randn(64, 64, generator=g, device="cuda")
    with pytest.raises(arcs.ArcsError):  # in place of the hidden states, which other workgroups read
        arcs.linear(h, sq, residual=h, out=h)
    # one row may have any row stride
    one = torch.randn(3, 64, generator=g, device="cuda")[1:2]
    same([arcs.linear(one.as_strided((1, 64), (7, 1)), w)], [arcs.linear(one.clone(), w)])
    with pytest.raises((ValueError, arcs.ArcsError)):
        arcs.adjust_logits(want[:1].expand(30, 50))
    with pytest.raises((ValueError, arcs.ArcsError)):
        arcs.adjust_logits(want, mask=torch.zeros(30, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises((ValueError, arcs.ArcsError)):
        arcs.adjust_logits(want, mask=torch.zeros(29, 2, dtype=torch.int32, device="cuda"))


def test_a_list_dropped_after_a_call_on_another_current_stream(arcs):
    """The list's plan belongs to the stream that it was made on; a call on another current stream
    keeps it until that stream is through.  (Nothing is written to the memory that is asked for.)"""
    import torch
    x = torch.ones(1_000_000, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plans = arcs.TensorList([x])
    at, size = plans.plan.data_ptr(), plans.plan_bytes
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
        norm = arcs.clip_gradients(plans, 10.0)
    del plans
    others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    busy = not side.query()
    taken = at in [t.data_ptr() for t in others]
    side.synchronize()
    assert busy and not taken
    assert float(norm) == 1000.0 and float(x[0]) == float(x[-1]) == float(torch.tensor(0.01))
