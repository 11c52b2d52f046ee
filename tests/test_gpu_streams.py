"""Calls on a given stream whose tensors are dropped as soon as they return.

The stream is kept busy first, so the kernels run after the caller's own stream
has allocated and filled memory of the same sizes; the allocator may not have
handed it the dropped tensors' blocks.
"""

import numpy as np
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


def calls(arcs):
    """name -> (make(): fresh inputs, call(inputs, stream): tuple of outputs)"""
    import torch
    from workloads import make_params
    gen = lambda seed: torch.Generator(device="cuda").manual_seed(seed)
    B, V, D, G = 40, 6000, 256, 64

    def logits():
        return (torch.randn(B, V, generator=gen(1), device="cuda") * 3).to(torch.bfloat16)

    def head():
        g = gen(2)
        h = torch.randn(B, D, generator=g, device="cuda").to(torch.bfloat16)
        w = (torch.randn(V, D, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
        t = torch.randint(0, V, (B,), generator=g, device="cuda").to(torch.int32)
        return [h, w, t, torch.full((B,), 8.0, device="cuda"), torch.ones(B, device="cuda")]

    def packed():
        g = gen(3)
        return [torch.randn(B, D, generator=g, device="cuda").to(torch.bfloat16),
                torch.randint(0, 256, (V, D // 2), generator=g, device="cuda").to(torch.uint8),
                torch.rand(V, D // G, generator=g, device="cuda"),
                torch.randint(0, 16, (V, D // G), generator=g, device="cuda").to(torch.uint8)]

    def params():
        return arcs.params_to_device(make_params(B, temperature=0.9, top_p=0.95))

    return {
        "argmax": (lambda: [logits()], lambda x, s: (arcs.argmax(*x, stream=s),)),
        "top_logprobs": (lambda: [logits()], lambda x, s: arcs.top_logprobs(*x, 5, stream=s)),
        "sample": (lambda: [logits(), params()], lambda x, s: (arcs.sample(*x, seed=3, stream=s),)),
        "sample_keyed": (lambda: [logits(), params(), arcs.make_key(5, 1)],
                         lambda x, s: (arcs.sample_keyed(*x, stream=s),)),
        "w4_logits": (packed, lambda x, s: (arcs.w4_logits(*x[:3], G, zeros=x[3], stream=s),)),
        "linear_cross_entropy": (head, lambda x, s: arcs.linear_cross_entropy(*x[:3], stream=s)),
        "linear_cross_entropy_backward": (head, lambda x, s: arcs.linear_cross_entropy_backward(*x, stream=s)),
    }


NAMES = ("argmax", "top_logprobs", "sample", "sample_keyed", "w4_logits", "linear_cross_entropy",
         "linear_cross_entropy_backward")


def refill(sizes, stream=None):
    """Takes blocks of these sizes, as often as a pool may hold them, and fills them."""
    import torch
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream()):
        return [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]


@pytest.mark.parametrize("name", NAMES)
def test_inputs_dropped_after_the_call(arcs, name):
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
    junk = refill(sizes)
    side.synchronize()
    for got, ref in zip(out, want):
        assert torch.equal(got, ref)
    del junk


@pytest.mark.parametrize("name", ("w4_logits", "linear_cross_entropy", "linear_cross_entropy_backward"))
def test_outputs_dropped_after_use_on_the_current_stream(arcs, name):
    import torch
    make, call = calls(arcs)[name]
    x = make()
    want = [t.clone() for t in call(x, None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(x, side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in out]
    sizes = [t.numel() * t.element_size() for t in out]
    del out
    junk = refill(sizes, side)
    torch.cuda.synchronize()
    for got, ref in zip(copies, want):
        assert torch.equal(got, ref)
    del junk


def test_a_stream_is_told_of_every_tensor(arcs, monkeypatch):
    """record_stream is called for inputs and for outputs, on the given stream and, for
    outputs, on the current one; and for nothing when no stream is given."""
    import torch
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append((t.data_ptr(), s.cuda_stream)))
    make, call = calls(arcs)["linear_cross_entropy_backward"]
    x = make()
    call(x, None)
    assert not seen
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = call(x, side)
    side.synchronize()
    here = torch.cuda.current_stream().cuda_stream
    assert {(t.data_ptr(), side.cuda_stream) for t in [*x, *out]} <= set(seen)
    assert {(t.data_ptr(), here) for t in out} <= set(seen)
