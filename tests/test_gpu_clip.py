"""arcs_gradient_norm and arcs_clip_gradients against 64 bits.

Tolerances.  The norm is summed in 64 bits and rounded once to float32: 2^-24 of it (and
2^-40 for the 64-bit sums).  A clipped element is the product in 64 bits rounded to float32,
2^-24, and for bfloat16 outputs once more, 2^-8 (the two together: at most their sum and
product).  The factor's own error (2^-40) is far below.  Elements below the smallest normal number of
the output's type are off by its smallest step.
"""

import numpy as np
import pytest

from _util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


def types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


def tensors(sizes, dtypes, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * 10.0 ** (i % 4 - 2)).to(types()[dtypes[i % len(dtypes)]])
            for i, n in enumerate(sizes)]


def norm_of(ts):
    return float(np.sqrt(np.sum([float((t.double() ** 2).sum()) for t in ts])))


def check_norm(got, want):
    assert got.shape == (1,) and abs(float(got.double()) - want) <= (2.0 ** -24 + 2.0 ** -40) * want


def check_scaled(got, before, scale):
    import torch
    half = torch.finfo(got.dtype).eps / 2
    want = before.double().cpu() * scale
    far = 2.0 ** -24 + half + 2.0 ** -30 if got.dtype == torch.bfloat16 else 2.0 ** -24 + 2.0 ** -38
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    assert ((got.double().cpu() - want).abs() <= far * want.abs() + tiny).all()


LISTS = [[1], [5], [4096], [4097], [0, 3, 0], [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 31, 33, 100, 255, 256, 257], [1000000],
         [4095, 4096, 4097, 8191, 8193, 12289], [333] * 700, [9000000, 1, 70000]]


@pytest.mark.parametrize("dtypes", [["bf16"], ["f32"], ["bf16", "f32", "f32"]])
@pytest.mark.parametrize("sizes", LISTS, ids=[str(i) for i in range(len(LISTS))])
def test_norm_and_clipping(arcs, sizes, dtypes):
    import torch
    ts = tensors(sizes, dtypes, len(sizes))
    before = [t.clone() for t in ts]
    want = norm_of(ts)
    plan = arcs.TensorList(ts)
    check_norm(arcs.gradient_norm(plan), want)
    # above the norm: nothing changes, not a bit
    for most in (want * 1.01, float("inf")):
        check_norm(arcs.clip_gradients(plan, most), want)
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    # to other tensors, of both types
    for o in types().values():
        for most in (want * 0.3, want * 2):
            outs = [torch.full((t.numel(),), 9.0, dtype=o, device="cuda") for t in ts]
            check_norm(arcs.clip_gradients(arcs.TensorList(ts, outs=outs), most), want)
            for a, b in zip(outs, before):
                check_scaled(a, b, min(1.0, most / want)) if most < want else None
                if most > want:
                    assert torch.equal(a, b.to(o))
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    # in place
    check_norm(arcs.clip_gradients(plan, want * 0.3), want)
    for a, b in zip(ts, before):
        check_scaled(a, b, 0.3)


def test_the_same_bits_each_time_and_odd_addresses(arcs):
    """Tensors at every element's alignment in one buffer; what lies between them stays."""
    import torch
    for t in types().values():
        buf = torch.randn(200000, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(t)
        at, views, gaps = 1, [], []
        for i in range(40):
            n = 997 + 13 * i
            views.append(buf[at: at + n])
            gaps.append(at + n)
            at += n + 1 + i % 3
        out = torch.full_like(buf, 5.0)
        outs, at = [], 3
        for v in views:
            outs.append(out[at: at + v.numel()])
            at += v.numel() + 1
        want = norm_of(views)
        plan = arcs.TensorList(views, outs=outs)
        first = arcs.clip_gradients(plan, want / 3)
        kept = out.clone()
        check_norm(first, want)
        for a, b in zip(outs, views):
            check_scaled(a, b, 1 / 3)
        out.fill_(5.0)
        assert torch.equal(arcs.clip_gradients(plan, want / 3), first) and torch.equal(out, kept)
        assert float((out == 5.0).sum()) >= out.numel() - sum(v.numel() for v in views)
        before = buf.clone()
        arcs.clip_gradients(arcs.TensorList(views), want / 3)
        assert torch.equal(buf[gaps], before[gaps]) and torch.equal(buf[:1], before[:1])


def test_large_and_small_values(arcs):
    """Squares past float32's range, and gradients that are nearly nothing."""
    import torch
    x = torch.full((5000,), 2e38, device="cuda")
    norm = arcs.clip_gradients(arcs.TensorList([x]), 1.0)
    assert float(norm) == float("inf")  # 1.4e40 does not fit float32; the gradients are still scaled by it
    check_scaled(x, torch.full((5000,), 2e38), 1.0 / (float(np.float32(2e38)) * np.sqrt(5000.0)))
    y = torch.full((5000,), 1e-38, device="cuda")
    check_norm(arcs.gradient_norm(arcs.TensorList([y])), float(np.float32(1e-38)) * np.sqrt(5000.0))
    z = torch.zeros(100, device="cuda")
    assert float(arcs.clip_gradients(arcs.TensorList([z]), 0.0)) == 0.0 and not z.any()
    w = torch.ones(100, dtype=torch.bfloat16, device="cuda")
    assert float(arcs.clip_gradients(arcs.TensorList([w]), 0.0)) == 10.0 and not w.any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_changes_nothing(arcs, bad):
    import torch
    for t in types().values():
        a, b = torch.ones(10000, device="cuda").to(t), torch.ones(33, device="cuda").to(t)
        b[7] = bad
        want = [a.clone(), b.clone()]
        norm = arcs.clip_gradients(arcs.TensorList([a, b]), 0.5)
        assert not bool(norm.isfinite()) and bool(norm.isnan()) == (bad != bad)
        assert torch.equal(a, want[0]) and torch.equal(b.nan_to_num(3.0), want[1].nan_to_num(3.0))


def test_overlapping_memory_is_refused(arcs):
    import torch
    x = torch.ones(100, device="cuda")
    for ts, outs in (([x, x], None), ([x[:60], x[50:]], None), ([x[:50]], [x[10:60]]), ([x[:50], x[50:]], [x[50:], x[:50]]),
                     ([x], [x.view(torch.bfloat16)[:100]])):
        with pytest.raises((ValueError, arcs.ArcsError)):
            arcs.TensorList(ts, outs=outs)
    with pytest.raises(ValueError):
        arcs.TensorList([x.view(10, 10).t()])
    with pytest.raises(TypeError):
        arcs.TensorList([x.half()])
    with pytest.raises(ValueError):
        arcs.TensorList([])
    with pytest.raises(arcs.ArcsError):
        arcs.clip_gradients(arcs.TensorList([x]), -1.0)
    with pytest.raises(arcs.ArcsError):
        arcs.clip_gradients(arcs.TensorList([x]), float("nan"))


def test_side_stream_and_replays(arcs):
    import torch
    ts = tensors([5000, 3, 70001], ["bf16", "f32"], 4)
    outs = [torch.empty_like(t) for t in ts]
    plan = arcs.TensorList(ts, outs=outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = arcs.clip_gradients(plan, 1.0, stream=side)
    side.synchronize()
    check_norm(norm, norm_of(ts))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        norm = arcs.clip_gradients(plan, 1.0)
    for i in range(4):
        for t in ts:
            t.copy_(torch.randn(t.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(i)))
        want = norm_of(ts)
        eager = arcs.gradient_norm(plan)
        graph.replay()
        torch.cuda.synchronize()
        check_norm(norm, want)
        assert torch.equal(norm, eager)
        for a, b in zip(outs, ts):
            check_scaled(a, b, 1.0 / want)


def test_a_training_step_of_a_block_in_front_of_the_head(arcs):
    """Block, loss over the head, both backward passes and clipping, against 64-bit autograd.

    Every tensor is rounded to bfloat16 between the calls, so the gradients are compared in the
    norm: each has at most six such roundings on its way (block output, dz of the head, dhidden,
    pre, dz of the block, result), each of 2^-8 of its elements, which move a gradient by no more than
    six times 2^-8 of the sums of magnitudes; signs being random, those sums are within
    a factor of 3 of the gradients' own norm at these sizes."""
    import torch
    N, V, D = 90, 700, 128
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)

    h, w, b, head = normal(N, D), normal(D, D, scale=D ** -0.5), normal(D), normal(V, D, scale=2 * D ** -0.5)
    targets = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    x, pre = arcs.linear(h, w, bias=b, activation="silu", residual=h, want_pre=True)
    loss, lse = arcs.linear_cross_entropy(x, head, targets)
    weight = torch.full((N,), 1.0 / N, device="cuda")
    dx, dhead = arcs.linear_cross_entropy_backward(x, head, targets, lse, weight)
    _, dw, db = arcs.linear_backward(h, w, dx, pre=pre, activation="silu", want_hidden=False, want_bias=True)
    leaves = [t.double().requires_grad_(True) for t in (w, b, head)]
    hd = h.double()
    z = torch.nn.functional.linear(hd, leaves[0], leaves[1])
    want = torch.nn.functional.cross_entropy((hd + z * torch.sigmoid(z)) @ leaves[2].t(), targets.long())
    want.backward()
    before = [dw, db, dhead]
    for a, r in zip(before, leaves):
        assert (a.double() - r.grad).norm() <= 6 * 3 * 2.0 ** -8 * r.grad.norm()
    total = norm_of(before)
    outs = [torch.empty(t.shape, device="cuda") for t in before]
    check_norm(arcs.clip_gradients(arcs.TensorList(before, outs=outs), total / 2), total)
    for a, t in zip(outs, before):
        check_scaled(a, t, 0.5)


def test_tensors_without_an_out_count_and_are_not_written(arcs):
    """A plan of the C interface whose first and last tensors have no `out`."""
    import torch
    a, b, c = (torch.full((n,), v, device="cuda") for n, v in ((9000, 2.0), (5000, 3.0), (7, 100.0)))
    records = np.zeros(3, arcs.TENSOR_DTYPE)
    records["data"] = [t.data_ptr() for t in (a, b, c)]
    records["out"] = [0, b.data_ptr(), 0]
    records["count"] = [t.numel() for t in (a, b, c)]
    records["dtype"] = records["out_dtype"] = arcs.DTYPE_F32
    lib = arcs.library()
    size = lib.arcs_gradient_plan_bytes(records.ctypes.data, 3)
    host = np.zeros(size, np.uint8)
    assert lib.arcs_gradient_plan(records.ctypes.data, 3, host.ctypes.data, size) == 0
    plan, norm = torch.from_numpy(host).cuda(), torch.empty(1, device="cuda")
    need = lib.arcs_gradient_workspace_bytes(size)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = float(np.sqrt(9000 * 4.0 + 5000 * 9.0 + 7 * 1e4))
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.arcs_clip_gradients(plan.data_ptr(), size, want / 2, norm.data_ptr(), work.data_ptr(), need, stream) == 0
    check_norm(norm, want)
    assert (a == 2.0).all() and (c == 100.0).all()
    check_scaled(b, torch.full((5000,), 3.0), 0.5)


def test_a_list_of_empty_tensors(arcs):
    import torch
    ts = [torch.empty(0, device="cuda"), torch.empty(0, 5, dtype=torch.bfloat16, device="cuda")]
    plan = arcs.TensorList(ts)
    out = torch.full((1,), 7.0, device="cuda")
    assert float(arcs.gradient_norm(plan)) == 0.0 and float(arcs.clip_gradients(plan, 0.0, out_norm=out)) == 0.0 and float(out) == 0.0
