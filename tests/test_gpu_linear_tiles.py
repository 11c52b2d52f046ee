"""The linear layer's tile kernels, each of them over several steps of k, every element checked.

On whole numbers small enough that every sum is one that float32 holds, results are the exact ones rounded
once, whatever the order of the sums: a piece of k left out, read twice or read before it has
come shows in the last bit.  With real numbers the tolerances are test_gpu_linear.py's.
"""

import pytest

from _util import ensure_built
from linear_tile_sizes import TILES
from test_gpu_linear import check_backward, check_forward, make, types

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


def whole(g, most, t, *shape):
    import torch
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).to(t)


def times(a, b):
    """a b exactly (the sums stay below 2^24)."""
    return a.double() @ b.double()


@pytest.mark.parametrize("case", TILES, ids=lambda c: "-".join(map(str, c)))
def test_exact_sums(arcs, case):
    import torch
    mode, dtype, N, V, D = case[:5]
    t = types()[dtype]
    g = torch.Generator("cuda").manual_seed(N + V + D)
    h, w = whole(g, 2, t, N, D), whole(g, 2, t, V, D)
    if mode == "forward":
        b, r = whole(g, 3, t, V), whole(g, 9, t, N, V)
        z = times(h, w.T) + b.double()
        y = z.clamp(min=0) + r.double()
        z, wants = z.to(t), [y.to(o) for o in types().values()]
        del y
        for _ in range(2):
            for o, want in zip(types().values(), wants):
                out, pre = arcs.linear(h, w, bias=b, activation="relu", residual=r, out_dtype=o, want_pre=True)
                assert torch.equal(pre, z) and torch.equal(out, want)
        return
    pre, grad = whole(g, 1, t, N, V), whole(g, 1, t, N, V)
    dz = torch.where(pre > 0, grad, torch.zeros_like(grad))
    want = (times(dz, w) if mode == "dhidden" else times(dz.T, h)).to(t)
    del dz
    for _ in range(3):
        dh, dw, _ = arcs.linear_backward(h, w, grad, pre=pre, activation="relu", want_hidden=mode == "dhidden", want_weight=mode == "dweight")
        assert torch.equal(dh if mode == "dhidden" else dw, want)


# sizes whose products take the large tiles, whole and shared, in all three directions
REAL = [("bf16", 1050, 4999, 1016), ("bf16", 1050, 4999, 1015), ("bf16", 2050, 4099, 1032), ("bf16", 513, 2051, 4104), ("bf16", 4097, 4099, 1032),
        ("bf16", 300, 20001, 777), ("f32", 520, 4099, 260), ("f32", 257, 20003, 516), ("f32", 1030, 2049, 1021)]


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype,N,V,D", REAL)
def test_real_numbers(arcs, dtype, N, V, D, act):
    import torch
    t = types()[dtype]
    s = make(N, V, D, t, N + V + D)
    out, pre = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation=act, residual=s["residual"], want_pre=True)
    check_forward(s, out, pre, act)
    grad = torch.randn(N, V, generator=torch.Generator("cuda").manual_seed(V), device="cuda").to(t)
    check_backward(s, pre, grad, act, arcs.linear_backward(s["hidden"], s["weight"], grad, pre=pre, activation=act, want_bias=True))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D", [(5, 16384, 64), (9, 16389, 264), (16, 20001, 1000), (13, 33333, 129), (16, 50000, 4097)])
def test_few_rows_of_a_wide_head(arcs, N, V, D, dtype):
    """Five to sixteen rows with 16,384 columns and more: two blocks of columns a workgroup."""
    import torch
    t = types()[dtype]
    s = make(N, V, D, t, N + V + D)
    for act in ("gelu", "none"):
        out, pre = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation=act, residual=s["residual"], out_dtype=torch.float32, want_pre=True)
        check_forward(s, out, pre, act)
    g = torch.Generator("cuda").manual_seed(D)
    h, w, b = whole(g, 2, t, N, D), whole(g, 2, t, V, D), whole(g, 3, t, V)
    assert torch.equal(arcs.linear(h, w, bias=b, out_dtype=torch.float32), (times(h, w.T) + b.double()).float())


@pytest.mark.parametrize("N,V,D", [(148, 34962, 199), (132, 100368, 211), (300, 11070, 2008)])
def test_the_residual_in_place_of_large_tiles(arcs, N, V, D):
    import torch
    s = make(N, V, D, torch.bfloat16, 4)
    want = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="silu", residual=s["residual"])
    x = s["residual"].clone()
    assert torch.equal(arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="silu", residual=x, out=x), want)


def test_replays_of_large_tiles(arcs):
    """Forward and backward of the largest tiles captured, replayed on new inputs between eager calls."""
    import torch
    t = torch.bfloat16
    s = make(2050, 4099, 1032, t, 13)

    def step():
        y, pre = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="silu", residual=s["residual"], want_pre=True)
        return (y, pre) + arcs.linear_backward(s["hidden"], s["weight"], y, pre=pre, activation="silu", want_bias=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        s["hidden"].copy_(torch.randn(2050, 1032, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(t))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


def far_rows(x, stride):
    """The rows of x, `stride` elements apart."""
    import torch
    wide = torch.empty((x.shape[0] - 1) * stride + x.shape[1], dtype=x.dtype, device="cuda").as_strided(x.shape, (stride, 1))
    wide.copy_(x)
    return wide


@pytest.mark.parametrize("over", [-1, 0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_lie_far_apart(arcs, dtype, over):
    """Rows just below 2^23 bytes apart, which the tiles read where they are (256 of them are 2^31 bytes), and
    2^23 bytes apart, which are copied; grad_out too."""
    import torch
    t = types()[dtype]
    size = 2 if dtype == "bf16" else 4
    stride = 2 ** 23 // size + over * (16 // size)
    g = torch.Generator("cuda").manual_seed(3)
    for N, V, D in ((9, 70, 72), (256, 34968, 200), (300, 248, 264)):
        h, w, b, grad = whole(g, 2, t, N, D), whole(g, 2, t, V, D), whole(g, 3, t, V), whole(g, 1, t, N, V)
        x = far_rows(h, stride)
        y = far_rows(w, stride) if V < 300 else w
        z = far_rows(grad, stride)
        assert torch.equal(arcs.linear(x, y, bias=b, out_dtype=torch.float32), (times(h, w.T) + b.double()).float())
        dh, dw, db = arcs.linear_backward(x, y, z, want_bias=True)
        assert torch.equal(dh, times(grad, w).to(t)) and torch.equal(dw, times(grad.T, h).to(t)) and torch.equal(db, grad.double().sum(0).to(t))
