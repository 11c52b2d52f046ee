"""arcs_linear and arcs_linear_backward against the formulas in 64 bits.

Tolerances, with u = 2^-24, h = 2^-8 for bfloat16 results and u for float32 ones (half a step):
  z     products of bfloat16 are exact in float32 and those of float32 are fused into the
        sum, so z has one rounding for each of its D terms, at most 16 more where parts of the
        sum meet, and one for the bias, each of at most u times A = sum |hidden weight| + |bias|:
        e_z = u (D + 18) A.
  act   no slope of an activation is above 1.13 (gelu's), so e_z comes through at most 1.13 times;
        evaluating it costs at most 8 u |z|: an exponential whose argument x is off by 4 u |x|
        moves z / (1 + e^x) by |z| 4 u |x| e^x / (1 + e^x)^2 <= 1.8 u |z|, three more roundings
        of the value, and two units each for exp2 and the reciprocal; the rational form of erfc is
        off by 1.5e-7, which is 1.3 u |z| of z erfc / 2; tanh by 4 u of its argument.
  out   e_y = 1.13 e_z + 8 u |z| + u |y| with the residual's addition, then h (|y| + e_y).
  dz    the slope is at most 1.13 and off by at most 16 u (1 + |z|) (the same functions, a
        few more operations); the product rounds once, and rounding to the type gives h |dz|:
        e_dz = |g| 18 u (1 + |z|) + h |dz|.
  dhidden, dweight   (terms + 18) u sum |dz factor| + sum e_dz |factor|, then h.
  dbias dz before its rounding: (N + 8) u sum |dz| + sum |g| 18 u (1 + |z|), then h.
The backward pass takes the pre-activations that it is given, so its formula does too.
"""

import math

import pytest

from _util import ensure_built

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "softcap"]
CAP = 1.5


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


def half(t):
    import torch
    return torch.finfo(t).eps / 2


def value(z, act):
    import torch
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "softcap":
        return CAP * torch.tanh(z / CAP)
    return z


def slope(z, act):
    """act' by torch's differentiation in 64 bits (relu' is 0 at 0)."""
    import torch
    if act == "none":
        return torch.ones_like(z)
    z = z.detach().clone().requires_grad_(True)
    return torch.autograd.grad(value(z, act).sum(), z)[0]


def rows(t, pad):
    """The same rows in a wider buffer, NaN between them."""
    import torch
    if not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def make(N, V, D, t, seed, bias=True, residual=True, pad=0, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(hidden=rows(normal(N, D).to(t), pad), weight=rows((scale * normal(V, D) / math.sqrt(D)).to(t), pad))
    s["bias"] = (0.5 * normal(V)).to(t) if bias else None
    s["residual"] = rows(normal(N, V).to(t), pad) if residual else None
    return s


def check_forward(s, out, pre, act):
    import torch
    h, w = s["hidden"].double(), s["weight"].double()
    z, size = h @ w.T.contiguous(), h.abs() @ w.abs().T.contiguous()
    if s["bias"] is not None:
        z, size = z + s["bias"].double(), size + s["bias"].double().abs()
    e_z = U * (h.shape[1] + 18) * size
    if pre is not None:
        worst = ((pre.double() - z).abs() - e_z - half(pre.dtype) * (z.abs() + e_z)).max()
        assert worst <= 0, float(worst)
    y = value(z, act)
    e_y = 1.13 * e_z + 8 * U * z.abs() * (act != "none")
    if s["residual"] is not None:
        y = y + s["residual"].double()
        e_y = e_y + U * (y.abs() + e_y)
    worst = ((out.double() - y).abs() - e_y - half(out.dtype) * (y.abs() + e_y)).max()
    assert worst <= 0, float(worst)


def check_backward(s, pre, grad, act, got):
    import torch
    dh, dw, db = got
    t = s["hidden"].dtype
    h, w, g = s["hidden"].double(), s["weight"].double(), grad.double()
    z = pre.double() if act != "none" else torch.zeros_like(g)
    dz = g * slope(z, act)
    e_f = g.abs() * 18 * U * (1 + z.abs()) * (act != "none")
    e_dz = e_f + half(t) * (dz.abs() + e_f)
    N, V = g.shape
    for name, x, a, b, e, n in (("dhidden", dh, dz, w, e_dz @ w.abs(), V),
                                ("dweight", dw, dz.T.contiguous(), h, e_dz.T.contiguous() @ h.abs(), N)):
        if x is not None:
            want = a @ b
            e = e + U * (n + 18) * (a.abs() @ b.abs() + e)
            worst = ((x.double() - want).abs() - e - half(t) * (want.abs() + e)).max()
            assert worst <= 0, (name, float(worst))
    if db is not None:
        want, e = dz.sum(0), e_f.sum(0)
        e = e + U * (N + 8) * (dz.abs().sum(0) + e)
        worst = ((db.double() - want).abs() - e - half(t) * (want.abs() + e)).max()
        assert worst <= 0, ("dbias", float(worst))


def types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


SIZES = [(1, 1, 1), (1, 7, 8), (1, 1000, 1024), (2, 129, 65), (3, 33, 1000), (8, 500, 2048), (15, 64, 100), (16, 257, 40),
         (17, 5, 8), (17, 300, 3), (31, 1003, 64), (33, 129, 1001), (64, 64, 64), (65, 2051, 320), (100, 1000, 1024),
         (129, 1, 63), (200, 513, 72), (257, 255, 264), (300, 1031, 520)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D", SIZES)
def test_forward(arcs, N, V, D, dtype, act):
    import torch
    t = types()[dtype]
    n = ACTS.index(act)
    s = make(N, V, D, t, N * 100 + V + D, bias=n % 2 == 0, residual=n % 3 != 0)
    for out_dtype in types().values():
        out, pre = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation=act, softcap=CAP,
                               residual=s["residual"], out_dtype=out_dtype, want_pre=True)
        assert out.dtype == out_dtype and pre.dtype == t
        check_forward(s, out, pre, act)
        again = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation=act, softcap=CAP,
                            residual=s["residual"], out_dtype=out_dtype)
        assert torch.equal(out, again)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D", SIZES)
def test_backward(arcs, N, V, D, dtype, act):
    import torch
    t = types()[dtype]
    s = make(N, V, D, t, N * 10 + V + D)
    g = torch.Generator(device="cuda").manual_seed(V)
    pre = (2 * torch.randn(N, V, generator=g, device="cuda")).to(t)
    for grad_dtype in types().values():
        grad = torch.randn(N, V, generator=g, device="cuda").to(grad_dtype)
        got = arcs.linear_backward(s["hidden"], s["weight"], grad, pre=None if act == "none" else pre, activation=act,
                                   softcap=CAP, want_bias=True)
        check_backward(s, pre, grad, act, got)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_only_what_is_wanted(arcs, want, act):
    import torch
    s = make(70, 203, 96, torch.bfloat16, 5)
    pre, grad = torch.randn(2, 70, 203, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    got = arcs.linear_backward(s["hidden"], s["weight"], grad, pre=pre, activation=act, want_hidden=want[0],
                               want_weight=want[1], want_bias=want[2])
    assert [x is not None for x in got] == list(want)
    check_backward(s, pre, grad, act, got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,D,pad", [(5, 100, 64, 8), (5, 100, 64, 3), (40, 100, 64, 8), (40, 101, 64, 5), (150, 300, 129, 1),
                                       (150, 304, 128, 24)])
def test_strided_rows_and_what_lies_between_them(arcs, N, V, D, pad, dtype):
    """Rows wider than their elements (off the 16-byte grid too): NaN between the inputs' rows
    reaches nothing, and what lies between the output's rows stays."""
    import torch
    t = types()[dtype]
    s = make(N, V, D, t, 11, pad=pad)
    for out_dtype in types().values():
        buf = torch.full((N, V + pad), 77.0, dtype=out_dtype, device="cuda")
        out = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="gelu", residual=s["residual"], out=buf[:, :V])
        check_forward(s, out, None, "gelu")
        assert (buf[:, V:] == 77.0).all()
    g = torch.Generator(device="cuda").manual_seed(3)
    pre, grad = torch.randn(N, V, generator=g, device="cuda").to(t), rows(torch.randn(N, V, generator=g, device="cuda").to(t), pad)
    for act in ("none", "silu"):
        check_backward(s, pre, grad, act, arcs.linear_backward(s["hidden"], s["weight"], grad, pre=pre, activation=act, want_bias=True))


@pytest.mark.parametrize("N", [4, 50])
def test_the_residual_in_place(arcs, N):
    import torch
    s = make(N, 250, 128, torch.bfloat16, 4)
    want = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="silu", residual=s["residual"])
    x = s["residual"].clone()
    got = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="silu", residual=x, out=x)
    assert got is x and torch.equal(got, want)


@pytest.mark.parametrize("N,V,D", [(3, 70, 72), (40, 300, 136), (140, 300, 137)])
def test_non_finite_rows_stay_where_they_are(arcs, N, V, D):
    """NaN and infinity in one hidden row and one weight row reach that row and column only."""
    import torch
    s = make(N, V, D, torch.bfloat16, 6, bias=False, residual=False)
    clean = arcs.linear(s["hidden"], s["weight"], out_dtype=torch.float32)
    h, w = s["hidden"].clone(), s["weight"].clone()
    h[1, D - 1], w[V - 1, 0] = float("nan"), float("inf")
    got = arcs.linear(h, w, out_dtype=torch.float32)
    r, c = torch.arange(N, device="cuda") != 1, torch.arange(V, device="cuda") != V - 1
    assert torch.equal(got[r][:, c], clean[r][:, c])
    assert got[1].isnan().all() and not got[:, V - 1].isfinite().any()
    grad = torch.randn(N, V, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16)
    dh, dw, db = arcs.linear_backward(s["hidden"], s["weight"], grad, want_bias=True)
    bad = grad.clone()
    bad[N - 1, 2] = float("nan")
    dh2, dw2, db2 = arcs.linear_backward(s["hidden"], s["weight"], bad, want_bias=True)
    v = torch.arange(V, device="cuda") != 2
    assert torch.equal(dh[:-1], dh2[:-1]) and torch.equal(dw[v], dw2[v]) and torch.equal(db[v], db2[v])
    assert dh2[-1].isnan().all() and dw2[2].isnan().all() and db2[2].isnan()


def test_extreme_pre_activations(arcs):
    """Values and slopes at the ends of the range: 0 and the identity, no NaN."""
    import torch
    z = torch.tensor([-1e30, -200.0, -30.0, -0.0, 0.0, 30.0, 200.0, 1e30], device="cuda")
    w = torch.zeros(8, 4, device="cuda")
    w[:, 0] = z
    h = torch.zeros(20, 4, device="cuda")
    h[:, 0] = 1.0
    for n in (20, 3):
        for act in ACTS:
            y, pre = arcs.linear(h[:n], w, activation=act, softcap=CAP, want_pre=True)
            lo, hi = (z[:3], z[5:]) if act == "none" else (torch.full((3,), -CAP), torch.full((3,), CAP)) if act == "softcap" else (
                torch.zeros(3), z[5:])
            assert torch.allclose(y[0, :3], lo.cuda(), rtol=1e-6, atol=1e-11) and torch.allclose(y[0, 5:], hi.cuda(), rtol=1e-6)
            assert (y[:, 3:5] == 0).all() and torch.equal(pre[0], z)
            _, _, db = arcs.linear_backward(h[:1], w, torch.ones(1, 8, device="cuda"), pre=pre[:1].contiguous(), activation=act, softcap=CAP,
                                            want_bias=True)
            ends = {"none": (1, 1), "softcap": (0, 0)}.get(act, (0, 1))
            assert torch.allclose(db[:3], torch.full((3,), float(ends[0]), device="cuda"), atol=3e-12), (act, db)
            assert torch.allclose(db[5:], torch.full((3,), float(ends[1]), device="cuda"), atol=1e-7), (act, db)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "softcap"])
def test_gradients_against_differences(arcs, act):
    """The directional derivative of sum(g out) in float32.  With step s the central difference
    is off by s^2 / 6 times the third derivative along the direction, and by the outputs' errors
    over s; both are bounded from the terms below."""
    import torch
    N, V, D, step = 21, 24, 16, 2.0 ** -6
    s = make(N, V, D, torch.float32, 9, residual=False)
    g = torch.Generator(device="cuda").manual_seed(8)
    grad = torch.randn(N, V, generator=g, device="cuda")
    dirs = [torch.randn(x.shape, generator=g, device="cuda") for x in (s["hidden"], s["weight"], s["bias"])]

    def loss(k):
        x = [a + k * step * d for a, d in zip((s["hidden"], s["weight"], s["bias"]), dirs)]
        return float((arcs.linear(x[0], x[1], bias=x[2], activation=act, softcap=CAP).double() * grad.double()).sum())

    _, pre = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation=act, softcap=CAP, want_pre=True)
    got = arcs.linear_backward(s["hidden"], s["weight"], grad, pre=pre, activation=act, softcap=CAP, want_bias=True)
    want = sum(float((a.double() * d.double()).sum()) for a, d in zip(got, dirs))
    # z along the direction is z + k s z1 + (k s)^2 z2; activations' derivatives up to the third are below 2
    h, w = s["hidden"].abs().double(), s["weight"].abs().double()
    dh, dw, db = (d.abs().double() for d in dirs)
    z1, z2 = dh @ w.T + h @ dw.T + db, dh @ dw.T
    first = z1 + 2 * step * z2
    third = (grad.abs().double() * 2 * (first ** 3 + 6 * first * z2)).sum()
    each = U * (grad.abs().double() * (h @ w.T + 4) * (D + 40)).sum()
    slopes = U * (grad.abs().double() * 1.13 * z1 * (N + V + 40 + 18 * (1 + pre.abs().double()))).sum()
    assert abs((loss(1) - loss(-1)) / (2 * step) - want) <= float(step ** 2 / 6 * third + each / step + slopes)


@pytest.mark.parametrize("N,V,D", [(3, 300, 128), (60, 301, 136), (60, 300, 1999)])
def test_side_stream_and_replays(arcs, N, V, D):
    """Calls on another stream, and forward and backward captured and replayed on new inputs
    between eager calls."""
    import torch
    t = torch.bfloat16
    s = make(N, V, D, t, 13)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="silu", residual=s["residual"], stream=side)
    side.synchronize()
    check_forward(s, out, None, "silu")

    def step(outs=None):
        outs = outs or {}
        y, pre = arcs.linear(s["hidden"], s["weight"], bias=s["bias"], activation="silu", residual=s["residual"], want_pre=True)
        return (y, pre) + arcs.linear_backward(s["hidden"], s["weight"], y, pre=pre, activation="silu", want_bias=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        s["hidden"].copy_(torch.randn(N, D, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(t))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


def test_a_large_call_far_rows(arcs):
    """Outputs past 2^31 elements from the start, checked at both ends."""
    import torch
    N, V, D = 16900, 130001, 8
    s = make(N, V, D, torch.bfloat16, 17, bias=False, residual=False)
    out = arcs.linear(s["hidden"], s["weight"])
    for r in (slice(0, 3), slice(N - 3, N)):
        check_forward(dict(s, hidden=s["hidden"][r]), out[r], None, "none")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_more_rows_than_a_grids_second_axis(arcs, dtype):
    """65,536 workgroups of 32 rows and one more, on whole numbers whose sums float32 holds, so each
    result is the exact one rounded once."""
    import torch
    t = getattr(torch, dtype)
    N, V, D = 65536 * 32 + 5, 9, 8
    g = torch.Generator("cuda").manual_seed(9)
    h = torch.randint(-1, 2, (N, D), generator=g, device="cuda").to(t)
    w = torch.randint(-2, 3, (V, D), generator=g, device="cuda").to(t)
    grad = torch.randint(0, 2, (N, V), generator=g, device="cuda").to(t)
    pre = torch.randint(-1, 2, (N, V), generator=g, device="cuda").to(t)
    dh, dw, db = arcs.linear_backward(h, w, grad, pre=pre, activation="relu", want_bias=True)
    dz = torch.where(pre > 0, grad, torch.zeros_like(grad)).float()
    assert torch.equal(db, dz.double().sum(0).to(t))
    assert torch.equal(dh, (dz[:, :, None] * w.float()).sum(1).to(t))
    want = torch.stack([(dz[:, v, None].double() * h.double()).sum(0) for v in range(V)])
    assert torch.equal(dw, want.to(t))


@pytest.mark.parametrize("D", [8, 9])
@pytest.mark.parametrize("N", [16, 17])
def test_the_largest_vocabulary(arcs, N, D):
    """2^24 columns, whose rows off the 16-byte grid are more than a launch has workgroups of 256
    threads for; whole numbers, so each result is exact."""
    import torch
    V = 2 ** 24
    g = torch.Generator("cuda").manual_seed(D)
    h = torch.randint(-2, 3, (N, D), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randint(-3, 4, (V, D), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    out = arcs.linear(h, w)
    for at in range(0, V, V // 8):
        want = sum(h[:, None, d].float() * w[None, at: at + V // 8, d].float() for d in range(D))
        assert torch.equal(out[:, at: at + V // 8].float(), want)
