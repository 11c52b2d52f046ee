"""arcs_linear_cross_entropy and its backward against the definition in 64 bits.

Tolerances.  A logit is a float32 sum of D products (exact for bfloat16
inputs, rounded once for float32 ones): its error is at most
  e = 2^-24 (D + 2) sum_d |h_d w_d| / T,
the sum's size being at most |h| |w| (Cauchy).  logsumexp moves by at most the
largest e of the row; its own arithmetic adds the roundings of exp2 and log2
(2^-22 relative on the weights, so 2^-22 on the logarithm), of the sums over
slices (2^-24 per addition, at most 64 + V / 64 of them on the longest path),
and of the base-2 result and its way back (3 * 2^-24 |lse|).  So
  |d lse|  <= e + 2^-22 + 2^-24 (64 + V / 64) + 2^-22 |lse|
  |d loss| <= 2 e + the same.
Gradients: p = exp(z - lse) is off by the factor 1 + delta with delta <= e +
|d lse| of the lse that is handed over, and dz is rounded to bfloat16 (2^-8
relative, matrix kernels) or not at all (general kernel, float32); the sums
over v or n round by 2^-24 per addition, and the result by half a step of its
type.  With S = sum |dz| |w| the bound is
  S (2^-8 + delta + 2^-24 (terms + 8)) + half a step |want|
for bfloat16, and the same without 2^-8 for float32, where delta also covers the
target's 1 - p.
"""

import numpy as np
import pytest

from _util import ensure_built

pytestmark = pytest.mark.gpu

IGNORE = -100


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


def make(N, V, D, dtype, seed, temperature=False, ignored=0.0, weighted=False, pad=0, shift=0):
    """Device tensors and their float64 values.  `pad` widens the rows, `shift`
    moves the first element (both in elements)."""
    import torch
    rng = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def matrix(x):
        full = torch.full((x.shape[0] * (x.shape[1] + pad) + shift,), float("nan"), dtype=dt)
        view = full[shift:].view(x.shape[0], x.shape[1] + pad)
        view[:, : x.shape[1]] = torch.from_numpy(x.astype(np.float32)).to(dt)
        full = full.cuda()
        return full[shift:].view(x.shape[0], x.shape[1] + pad)[:, : x.shape[1]]

    w = rng.standard_normal((V, D)) * 2.0 / np.sqrt(D)
    t = rng.integers(0, V, N).astype(np.int32)
    h = rng.standard_normal((N, D)) + 2.0 * rng.uniform(0, 1, (N, 1)) * w[t]
    t[rng.permutation(N)[: int(ignored * N)]] = IGNORE
    s = dict(hidden=matrix(h), weight=matrix(w), targets=torch.from_numpy(t).cuda(),
             temperature=torch.from_numpy(rng.uniform(0.3, 2.0, N).astype(np.float32)).cuda() if temperature else None)
    g = (rng.standard_normal(N) if weighted else np.full(N, 1.0 / max(1, N))).astype(np.float32)
    return s, torch.from_numpy(g).cuda()


def reference(s, g=None, ignore=IGNORE):
    """Everything in float64 on the CPU: loss, lse, gradients and the sizes the bounds need."""
    h, w = s["hidden"].double().cpu().numpy(), s["weight"].double().cpu().numpy()
    t = s["targets"].cpu().numpy()
    N, V, D = h.shape[0], w.shape[0], w.shape[1]
    T = s["temperature"].double().cpu().numpy() if s["temperature"] is not None else np.ones(N)
    on = (t != ignore) & (t >= 0) & (t < V) & (T > 0) & np.isfinite(T)
    hz = np.where(on[:, None], h, 0.0)
    Tz = np.where(on, T, 1.0)
    tz = np.where(on, t, 0)
    z = hz @ w.T / Tz[:, None]
    m = z.max(axis=1)
    e = np.exp(z - m[:, None])
    lse = m + np.log(e.sum(axis=1))
    at = np.arange(N)
    size = np.abs(hz) @ np.abs(w).T
    r = dict(on=on, lse=np.where(on, lse, 0.0), loss=np.where(on, lse - z[at, tz], 0.0),
             e=2.0 ** -24 * (D + 2) * size.max(axis=1) / Tz)
    if g is not None:
        p = np.exp(z - lse[:, None])
        d = p.copy()
        d[at, tz] -= 1.0
        f = np.where(on, g.double().cpu().numpy() / Tz, 0.0)
        d *= f[:, None]
        r["dz"], r["p"], r["f"] = d, p, f
        r["dh"], r["dw"] = d @ w, d.T @ hz
        r["h"], r["w"] = hz, w
    return r


def lse_bound(r, V):
    return r["e"] + 2.0 ** -22 + 2.0 ** -24 * (64 + V / 64) + 2.0 ** -22 * np.abs(r["lse"])


def check_forward(loss, lse, r, V):
    b = lse_bound(r, V)
    err = np.abs(lse.double().cpu().numpy() - r["lse"])
    assert np.all(err <= b), np.max(err - b)
    err = np.abs(loss.double().cpu().numpy() - r["loss"])
    assert np.all(err <= b + r["e"]), np.max(err - b - r["e"])


def check_gradients(dh, dw, r, V, dtype, rounded):
    """`rounded`: dz may have been held in bfloat16."""
    N, D = r["h"].shape
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    delta = (lse_bound(r, V) + r["e"])[:, None]
    # the error of one dz: relative on p, and on the rounded value
    dz_err = np.abs(r["f"])[:, None] * r["p"] * delta + (2.0 ** -8 if rounded else 2.0 ** -23) * np.abs(r["dz"])
    for got, want, err, size, terms in (
            (dh, r["dh"], dz_err @ np.abs(r["w"]), np.abs(r["dz"]) @ np.abs(r["w"]), V),
            (dw, r["dw"], dz_err.T @ np.abs(r["h"]), np.abs(r["dz"]).T @ np.abs(r["h"]), N)):
        if got is None:
            continue
        bound = err + 2.0 ** -24 * (terms + 8) * size
        bound = 1.01 * bound + half * (np.abs(want) + bound) + 1e-38
        off = np.abs(got.double().cpu().numpy() - want)
        assert np.all(off <= bound), (np.max(off - bound), np.max(off / bound))


CASES = [
    # N, V, D, dtype, temperature, ignored, weighted
    (1, 1, 1, "f32", False, 0.0, False),
    (1, 1, 8, "bf16", False, 0.0, True),
    (1, 2, 16, "bf16", True, 0.0, True),
    (2, 129, 24, "bf16", False, 0.5, False),
    (3, 1000, 7, "bf16", True, 0.0, True),
    (5, 300, 33, "f32", True, 0.2, True),
    (16, 4096, 64, "bf16", False, 0.0, False),
    (17, 257, 136, "bf16", True, 0.3, True),
    (63, 511, 1000, "bf16", False, 0.0, True),
    (64, 2049, 256, "bf16", True, 0.5, True),
    (65, 640, 520, "bf16", True, 0.0, False),
    (127, 1025, 96, "f32", False, 0.3, True),
    (128, 129, 2048, "bf16", False, 0.0, True),
    (129, 3001, 264, "bf16", True, 0.9, True),
    (257, 777, 1032, "bf16", False, 0.1, True),
    (300, 5000, 128, "bf16", True, 0.25, True),
    (513, 300, 72, "f32", True, 0.1, True),
    (1100, 600, 320, "bf16", False, 0.6, True),
    # vocabularies with enough tiles for the larger ones of each row count
    (20, 16500, 64, "bf16", True, 0.2, True),
    (20, 66003, 64, "bf16", False, 0.0, True),
    (64, 33000, 64, "bf16", True, 0.0, True),
    (100, 33001, 72, "bf16", False, 0.3, True),
    (130, 33000, 1032, "bf16", True, 0.1, True),
    (300, 16500, 64, "bf16", False, 0.5, False),
    (20, 16500, 64, "f32", True, 0.2, True),
    (50, 33001, 36, "f32", False, 0.0, True),
    (200, 12500, 64, "f32", True, 0.3, True),
    (1024, 500, 48, "bf16", True, 0.4, True),
]


@pytest.mark.parametrize("N,V,D,dtype,temperature,ignored,weighted", CASES)
def test_against_the_definition(arcs, N, V, D, dtype, temperature, ignored, weighted):
    import torch
    s, g = make(N, V, D, dtype, N * 7 + V, temperature, ignored, weighted)
    r = reference(s, g)
    status = torch.full((N,), 99, dtype=torch.int32, device="cuda")
    loss, lse = arcs.linear_cross_entropy(**s, out_status=status)
    check_forward(loss, lse, r, V)
    assert (status == 0).all()
    dh, dw = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                temperature=s["temperature"])
    check_gradients(dh, dw, r, V, dtype, dtype == "bf16")
    # the same bits again, and one gradient at a time
    loss2, lse2 = arcs.linear_cross_entropy(**s)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    only_h, none = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                      temperature=s["temperature"], want_weight=False)
    assert none is None and torch.equal(only_h, dh)
    none, only_w = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                      temperature=s["temperature"], want_hidden=False)
    assert none is None and torch.equal(only_w, dw)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (8, 8), (5, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_alignments(arcs, dtype, pad, shift):
    """Wider rows and first elements off the 16-byte grid; the padding holds NaN."""
    s, g = make(150, 700, 160, dtype, 5, True, 0.2, True, pad=pad, shift=shift)
    r = reference(s, g)
    loss, lse = arcs.linear_cross_entropy(**s)
    check_forward(loss, lse, r, 700)
    dh, dw = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                temperature=s["temperature"])
    check_gradients(dh, dw, r, 700, dtype, dtype == "bf16")


@pytest.mark.parametrize("N", [5, 70, 400])
def test_masked_and_refused_rows(arcs, N):
    """Ignored and refused rows hold NaN and infinities in their hidden states and
    upstream gradients; nothing of them reaches another row or the head's gradient."""
    import torch
    V, D = 900, 256
    s, g = make(N, V, D, "bf16", 21, True, 0.0, True)
    clean, lse0 = arcs.linear_cross_entropy(**s)
    t, T, h = s["targets"].clone(), s["temperature"].clone(), s["hidden"].clone()
    t[0] = IGNORE
    t[1] = V
    t[2] = -1
    T[3] = float("nan") if N < 50 else 0.0
    g = g.clone()
    for n, bad in ((0, "nan"), (1, "inf"), (2, "nan"), (3, "-inf")):
        h[n] = float(bad)
        g[n] = float(bad)
    s2 = dict(hidden=h, weight=s["weight"], targets=t, temperature=T)
    status = torch.empty(N, dtype=torch.int32, device="cuda")
    loss, lse = arcs.linear_cross_entropy(**s2, out_status=status)
    assert status[:4].tolist() == [0, arcs.ROW_BAD_TARGET, arcs.ROW_BAD_TARGET, arcs.ROW_BAD_TEMPERATURE]
    assert (status[4:] == 0).all()
    assert loss[0] == 0 and lse[0] == 0 and loss[1:4].isnan().all() and lse[1:4].isnan().all()
    r = reference(dict(s2, hidden=s["hidden"]), g)
    loss[1:4] = lse[1:4] = 0
    check_forward(loss, lse, r, V)
    lse[1:4] = float("nan")
    dh, dw = arcs.linear_cross_entropy_backward(h, s["weight"], t, lse, g, temperature=T)
    assert (dh[:4] == 0).all()
    check_gradients(dh, dw, r, V, "bf16", True)


def test_every_row_ignored(arcs):
    import torch
    for N, D in ((1, 64), (300, 64), (40, 13)):
        s, g = make(N, 333, D, "bf16", 2)
        s["targets"].fill_(IGNORE)
        s["hidden"].fill_(float("nan"))
        loss, lse = arcs.linear_cross_entropy(**s)
        assert (loss == 0).all() and (lse == 0).all()
        dh, dw = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g)
        assert (dh == 0).all() and (dw == 0).all()


def test_an_ignore_index_inside_the_vocabulary(arcs):
    s, g = make(80, 50, 64, "bf16", 3)
    s["targets"][::3] = 7
    r = reference(s, g, ignore=7)
    loss, lse = arcs.linear_cross_entropy(**s, ignore_index=7)
    check_forward(loss, lse, r, 50)
    dh, dw = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g, ignore_index=7)
    check_gradients(dh, dw, r, 50, "bf16", True)


@pytest.mark.parametrize("N,D", [(6, 64), (200, 64), (6, 15)])
def test_non_finite_logits(arcs, N, D):
    """A row with NaN or +inf logits has a NaN loss; other rows are untouched.  A
    weight row of -inf logits is a token of probability zero."""
    import torch
    s, g = make(N, 400, D, "bf16", 9)
    loss0, _ = arcs.linear_cross_entropy(**s)
    h = s["hidden"].clone()
    h[1, 3] = float("nan")
    h[4, 0] = float("inf")
    loss, lse = arcs.linear_cross_entropy(h, s["weight"], s["targets"])
    keep = torch.ones(N, dtype=torch.bool)
    keep[[1, 4]] = False
    assert torch.equal(loss[keep], loss0[keep])
    assert loss[1].isnan() and loss[4].isnan()
    # one token at -inf: dot of positive hidden states with a row of -inf
    hp, w = s["hidden"].abs() + 0.5, s["weight"].clone()
    w[11] = float("-inf")
    t = torch.where(s["targets"] == 11, torch.zeros_like(s["targets"]), s["targets"])
    loss, lse = arcs.linear_cross_entropy(hp, w, t)
    keepv = torch.ones(400, dtype=torch.bool)
    keepv[11] = False
    z = hp.double().cpu() @ w[keepv.cuda()].double().cpu().T
    assert (lse.double().cpu() - torch.logsumexp(z, 1)).abs().max() < 1e-3


def test_large_logits_do_not_overflow(arcs):
    import torch
    s, g = make(70, 300, 64, "bf16", 4)
    h = s["hidden"] * 300.0
    r = reference(dict(s, hidden=h), g)
    loss, lse = arcs.linear_cross_entropy(h, s["weight"], s["targets"])
    check_forward(loss, lse, r, 300)
    assert lse.abs().max() > 500


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(arcs, dtype):
    """Central differences of the 64-bit loss along random directions."""
    import torch
    N, V, D = 40, 333, 48
    s, g = make(N, V, D, dtype, 13, True, 0.2, True)
    loss, lse = arcs.linear_cross_entropy(**s)
    dh, dw = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                temperature=s["temperature"])
    h, w = s["hidden"].double().cpu(), s["weight"].double().cpu()
    t, T = s["targets"].long().cpu(), s["temperature"].double().cpu()
    on = t != IGNORE

    def total(h, w):
        z = (h @ w.T) / T[:, None]
        l = torch.logsumexp(z, 1) - z.gather(1, torch.where(on, t, 0)[:, None])[:, 0]
        return (torch.where(on, l, 0.0) * g.double().cpu()).sum()

    gen = torch.Generator().manual_seed(1)
    eps = 1e-5
    r = reference(s, g)
    for which, grad in (("h", dh), ("w", dw)):
        for _ in range(5):
            u = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
            a = (h + eps * u, w) if which == "h" else (h, w + eps * u)
            b = (h - eps * u, w) if which == "h" else (h, w - eps * u)
            slope = (total(*a) - total(*b)) / (2 * eps)
            got = (grad.double().cpu() * u).sum()
            # the entries' bounds of check_gradients, added with the direction's size
            half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
            size = np.abs(r["dz"]) @ np.abs(r["w"]) if which == "h" else np.abs(r["dz"]).T @ np.abs(r["h"])
            tol = float((size * (2 * half + 1e-5) * np.abs(u.numpy())).sum()) + 1e-6
            assert abs(slope - got) <= tol, (which, float(slope), float(got), tol)


def test_workspace_contents_do_not_matter(arcs):
    """A caller's workspace, full of NaN patterns and larger than needed, used for
    calls of different shapes in a row."""
    import torch
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    for N, V, D, dtype in ((200, 1500, 256, "bf16"), (3, 400, 64, "bf16"), (60, 900, 31, "f32"), (200, 1500, 256, "bf16")):
        s, g = make(N, V, D, dtype, 17, True, 0.3, True)
        want = arcs.linear_cross_entropy(**s)
        got = arcs.linear_cross_entropy(**s, workspace=ws)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        args = (s["hidden"], s["weight"], s["targets"], want[1], g)
        wd = arcs.linear_cross_entropy_backward(*args, temperature=s["temperature"])
        ws.fill_(255)
        gd = arcs.linear_cross_entropy_backward(*args, temperature=s["temperature"], workspace=ws)
        assert torch.equal(wd[0], gd[0]) and torch.equal(wd[1], gd[1])


def test_side_stream_and_replays(arcs):
    """A pair of calls on another stream, and captured forward and backward calls
    replayed on inputs rewritten in place, with eager work in between."""
    import torch
    N, V, D = 140, 2000, 192
    s, g = make(N, V, D, "bf16", 23, True, 0.2, True)
    want, want_lse = arcs.linear_cross_entropy(**s)
    wd = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], want_lse, g,
                                            temperature=s["temperature"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = arcs.linear_cross_entropy(**s, stream=side)
    dh, dw = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                temperature=s["temperature"], stream=side)
    side.synchronize()
    assert torch.equal(loss, want) and torch.equal(dh, wd[0]) and torch.equal(dw, wd[1])
    h = s["hidden"].clone()
    t = s["targets"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = arcs.linear_cross_entropy(h, s["weight"], t, temperature=s["temperature"])
        dh, dw = arcs.linear_cross_entropy_backward(h, s["weight"], t, lse, g, temperature=s["temperature"])
    for step in range(5):
        h.copy_(torch.randn(N, D, device="cuda").to(torch.bfloat16))
        t.copy_(torch.randint(-3, V, (N,), device="cuda").to(torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        e_loss, e_lse = arcs.linear_cross_entropy(h, s["weight"], t, temperature=s["temperature"])
        e_dh, e_dw = arcs.linear_cross_entropy_backward(h, s["weight"], t, e_lse, g, temperature=s["temperature"])
        assert torch.equal(loss.nan_to_num(7), e_loss.nan_to_num(7)), step
        assert torch.equal(dh, e_dh) and torch.equal(dw, e_dw), step


def test_agrees_with_top_logprobs(arcs):
    """-loss is the log-probability top_logprobs reports for the same logits."""
    import torch
    N, V, D = 12, 3000, 128
    s, g = make(N, V, D, "f32", 31, True)
    logits = (s["hidden"].double() @ s["weight"].double().T).float()
    ids, lps = arcs.top_logprobs(logits, 4, temperature=s["temperature"])
    for k in range(4):
        loss, _ = arcs.linear_cross_entropy(s["hidden"], s["weight"], ids[:, k].contiguous(),
                                            temperature=s["temperature"])
        assert (-loss - lps[:, k]).abs().max() < 2e-4


def test_decode_and_train_run(arcs):
    """The head's operators as they are used together: a decode step draws tokens
    from 4-bit logits, the drawn tokens are scored at their temperature and become
    the targets of a policy gradient on the head in bfloat16."""
    import torch
    B, V, D, G = 24, 4000, 256, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    hidden = torch.randn(B, D, generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randint(0, 16, (V, D), generator=gen, device="cuda").to(torch.uint8)
    scales = (0.5 + torch.rand(V, D // G, generator=gen, device="cuda")) * 0.03
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    logits = arcs.w4_logits(hidden, packed, scales, G, out_dtype=torch.float32)
    from workloads import make_params
    T = torch.full((B,), 0.8, device="cuda")
    ids = arcs.sample(logits, arcs.params_to_device(make_params(B, temperature=0.8)), seed=5, step=1)
    assert ((ids >= 0) & (ids < V)).all()
    weight = ((q.float() - 8).view(V, D // G, G) * scales[:, :, None]).view(V, D).to(torch.bfloat16)
    loss, lse = arcs.linear_cross_entropy(hidden, weight, ids, temperature=T)
    # the 4-bit logits and the bfloat16 copy of the head agree to the copy's rounding
    z = logits.double() / 0.8
    want = torch.logsumexp(z, 1) - z.gather(1, ids.long()[:, None])[:, 0]
    assert (loss.double() - want).abs().max() < 0.1
    advantage = torch.randn(B, generator=gen, device="cuda")
    dh, dw = arcs.linear_cross_entropy_backward(hidden, weight, ids, lse, advantage, temperature=T)
    s = dict(hidden=hidden, weight=weight, targets=ids, temperature=T)
    check_gradients(dh, dw, reference(s, advantage), V, "bf16", True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_far_apart(arcs, dtype):
    """Offsets past 32 bits: hidden rows 8 MiB apart (2.5 GB in all, read through a
    copy), and head rows 4 MiB apart (5 GB)."""
    import torch
    N, V, D = 300, 1230, 64
    s, g = make(N, V, D, dtype, 41, True, 0.2, True)
    want, lse = arcs.linear_cross_entropy(**s)
    wh, ww = arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                temperature=s["temperature"])
    dt = s["hidden"].dtype
    step_h, step_w = (8 << 20) // dt.itemsize, (4 << 20) // dt.itemsize - 64
    far_h = torch.empty(N * step_h, dtype=dt, device="cuda").as_strided((N, D), (step_h, 1))
    far_w = torch.empty(V * step_w, dtype=dt, device="cuda").as_strided((V, D), (step_w, 1))
    far_h.copy_(s["hidden"])
    far_w.copy_(s["weight"])
    got, lse2 = arcs.linear_cross_entropy(far_h, far_w, s["targets"], temperature=s["temperature"])
    dh, dw = arcs.linear_cross_entropy_backward(far_h, far_w, s["targets"], lse2, g, temperature=s["temperature"])
    assert torch.equal(got, want) and torch.equal(dh, wh) and torch.equal(dw, ww)


def test_many_pieces_and_tiles(arcs):
    """Enough rows that the vocabulary is taken in several pieces, and enough tiles
    that a workgroup takes more than one; rows checked against 64 bits on the GPU."""
    import torch
    N, V, D = 12000, 20000, 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(N, D, generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, D, generator=gen, device="cuda") * 0.2).to(torch.bfloat16)
    t = torch.randint(0, V, (N,), generator=gen, device="cuda").to(torch.int32)
    t[::7] = IGNORE
    g = torch.full((N,), 1.0 / N, device="cuda")
    loss, lse = arcs.linear_cross_entropy(h, w, t)
    on = t != IGNORE
    rows = torch.nonzero(on)[:, 0]
    z = h[rows].double() @ w.double().T
    want_lse = torch.logsumexp(z, 1)
    tr = t[rows].long()
    # the bound of a logit, D = 128 terms of size |h| |w| (about 11 * 2.3), and its logarithm
    assert (lse[rows].double() - want_lse).abs().max() < 2e-5
    assert (loss[rows].double() - (want_lse - z.gather(1, tr[:, None])[:, 0])).abs().max() < 4e-5
    assert (loss[~on] == 0).all() and (lse[~on] == 0).all()
    dh, dw = arcs.linear_cross_entropy_backward(h, w, t, lse, g)
    p = torch.exp(z - want_lse[:, None])
    p.scatter_add_(1, tr[:, None], torch.full((len(rows), 1), -1.0, dtype=torch.float64, device="cuda"))
    p /= N
    for got, ref in ((dh[rows], p @ w.double()), (dw, p.T.contiguous() @ h[rows].double())):
        # dz is rounded to bfloat16 (2^-9 on average at most) and so is the result
        assert torch.linalg.norm(got.double() - ref) <= 2.0 ** -8 * torch.linalg.norm(ref)
    assert (dh[~on] == 0).all()


def test_calls_on_two_streams_at_once(arcs):
    """Calls that overlap, each with a workspace of its own, do not meet."""
    import torch
    cases = [make(900, 3000, 256, "bf16", 50 + k, True, 0.2, True) for k in range(2)]
    want = []
    for s, g in cases:
        loss, lse = arcs.linear_cross_entropy(**s)
        want.append((loss, *arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                               temperature=s["temperature"])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(4):
        for k, (s, g) in enumerate(cases):
            loss, lse = arcs.linear_cross_entropy(**s, stream=streams[k])
            got[k].append((loss, *arcs.linear_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], lse, g,
                                                                     temperature=s["temperature"], stream=streams[k])))
    torch.cuda.synchronize()
    for k in range(2):
        for one in got[k]:
            assert all(torch.equal(x, y) for x, y in zip(one, want[k]))


def test_binding_refuses(arcs):
    """Mistakes in tensors raise before anything is launched."""
    import torch
    s, g = make(6, 40, 64, "bf16", 1)
    h, w, t = s["hidden"], s["weight"], s["targets"]
    for bad in (dict(targets=t.long()), dict(targets=t[:5]), dict(weight=w.float()), dict(weight=w[:, :32]),
                dict(hidden=h.t()), dict(temperature=torch.ones(5, device="cuda")), dict(ignore_index=2**31),
                dict(out_loss=torch.empty(6, device="cuda", dtype=torch.float64)),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            arcs.linear_cross_entropy(**{**s, **bad})
    with pytest.raises(TypeError):
        arcs.linear_cross_entropy(h.half(), w.half(), t)
    with pytest.raises(arcs.ArcsError):
        arcs.linear_cross_entropy(h, w, t, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(arcs.ArcsError):
        arcs.linear_cross_entropy_backward(h, w, t, g, g, want_hidden=False, want_weight=False)
    with pytest.raises(ValueError):
        arcs.linear_cross_entropy_backward(h, w, t, g, g, out_dweight=torch.empty(40, 64, device="cuda"))
