"""arcs_w4_logits against the definition in 64 bits.

Tolerance.  Weights, offsets and hidden states enter exactly, so the error is
that of float32 sums.  In a group the kernel adds (16 + q) h and takes
(16 + z) sum h away: every partial sum is at most A = sum (16 + q + 16 + z) |h|
<= 62 sum |h|, and each of at most G + 2 additions rounds by 2^-24 of it (a
product of two bfloat16 is exact in float32).  Over the groups the scaled sums
add D / G more roundings of the running total.  The bound used per logit is
  2^-24 (G + 2 + D / G + 4) sum_g |s_g| A_g
plus half a step of the output type, 2^-8 |logit| for bfloat16 and 2^-24 for
float32 (which the first term covers many times over).
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


def make(B, V, D, G, zeros, scales, seed, pad=0):
    """Host inputs (float64 views of what the device holds) and device tensors;
    `pad` widens every row (in 16-byte steps where rows must stay aligned)."""
    import torch
    rng = np.random.default_rng(seed)
    h = torch.from_numpy(rng.standard_normal((B, D + 8 * pad)).astype(np.float32)).to(torch.bfloat16)
    h[0, :D] += 0.5  # a row whose groups do not cancel
    q = rng.integers(0, 16, (V, D), dtype=np.uint8)
    packed = np.zeros((V, D // 2 + 16 * pad), np.uint8)
    packed[:, : D // 2] = q[:, 0::2] | (q[:, 1::2] << 4)
    dt = torch.bfloat16 if scales == "bf16" else torch.float32
    s = torch.from_numpy((rng.uniform(0.2, 1.5, (V, D // G + pad)) * rng.choice([-1, 1], (V, D // G + pad))
                          / np.sqrt(D)).astype(np.float32)).to(dt)
    z = rng.integers(0, 16, (V, D // G + pad), dtype=np.uint8) if zeros else None
    dev = dict(hidden=h.cuda()[:, :D], qweight=torch.from_numpy(packed).cuda()[:, : D // 2],
               scales=s.cuda()[:, : D // G], zeros=torch.from_numpy(z).cuda()[:, : D // G] if zeros else None)
    host = dict(h=h[:, :D].double().numpy(), q=q.astype(np.float64), s=s[:, : D // G].double().numpy(),
                z=z[:, : D // G].astype(np.float64) if zeros else np.full((V, D // G), 8.0))
    return host, dev


def reference(host, G):
    V, D = host["q"].shape
    level = (host["q"].reshape(V, D // G, G) - host["z"][:, :, None]) * host["s"][:, :, None]
    want = host["h"] @ level.reshape(V, D).T
    size = (host["q"].reshape(V, D // G, G) + 32 + host["z"][:, :, None]) * np.abs(host["s"])[:, :, None]
    bound = np.abs(host["h"]) @ size.reshape(V, D).T * 2.0 ** -24 * (G + 6 + D // G)
    return want, bound


def check(got, host, G, out):
    want, bound = reference(host, G)
    half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    err = np.abs(got.double().cpu().numpy() - want)
    worst = np.max(err - bound * 1.01 - half * (np.abs(want) + bound))
    assert worst <= 0, worst


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("B,V,D,G,scales", [
    (1, 1, 32, 32, "bf16"), (1, 5, 128, 128, "f32"), (1, 1000, 1024, 64, "bf16"), (2, 129, 96, 32, "f32"),
    (3, 257, 192, 64, "bf16"), (5, 4099, 4064, 32, "bf16"), (15, 77, 640, 128, "f32"), (16, 320, 512, 32, "bf16"),
    (17, 500, 1088, 64, "f32"), (31, 1023, 2048, 128, "bf16"), (33, 130, 160, 32, "bf16"),
    (64, 2051, 1152, 128, "bf16"), (65, 515, 320, 64, "f32"), (100, 64, 4096, 128, "bf16"),
    (129, 1111, 736, 32, "bf16"), (256, 700, 1024, 64, "bf16"), (300, 259, 384, 128, "f32"),
])
def test_against_the_definition(arcs, B, V, D, G, scales, zeros, out):
    import torch
    host, dev = make(B, V, D, G, zeros, scales, seed=B * 1000 + V)
    got = arcs.w4_logits(dev["hidden"], dev["qweight"], dev["scales"], G, zeros=dev["zeros"],
                         out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    check(got, host, G, out)
    again = arcs.w4_logits(dev["hidden"], dev["qweight"], dev["scales"], G, zeros=dev["zeros"], out_dtype=got.dtype)
    assert torch.equal(got, again)


@pytest.mark.parametrize("B,V,D,G", [(3, 133, 416, 32), (40, 300, 1024, 128), (130, 200, 320, 64)])
def test_strided_rows_and_what_lies_between_them(arcs, B, V, D, G):
    """Rows wider than their elements; the padding of the output stays as it was,
    and NaN in the padding of the hidden states reaches nothing."""
    import torch
    host, dev = make(B, V, D, G, True, "bf16", seed=7, pad=3)
    dev["hidden"].as_strided((B, 8), (dev["hidden"].stride(0), 1), D).fill_(float("nan"))
    for width in (V, V + 1, V + 64):
        buf = torch.full((B, width), 77.0, dtype=torch.bfloat16, device="cuda")
        got = arcs.w4_logits(dev["hidden"], dev["qweight"], dev["scales"], G, zeros=dev["zeros"], out=buf[:, :V])
        check(got, host, G, "bf16")
        assert (buf[:, V:] == 77.0).all()


def test_non_finite_rows_stay_in_their_row(arcs):
    """NaN or infinity in one hidden row, or one weight row's scale, reaches only that row or column."""
    import torch
    B, V, D, G = 20, 300, 512, 64
    host, dev = make(B, V, D, G, False, "f32", seed=3)
    clean = arcs.w4_logits(dev["hidden"], dev["qweight"], dev["scales"], G, out_dtype=torch.float32)
    h, s = dev["hidden"].clone(), dev["scales"].clone()
    h[3, 100], h[17, 5] = float("nan"), float("inf")
    s[250, 2] = float("nan")
    got = arcs.w4_logits(h, dev["qweight"], s, G, out_dtype=torch.float32)
    rows = torch.ones(B, dtype=torch.bool)
    rows[[3, 17]] = False
    cols = torch.ones(V, dtype=torch.bool)
    cols[250] = False
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    assert got[3].isnan().all() and not got[17].isfinite().any() and got[:, 250].isnan().all()


@pytest.mark.parametrize("B,D,G", [(5, 96, 32), (16, 640, 64), (20, 96, 32), (70, 320, 64), (33, 128, 128)])
def test_an_infinite_scale_in_the_last_group(arcs, B, D, G):
    """A hidden size that ends inside a step: the infinite last scale gives what the definition
    gives, an infinity of the group's sign, and no NaN from beyond the end."""
    import torch
    host, dev = make(B, 150, D, G, False, "f32", seed=D + B)
    s = dev["scales"].clone()
    s[70, -1] = float("inf")
    dev["qweight"][70, -G // 2:] = 0xff  # 15 - 8 everywhere: no product with a zero level
    h = dev["hidden"].clone()
    h[:, -G:] = h[:, -G:].abs() + 0.25
    got = arcs.w4_logits(h, dev["qweight"], s, G, out_dtype=torch.float32)
    assert (got[:, 70] == float("inf")).all()
    assert got[:, :70].isfinite().all() and got[:, 71:].isfinite().all()


@pytest.mark.parametrize("B", [8, 40])
def test_side_stream_and_replays(arcs, B):
    """A call on another stream, and a captured call replayed on new inputs."""
    import torch
    V, D, G = 1000, 1024, 128
    host, dev = make(B, V, D, G, True, "bf16", seed=11)
    args = (dev["qweight"], dev["scales"], G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = arcs.w4_logits(dev["hidden"], *args, zeros=dev["zeros"], stream=side)
    side.synchronize()
    check(got, host, G, "bf16")
    h = dev["hidden"].clone()
    out = torch.empty((B, V), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    arcs.w4_logits(h, *args, zeros=dev["zeros"], out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        arcs.w4_logits(h, *args, zeros=dev["zeros"], out=out)
    for step in range(4):
        h.copy_(torch.randn(B, D, device="cuda").to(torch.bfloat16))
        graph.replay()
        want = arcs.w4_logits(h, *args, zeros=dev["zeros"])
        torch.cuda.synchronize()
        assert torch.equal(out, want), step


def test_logits_feed_the_sampler(arcs):
    """Head logits to the greedy token and to top_logprobs without a copy."""
    import torch
    B, V, D, G = 6, 5000, 512, 64
    host, dev = make(B, V, D, G, True, "bf16", seed=5)
    logits = arcs.w4_logits(dev["hidden"], dev["qweight"], dev["scales"], G, zeros=dev["zeros"])
    ids = arcs.argmax(logits)
    assert torch.equal(ids.long(), logits.float().argmax(dim=1))
    top, lp = arcs.top_logprobs(logits, 3)
    assert torch.equal(top[:, 0], ids)
    want = torch.log_softmax(logits.double(), dim=1).gather(1, top.long())
    assert (lp.double() - want).abs().max() < 1e-5


@pytest.mark.parametrize("B", [3, 40])
def test_rows_far_apart(arcs, B):
    """Offsets past 32 bits: weight rows 2 MiB apart (4.6 GB) and logit rows 2^30
    elements apart (B = 3: 6 GB)."""
    import torch
    V, D, G = 2200, 320, 64
    host, dev = make(B, V, D, G, True, "bf16", seed=19)
    want = arcs.w4_logits(dev["hidden"], dev["qweight"], dev["scales"], G, zeros=dev["zeros"])
    far = torch.empty(V << 21, dtype=torch.uint8, device="cuda").as_strided((V, D // 2), (1 << 21, 1))
    far.copy_(dev["qweight"])
    width = 1 << 30 if B == 3 else V
    out = torch.empty(B * width, dtype=torch.bfloat16, device="cuda").as_strided((B, V), (width, 1))
    got = arcs.w4_logits(dev["hidden"], far, dev["scales"], G, zeros=dev["zeros"], out=out)
    assert torch.equal(got, want)


@pytest.mark.parametrize("B,D,G", [(20, 32, 32), (70, 64, 64), (200, 128, 128), (33, 96, 32), (130, 320, 64)])
def test_the_last_weight_row_ends_the_allocation(arcs, B, D, G):
    """Hidden sizes that end inside a part of 256 k, and a vocabulary that ends
    inside a tile: what lies past the rows meets zeros."""
    import torch
    V = 129
    host, dev = make(B, V, D, G, True, "f32", seed=D)
    got = arcs.w4_logits(dev["hidden"], dev["qweight"], dev["scales"], G, zeros=dev["zeros"], out_dtype=torch.float32)
    check(got, host, G, "f32")


def test_binding_refuses(arcs):
    """Mistakes in tensors raise before anything is launched."""
    import torch
    host, dev = make(20, 64, 256, 64, True, "bf16", seed=1)
    h, q, s, z = dev["hidden"], dev["qweight"], dev["scales"], dev["zeros"]
    for args, kw in (((h.float(), q, s, 64), {}), ((h, q[:, :64], s, 64), {}), ((h, q, s, 32), {}),
                     ((h, q.to(torch.int32), s, 64), {}), ((h, q, s, 64), dict(zeros=z[:32])),
                     ((h, q, s, 64), dict(out=torch.empty(20, 63, device="cuda"))),
                     ((h, q, s, 64), dict(out=torch.empty(20, 64, device="cuda"), out_dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            arcs.w4_logits(*args, **kw)
    with pytest.raises(TypeError):
        arcs.w4_logits(h, q, s.half(), 64)
    with pytest.raises(arcs.ArcsError):
        arcs.w4_logits(h, q, s, 64, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(arcs.ArcsError):
        arcs.w4_logits(h[:, 1:225].as_strided((20, 192), (256, 1)), q[:, :96], s[:, :3], 64)
