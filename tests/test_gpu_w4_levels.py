"""arcs_w4_logits where the definition leaves no rounding, or one result only.

A level (q - z) is a whole number of at most 15, so a hidden state at a level
of zero adds nothing, an infinite one gives the infinity of its level's sign,
and whole hidden states with scales that are powers of two give whole sums:
the float32 logits then equal the definition's, whatever the order of the sums.
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


def make(B, V, D, G, zeros, seed, hidden=None, scale=None):
    """Device tensors and the float64 levels [V, D] and scales [V, D / G]."""
    import torch
    rng = np.random.default_rng(seed)
    h = rng.standard_normal((B, D)) if hidden is None else rng.choice(hidden, (B, D))
    q = rng.integers(0, 16, (V, D), dtype=np.uint8)
    z = rng.integers(0, 16, (V, D // G), dtype=np.uint8)
    s = rng.uniform(0.5, 1.5, (V, D // G)) / np.sqrt(D) if scale is None else rng.choice(scale, (V, D // G))
    s = torch.from_numpy(s.astype(np.float32)).cuda()
    dev = dict(hidden=torch.from_numpy(h.astype(np.float32)).to(torch.bfloat16).cuda(), q=q,
               z=z if zeros else np.full_like(z, 8), zeros=zeros, scales=s, G=G)
    return dev


def levels(x):
    V, D = x["q"].shape
    return (x["q"].astype(np.float64).reshape(V, -1, x["G"]) - x["z"][:, :, None]).reshape(V, D)


def definition(x):
    V, D = x["q"].shape
    w = levels(x).reshape(V, -1, x["G"]) * x["scales"].double().cpu().numpy()[:, :, None]
    return x["hidden"].double().cpu().numpy() @ w.reshape(V, D).T


def call(arcs, x, hidden=None, out_dtype=None):
    import torch
    q = torch.from_numpy(x["q"][:, 0::2] | (x["q"][:, 1::2] << 4)).cuda()
    z = torch.from_numpy(x["z"]).cuda() if x["zeros"] else None
    return arcs.w4_logits(x["hidden"] if hidden is None else hidden, q, x["scales"], x["G"], zeros=z,
                          out_dtype=torch.float32 if out_dtype is None else out_dtype)


SHAPES = [(1, 70, 64, 32), (3, 130, 192, 64), (16, 65, 640, 128), (20, 129, 96, 32), (32, 300, 4096, 128),
          (50, 70, 320, 64), (64, 257, 160, 32), (70, 130, 1024, 64), (129, 33, 384, 128)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("B,V,D,G", SHAPES + [(2, 40, 65536, 128), (20, 40, 65536, 32), (40, 40, 65536, 64),
                                              (66, 40, 65536, 128), (256, 40, 65536, 32)])
def test_whole_numbers_are_exact(arcs, B, V, D, G, zeros):
    """Hidden states -1, 0, 1 and scales 1, 2: every partial sum is a whole number of
    at most 2 * 15 * 65,536 < 2^24 in whatever order, so float32 holds it; every
    nibble, zero point and scale has its place in the answer."""
    import torch
    x = make(B, V, D, G, zeros, B + D, hidden=(-1.0, 0.0, 1.0), scale=(1.0, 2.0))
    want = torch.from_numpy(definition(x))
    assert torch.equal(call(arcs, x).double().cpu(), want)
    assert torch.equal(call(arcs, x, out_dtype=torch.bfloat16).cpu(), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("B,V,D,G", SHAPES)
def test_a_level_of_zero_adds_nothing(arcs, B, V, D, G, zeros):
    """A channel of 10,000 whose weights are at their zero point: the same bits as with
    that channel at 0 (x * 0 is 0, and adding 0 rounds nothing)."""
    import torch
    x = make(B, V, D, G, zeros, B + D)
    for d in (1, D // 2, D - 1):
        x["q"][:, d] = x["z"][:, d // G]
    h = x["hidden"].clone()
    h[:, [1, D // 2, D - 1]] = 0.0
    want = call(arcs, x, h)
    h[:, [1, D // 2, D - 1]] = 10000.0
    h[0, 1] = -10000.0
    assert torch.equal(call(arcs, x, h), want)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("B,V,D,G", SHAPES)
def test_infinite_hidden_states(arcs, B, V, D, G, zeros):
    """An infinity times the level: +inf, -inf, or NaN where the level is 0; other rows keep their bits."""
    import torch
    x = make(B, V, D, G, zeros, B + D)
    clean = call(arcs, x)
    h = x["hidden"].clone()
    edits = [(0, D - 1, float("inf")), (B - 1, 5, float("-inf"))][: B]
    for b, d, value in edits:
        h[b, d] = value
    got = call(arcs, x, h).cpu()
    lev = torch.from_numpy(levels(x))
    for b, d, value in edits:
        want = (lev[:, d] * value).float()
        assert torch.equal(got[b].nan_to_num(7.0), want.nan_to_num(7.0)), b
    assert torch.equal(got[1:B - 1], clean[1:B - 1].cpu())


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("B,V,D,G", SHAPES)
def test_large_hidden_states_do_not_overflow(arcs, B, V, D, G, zeros):
    """One channel of 2^124 a row, the others 0: at most 15 * 2^124 < 2^128, so each
    logit is finite, and exact at scales that are powers of two."""
    import torch
    x = make(B, V, D, G, zeros, B + D, scale=(2.0 ** -10, 2.0 ** -11))
    h = torch.zeros_like(x["hidden"])
    at = (torch.arange(B, device="cuda") * 37) % D
    h[torch.arange(B, device="cuda"), at] = 2.0 ** 124
    x["hidden"] = h
    assert torch.equal(call(arcs, x).double().cpu(), torch.from_numpy(definition(x)))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("B,V,D,G", SHAPES)
def test_small_hidden_states(arcs, B, V, D, G, zeros):
    """One channel of 2^-107 a row, the smallest that keeps every bit, the others 0."""
    import torch
    x = make(B, V, D, G, zeros, B + D, scale=(2.0 ** 10, 2.0 ** 11))
    h = torch.zeros_like(x["hidden"])
    at = (torch.arange(B, device="cuda") * 37) % D
    h[torch.arange(B, device="cuda"), at] = 2.0 ** -107
    x["hidden"] = h
    assert torch.equal(call(arcs, x).double().cpu(), torch.from_numpy(definition(x)))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("outlier", [False, True])
@pytest.mark.parametrize("B,V,D,G", [(4, 500, 4096, 128), (24, 500, 4096, 32), (64, 500, 4096, 64), (100, 64, 4096, 128),
                                     (200, 300, 8192, 64)])
def test_error_in_the_norm(arcs, B, V, D, G, zeros, outlier):
    """Products are exact (4 bits by 8), so the error is that of about D + D / G additions,
    each at most 2^-23 of a partial sum if they are truncated (2^-24 rounded).
    Partial sums of random terms are no larger than the logit in the root of the mean square,
    and the roundings do not add up in one direction: 2 * 2^-23 sqrt(D + D / G) of the norm,
    twice what that gives.  An outlier of 10,000 with its weights at the zero point changes nothing of it."""
    import torch
    x = make(B, V, D, G, zeros, B + V)
    if outlier:
        x["q"][:, 77] = x["z"][:, 77 // G]
        x["hidden"][:, 77] = 10000.0
    want = torch.from_numpy(definition(x))
    err = torch.linalg.norm(call(arcs, x).double().cpu() - want) / torch.linalg.norm(want)
    assert err <= 2.0 ** -22 * np.sqrt(D + D / G), float(err)
