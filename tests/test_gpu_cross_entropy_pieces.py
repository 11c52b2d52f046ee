"""The linear cross entropy where the vocabulary is taken in several pieces, at the largest
hidden size, and on the general kernel, against the definition in 64 bits on the GPU.

Bounds are those of test_gpu_cross_entropy.py: with e the error of a logit, 2^-24 (D + 2)
sum |h w| / T,
  |d lse| <= e + 2^-22 + 2^-24 (64 + V / 64) + 2^-22 |lse|,   |d loss| <= 2 e + the same,
and for gradients, dz off by the factor 1 + e + |d lse| and rounded to bfloat16 (2^-8) only
in the matrix kernels of bfloat16 calls (the general kernel holds it in float32: 2^-23
covers its arithmetic), 2^-24 for each addition, and half a step of the result's type.
The products of the 64-bit side are not rounded to anything that counts here.
"""

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


def make(N, V, D, dtype, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    w = (rnd(V, D) * 2.0 / D ** 0.5).to(dt)
    t = torch.randint(0, V, (N,), generator=gen, device="cuda")
    # targets in every piece, the last rows of the vocabulary among them
    t[: min(N, 8)] = V - 1 - torch.arange(min(N, 8), device="cuda") % V
    h = (rnd(N, D) + 2.0 * torch.rand(N, 1, generator=gen, device="cuda") * w[t].float()).to(dt)
    t[5::6] = IGNORE
    T = 0.3 + 1.7 * torch.rand(N, generator=gen, device="cuda")
    return h, w, t.to(torch.int32), T, rnd(N)


def check(arcs, N, V, D, dtype, rounded, seed=1, spread=0):
    import torch
    h, w, t, T, g = make(N, V, D, dtype, seed)
    if spread:  # upstream gradients from 2^-spread to 1
        g = g * torch.exp2(-spread * torch.arange(N, device="cuda") / (N - 1)).float()
    loss, lse = arcs.linear_cross_entropy(h, w, t, temperature=T)
    dh, dw = arcs.linear_cross_entropy_backward(h, w, t, lse, g, temperature=T)
    rows = torch.nonzero(t != IGNORE)[:, 0]
    off = torch.nonzero(t == IGNORE)[:, 0]
    assert (loss[off] == 0).all() and (lse[off] == 0).all() and (dh[off] == 0).all()
    h8, w8, T8, tr = h[rows].double(), w.double(), T[rows].double(), t[rows].long()
    z = h8 @ w8.t().contiguous() / T8[:, None]
    lse8 = torch.logsumexp(z, 1)
    loss8 = lse8 - z.gather(1, tr[:, None])[:, 0]
    e = 2.0 ** -24 * (D + 2) * (h8.abs() @ w8.abs().t().contiguous()).max(1).values / T8
    b = e + 2.0 ** -22 + 2.0 ** -24 * (64 + V / 64) + 2.0 ** -22 * lse8.abs()
    assert ((lse[rows].double() - lse8).abs() <= b).all()
    assert ((loss[rows].double() - loss8).abs() <= b + e).all()
    p = torch.exp(z - lse8[:, None])
    del z
    f = g[rows].double() / T8
    dz = p.clone()
    dz[torch.arange(len(rows), device="cuda"), tr] -= 1.0
    dz *= f[:, None]
    err = f.abs()[:, None] * p * (b + e)[:, None] + (2.0 ** -8 if rounded else 2.0 ** -23) * dz.abs()
    del p
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for got, want, er, size, terms in (
            (dh[rows], dz @ w8, err @ w8.abs(), dz.abs() @ w8.abs(), V),
            (dw, dz.t().contiguous() @ h8, err.t().contiguous() @ h8.abs(), dz.abs().t().contiguous() @ h8.abs(), N)):
        bound = 1.01 * (er + 2.0 ** -24 * (terms + 8) * size)
        bound = bound + half * (want.abs() + bound) + 1e-38
        over = (got.double() - want).abs() / bound
        assert (over <= 1).all(), float(over.max())
    # one gradient at a time: the same bits
    only = arcs.linear_cross_entropy_backward(h, w, t, lse, g, temperature=T, want_weight=False)[0]
    assert torch.equal(only, dh)
    only = arcs.linear_cross_entropy_backward(h, w, t, lse, g, temperature=T, want_hidden=False)[1]
    assert torch.equal(only, dw)


# 12,000 rows take pieces of 5,376 tokens (dz of a piece is held in about 256 MB): the last
# piece of 10,822 holds 70, of 10,753 one
@pytest.mark.parametrize("V", [10822, 10753])
@pytest.mark.parametrize("D,dtype,matrix", [(16, "f32", True), (15, "f32", False), (15, "bf16", False), (24, "bf16", True)])
def test_pieces_of_the_vocabulary(arcs, V, D, dtype, matrix):
    check(arcs, 12000, V, D, dtype, rounded=matrix and dtype == "bf16")


@pytest.mark.parametrize("N,V,D,dtype,matrix", [
    (3, 300, 65536, "bf16", True), (200, 130, 65536, "f32", True), (300, 200, 65536, "bf16", True),
    (5, 130, 65535, "bf16", False), (140, 70, 65535, "f32", False), (70, 300, 8192, "bf16", True),
])
def test_large_hidden_sizes(arcs, N, V, D, dtype, matrix):
    check(arcs, N, V, D, dtype, rounded=matrix and dtype == "bf16")


@pytest.mark.parametrize("N,V,D", [(3, 1000, 7), (130, 700, 161), (300, 2100, 33)])
def test_general_kernel_does_not_round_dz(arcs, N, V, D):
    """bfloat16 rows off the 16-byte grid: only the inputs and the results are bfloat16."""
    check(arcs, N, V, D, "bf16", rounded=False)


@pytest.mark.parametrize("D,dtype,matrix", [(64, "bf16", True), (64, "f32", True), (33, "bf16", False)])
def test_upstream_gradients_of_very_different_sizes(arcs, D, dtype, matrix):
    """dz is held in units of the call's largest upstream gradient: rows down to 2^-90 of it
    keep the precision of their own gradient."""
    check(arcs, 200, 1500, D, dtype, rounded=matrix and dtype == "bf16", spread=90)
