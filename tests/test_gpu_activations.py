"""The values and slopes of arcs_linear's activations, relative to themselves, against 64 bits.

With u = 2^-24 (half a step of float32).  exp2 and the reciprocal are off by 2 u, and each operation
rounds once:
  h     the square root of the exponential: 2 for exp2, 1 for the step that its argument's rest makes: 3 u.
  tail  H of Phi(-a) = H h^2: 6.3 for the polynomial with the roundings of its steps (measured over 0 .. 14
        in float32 where the fused steps round once), 2 more for the reciprocal in its argument: 8.3 u.
  value z < 0: h twice (6), tail (8.3), three products: 17.3; z >= 0: 1 - tail h^2, where what is taken away is
        at most half of 1 and off by 16.3, and two roundings: 18.3 (tail h^2 is at most what remains).
        z (h^2) / (1 + h^2): h twice (6), three for its denominator with the exponential's error in it at half,
        2 for the reciprocal, three products: 14.5.
        softcap, u = z / c: its two roundings and the two of the exponential's argument reach tanh u at most
        once, as 4, 2 for exp2, two sums, the reciprocal (2) and two products: 12; below 1/4 less.
  slope two terms, each of at most two exponentials h, a tail or two reciprocals, and ten roundings:
        6 + 8.3 + 10 of each of the two.
        softcap: 4 e / (1 + e)^2 with e = exp(-2 |u|): four roundings of the argument, 8 |u|, 2 for exp2, two
        reciprocals of a sum (6), three products: 11 + 8 |u| of itself.
So values are within 20 u of themselves, and slopes within 32 u of the sum of their terms' sizes, the
softcap's within 16 (1 + |u|) of themselves.
Values below the smallest normal number are off by steps of 2^-149; the exponential h^2 of a
slope is below it from 87 on, and multiplied by at most 2^12.
"""

import math

import numpy as np
import pytest

from _util import ensure_built

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


def exact(act, z):
    """act(z), and the two terms of act'(z)."""
    if act == "gelu":
        phi = np.vectorize(math.erfc)(z / -math.sqrt(2)) / 2
        return z * phi, phi, z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    twice = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    slope = 1.0 if act == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    small = np.exp(-np.abs(twice))
    half = np.where(z >= 0, 1.0, small) / (1 + small)
    return z * half, half, z * slope * small / (1 + small) ** 2


def points():
    """From the smallest numbers to far beyond where values vanish, both signs."""
    rng = np.random.default_rng(5)
    a = np.concatenate([np.linspace(0, 20, 4001), np.linspace(20, 200, 901), 10.0 ** rng.uniform(-38, 0, 1000), 10.0 ** rng.uniform(2, 38, 97)])
    return np.concatenate([a, -a]).astype(np.float32)


ACTS = ["gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("rows", [1, 9, 20])
@pytest.mark.parametrize("act", ACTS)
def test_values(arcs, act, rows):
    import torch
    z = points()
    w = torch.zeros(len(z), 4, device="cuda")
    w[:, 0] = torch.from_numpy(z)
    h = torch.zeros(rows, 4, device="cuda")
    h[:, 0] = 1.0
    out, pre = arcs.linear(h, w, activation=act, want_pre=True)
    assert torch.equal(pre[-1].cpu(), torch.from_numpy(z))
    with np.errstate(all="ignore"):
        want = exact(act, z.astype(np.float64))[0]
    for row in (out[0], out[-1]):
        far = np.abs(row.cpu().numpy().astype(np.float64) - want) - 20 * U * np.abs(want) - 2.0 ** -147
        assert far.max() <= 0, (float(z[far.argmax()]), float(row[far.argmax()]), want[far.argmax()])


@pytest.mark.parametrize("rows", [1, 20])
@pytest.mark.parametrize("cap", [2.0 ** -100, 1e-3, 1.5, 30.0, 1e10, 2.0 ** 100])
def test_softcap(arcs, cap, rows):
    """From pre-activations whose z / c float32 does not hold to those far beyond c."""
    import torch
    z = points()
    w = torch.zeros(len(z), 4, device="cuda")
    w[:, 0] = torch.from_numpy(z)
    h = torch.zeros(rows, 4, device="cuda")
    h[:, 0] = 1.0
    got = arcs.linear(h, w, activation="softcap", softcap=cap)[-1].cpu().numpy().astype(np.float64)
    c = float(np.float32(cap))
    want = c * np.tanh(z.astype(np.float64) / c)
    far = np.abs(got - want) - 20 * U * np.abs(want) - 2.0 ** -147
    assert far.max() <= 0, (float(z[far.argmax()]), got[far.argmax()], want[far.argmax()])


@pytest.mark.parametrize("cap", [2.0 ** -100, 1e-3, 1.5, 30.0, 1e10, 2.0 ** 100])
def test_the_slope_of_softcap(arcs, cap):
    """1 - tanh^2 (z / c), which is below the smallest normal number past 44."""
    import torch
    z = points()
    h, w = torch.zeros(1, 4, device="cuda"), torch.zeros(len(z), 4, device="cuda")
    pre = torch.from_numpy(z).cuda()[None]
    _, _, db = arcs.linear_backward(h, w, torch.ones_like(pre), pre=pre, activation="softcap", softcap=cap, want_bias=True)
    with np.errstate(all="ignore"):
        u = np.minimum(np.abs(z.astype(np.float64)) / float(np.float32(cap)), 300.0)
        want = 1 / np.cosh(u) ** 2
    far = np.abs(db.cpu().numpy().astype(np.float64) - want) - 16 * U * (1 + u) * want - 2.0 ** -123
    assert far.max() <= 0, (float(z[far.argmax()]), float(db[far.argmax()]), want[far.argmax()])


@pytest.mark.parametrize("act", ACTS)
def test_slopes(arcs, act):
    import torch
    z = points()
    h, w = torch.zeros(1, 4, device="cuda"), torch.zeros(len(z), 4, device="cuda")
    pre = torch.from_numpy(z).cuda()[None]
    _, _, db = arcs.linear_backward(h, w, torch.ones_like(pre), pre=pre, activation=act, want_bias=True)
    with np.errstate(all="ignore"):
        _, a, b = exact(act, z.astype(np.float64))
    a, b = np.nan_to_num(a), np.nan_to_num(b)
    far = np.abs(db.cpu().numpy().astype(np.float64) - (a + b)) - 32 * U * (np.abs(a) + np.abs(b)) - 2.0 ** -137
    assert far.max() <= 0, (float(z[far.argmax()]), float(db[far.argmax()]), (a + b)[far.argmax()])


@pytest.mark.parametrize("act", ACTS)
def test_what_is_not_finite(arcs, act):
    """NaN stays NaN, and the ends of the range are the limits (z act(z) has none at -inf, where
    its formula is infinity times zero)."""
    import torch
    z = torch.tensor([float("nan"), float("inf"), 3e38, -3e38], device="cuda")
    w = torch.zeros(4, 4, device="cuda")
    w[:, 0] = z
    for rows in (1, 20):
        h = torch.zeros(rows, 4, device="cuda")
        h[:, 0] = 1.0
        w0 = w.clone()
        w0[1, 0] = 3e38  # infinity times the other columns' zeros would be NaN
        y = arcs.linear(h, w0, activation=act)[-1]
        assert y[0].isnan() and float(y[1]) == float(y[2]) == float(w0[2, 0]) and float(y[3]) == 0.0
    pre = z[None].contiguous()
    _, _, db = arcs.linear_backward(h[:1], w, torch.ones_like(pre), pre=pre, activation=act, want_bias=True)
    assert db[0].isnan() and float(db[1]) == float(db[2]) == 1.0 and float(db[3]) == 0.0
