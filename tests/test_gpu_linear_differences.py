"""The linear layer's gradients against differences of its own outputs.

The loss is sum(grad out) in 64 bits over float32 outputs.  Along a direction d of one operand its
central difference over steps s and -s is the derivative plus what the step is too long by; the latter is
taken from the formula in 64 bits (its difference minus its derivative, at the same s), so what is left
is rounding: of the outputs, over s, and of the gradient.  An output is off by e_y = 1.13 e_z + 21 u |out|,
e_z = u (D + 18) (|hidden| |weight| + |bias|) with u = 2^-24 (20 u for the activation, one rounding; no slope is
above 1.13), the gradient by the bounds of test_gpu_linear.py.  Directions are the gradient's elements times
0.5 to 1.5, so that every element counts and the derivative is large: the tolerance has to be
below 5 % of it, so a set of elements that is missing or wrong by more than that fails.  (Most of the tolerance
is e_z over the step: with D = 133 and |hidden| |weight| about 0.64 sqrt(133), u 151 7.4 / s = 5.3e-4 for each of
300 x 520 outputs of mean |grad| 0.8, 67 of a derivative of some 6,600, and 4,500
where the activation halves it.)
"""

import math

import pytest

from _util import ensure_built
from test_gpu_linear import CAP, U, make, slope, value

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -3


@pytest.fixture(scope="module")
def arcs():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return ensure_built()


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "softcap"])
@pytest.mark.parametrize("N,V,D", [(7, 24, 16), (21, 24, 16), (130, 203, 72), (300, 520, 133)])
def test_each_operand(arcs, N, V, D, act):
    import torch
    s = make(N, V, D, torch.float32, 9)
    g = torch.Generator(device="cuda").manual_seed(8)
    grad = torch.randn(N, V, generator=g, device="cuda")
    names = ("hidden", "weight", "bias")
    x = [s[k] for k in names]
    _, pre = arcs.linear(*x, activation=act, softcap=CAP, residual=s["residual"], want_pre=True)
    got = arcs.linear_backward(x[0], x[1], grad, pre=None if act == "none" else pre, activation=act, softcap=CAP, want_bias=True)

    def exact(x):
        h, w, b = (t.double() for t in x)
        z = h @ w.T.contiguous() + b
        return z, value(z, act) + s["residual"].double()

    z, _ = exact(x)
    dz = grad.double() * slope(z, act)
    grads = (dz @ x[1].double(), dz.T.contiguous() @ x[0].double(), dz.sum(0))
    # of the gradients: each term's slope, 18 u (1 + |z|) of it, and the sums
    e_dz = grad.double().abs() * 18 * U * (1 + z.abs()) + U * dz.abs()
    aw, ah = x[1].double().abs(), x[0].double().abs()
    e_pre = 2 * 1.13 * U * (D + 18) * (ah @ aw.T.contiguous() + x[2].double().abs()) * grad.double().abs()  # no activation's second derivative is above 2
    e_dz = e_dz + e_pre
    errors = (U * (V + 18) * (dz.abs() @ aw) + e_dz @ aw, U * (N + 18) * (dz.abs().T.contiguous() @ ah) + e_dz.T.contiguous() @ ah,
              U * (N + 8) * dz.abs().sum(0) + e_dz.sum(0))
    for i in range(3):
        d = (grads[i] * (0.5 + torch.rand(grads[i].shape, generator=g, device="cuda")))
        d = (d / d.square().mean().sqrt() * (1 / math.sqrt(D) if i < 2 else 1.0)).float()
        ends = []
        for k in (STEP, -STEP):
            at = list(x)
            at[i] = x[i] + k * d
            ends.append(at)
        # the step that was really made, operands being rounded
        d64 = (ends[0][i].double() - ends[1][i].double()) / (2 * STEP)
        outs = [arcs.linear(*at, activation=act, softcap=CAP, residual=s["residual"]).double() for at in ends]
        found = float((grad.double() * (outs[0] - outs[1])).sum()) / (2 * STEP)
        sides = [exact(at)[1] for at in ends]
        too_long = float((grad.double() * (sides[0] - sides[1])).sum()) / (2 * STEP) - float((grads[i] * d64).sum())
        want = float((got[i].double() * d64).sum())
        far = 0.0
        for at, y in zip(ends, sides):
            e_z = U * (D + 18) * (at[0].double().abs() @ at[1].double().abs().T.contiguous() + at[2].double().abs())
            far += float((grad.double().abs() * (1.13 * e_z + 21 * U * (y.abs() + s["residual"].double().abs()))).sum()) / (2 * STEP)
        far += float((errors[i] * d64.abs()).sum())
        assert far < 0.05 * abs(want), (names[i], far, want)
        assert abs(found - too_long - want) <= far, (names[i], found, too_long, want, far)
