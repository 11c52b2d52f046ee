"""The linear layer, the adjustment of logits and the gradients' calls refuse bad host
arguments before launching anything (no GPU needed: the addresses below are never
dereferenced)."""

import ctypes
import re

import numpy as np
import pytest

from _util import HEADER, ensure_built, header_functions


@pytest.fixture(scope="module")
def arcs():
    return ensure_built()


BF16, F32 = 0, 1
NULL, BATCH, VOCAB, STRIDE, DTYPE, SMALL, MISALIGNED, HISTORY, HIDDEN = -1, -2, -3, -4, -5, -6, -8, -9, -15
ACT, BIAS, MASK, OVERLAP, NORM, PLAN = -17, -18, -19, -20, -21, -22
_buf = (ctypes.c_uint8 * 131072)()
BASE = (ctypes.addressof(_buf) + 255) // 256 * 256


def p(off=0):
    return None if off is None else ctypes.c_void_p(BASE + off)


def test_declared_and_described(arcs):
    for name in ("arcs_linear", "arcs_linear_backward", "arcs_linear_workspace_bytes", "arcs_linear_backward_workspace_bytes",
                 "arcs_adjust_logits", "arcs_gradient_plan", "arcs_gradient_plan_bytes", "arcs_gradient_norm",
                 "arcs_clip_gradients", "arcs_gradient_workspace_bytes"):
        assert name in header_functions() and hasattr(arcs.library(), name)
    src = open(HEADER).read()
    codes = {k: int(v) for k, v in re.findall(r"ARCS_((?:ERR|ROW)_[A-Z_]+) = (-?\d+)", src)}
    for name, code in codes.items():
        assert arcs.status_string(code) != "unknown status", name
        if hasattr(arcs, name):
            assert getattr(arcs, name) == code
    acts = {k.lower(): int(v) for k, v in re.findall(r"ARCS_ACT_([A-Z_]+) = (\d+)", src)}
    assert acts == arcs.ACTIVATIONS


LINEAR = dict(h=0, hs=64, w=0, ws=64, dt=BF16, N=40, V=100, D=64, b=0, act=0, cap=0.0, r=0, rs=100, out=4096, odt=BF16, os=100,
              pre=0, at=0, more=0, aligned=1)
BACK = dict(h=0, hs=64, w=0, ws=64, dt=BF16, N=40, V=100, D=64, act=0, cap=0.0, pre=0, g=0, gdt=BF16, gs=100, dh=0, dw=0, db=0, at=0,
            more=0, aligned=1)
SHARED = [
    (dict(h=None), NULL), (dict(w=None), NULL), (dict(dt=2), DTYPE), (dict(dt=-1), DTYPE), (dict(N=0), BATCH), (dict(N=-1), BATCH),
    (dict(N=2**22 + 1), BATCH), (dict(V=0), VOCAB), (dict(V=2**24 + 1), VOCAB), (dict(D=0), HIDDEN), (dict(D=65537, hs=65537, ws=65537), HIDDEN),
    (dict(hs=63), STRIDE), (dict(ws=63), STRIDE), (dict(act=-1), ACT), (dict(act=6), ACT), (dict(act=5), ACT), (dict(act=5, cap=-1.0), ACT),
    (dict(act=5, cap=float("nan")), ACT), (dict(act=5, cap=float("inf")), ACT), (dict(h=1), MISALIGNED), (dict(w=1), MISALIGNED),
    (dict(dt=F32, h=2), MISALIGNED), (dict(at=128, aligned=0, hs=65), MISALIGNED), (dict(more=-1, aligned=0, hs=65), SMALL),
    (dict(at=None, aligned=0, hs=65), NULL),
]


def linear(arcs, change):
    a = {**LINEAR, **change}
    need = arcs.library().arcs_linear_workspace_bytes(a["N"], a["V"], a["D"], a["dt"], a["aligned"])
    return arcs.library().arcs_linear(p(a["h"]), a["hs"], p(a["w"]), a["ws"], a["dt"], a["N"], a["V"], a["D"], p(a["b"]), a["act"], a["cap"],
                                      p(a["r"]), a["rs"], p(a["out"]), a["odt"], a["os"], p(a["pre"]), p(a["at"]), need + a["more"], None)


def backward(arcs, change):
    a = {**BACK, **change}
    need = arcs.library().arcs_linear_backward_workspace_bytes(a["N"], a["V"], a["D"], a["dt"], a["aligned"])
    return arcs.library().arcs_linear_backward(p(a["h"]), a["hs"], p(a["w"]), a["ws"], a["dt"], a["N"], a["V"], a["D"], a["act"], a["cap"],
                                               p(a["pre"]), p(a["g"]), a["gdt"], a["gs"], p(a["dh"]), p(a["dw"]), p(a["db"]), p(a["at"]),
                                               need + a["more"], None)


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(out=None), NULL), (dict(odt=7), DTYPE), (dict(os=99), STRIDE), (dict(rs=99), STRIDE), (dict(b=1), MISALIGNED), (dict(r=1), MISALIGNED),
    (dict(pre=1), MISALIGNED), (dict(out=1), MISALIGNED), (dict(odt=F32, out=2), MISALIGNED), (dict(N=2**21, V=2**20, os=2**20, rs=2**20), BATCH),
    (dict(out=0, r=0, odt=F32), OVERLAP), (dict(out=0, r=0, rs=101), OVERLAP),
    # in place of the hidden states, whose rows other workgroups still read
    (dict(V=64, rs=64, os=64, out=0, r=0, h=0, w=32768, b=None, pre=None), OVERLAP),
    (dict(out=8192, r=None, h=0, w=9008, b=None, pre=None), OVERLAP), (dict(out=16384, r=None, h=0, w=32768, b=24000, pre=None), OVERLAP),
    (dict(out=16384, r=None, h=0, w=32768, b=None, pre=20000), OVERLAP), (dict(out=16384, r=40000, h=0, w=32768, b=None, pre=44000), OVERLAP),
    (dict(out=16384, r=None, h=0, w=32768, b=None, pre=4000), OVERLAP),
])
def test_linear(arcs, change, status):
    assert linear(arcs, change) == status


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(g=None), NULL), (dict(dh=None, dw=None, db=None), NULL), (dict(act=4, pre=None), NULL), (dict(gdt=2), DTYPE), (dict(gs=99), STRIDE),
    (dict(g=1), MISALIGNED), (dict(gdt=F32, g=2), MISALIGNED), (dict(pre=1), MISALIGNED), (dict(dh=1), MISALIGNED), (dict(dw=1), MISALIGNED),
    (dict(db=1), MISALIGNED), (dict(V=2**21 - 7), VOCAB), (dict(more=-1), SMALL), (dict(at=None), NULL), (dict(at=64), MISALIGNED),
    (dict(dh=0, dw=None, db=None), OVERLAP), (dict(dh=None, dw=12000, db=None, h=30000, w=0, pre=None, g=20000), OVERLAP),
    (dict(dh=40000, dw=44000, db=None, h=30000, w=0, pre=None, g=20000), OVERLAP),
    (dict(dh=None, dw=None, db=21000, h=30000, w=0, pre=None, g=20000), OVERLAP),
])
def test_linear_backward(arcs, change, status):
    assert backward(arcs, change) == status


def test_linear_workspaces(arcs):
    f, b = arcs.library().arcs_linear_workspace_bytes, arcs.library().arcs_linear_backward_workspace_bytes
    assert f(16, 100, 63, BF16, 0) == 0  # few rows need none
    assert f(100, 1000, 63, BF16, 0) >= 1100 * 64 * 2 and b(100, 1000, 64, F32, 1) >= 100 * 1000 * 4
    for bad in ((0, 1, 1, 0), (1, 0, 1, 0), (1, 1, 0, 0), (1, 1, 65537, 0), (1, 1, 1, 3), (2**22 + 1, 1, 1, 0)):
        assert f(*bad, 0) == 0 and b(*bad, 0) == 0
    for sizes in ((17, 5, 8), (300, 4096, 4096), (4096, 129280, 64), (1, 1, 1)):
        for dt in (BF16, F32):
            assert f(*sizes, dt, 0) >= f(*sizes, dt, 1) and b(*sizes, dt, 0) >= b(*sizes, dt, 1)


ADJUST = dict(z=0, dt=BF16, B=4, V=100, rs=100, P=0, hi=0, ho=0, bi=0, bv=0, bo=0, m=0, ms=4, mw=4, mr=0, out=8192, odt=BF16, os=100, st=0)


@pytest.mark.parametrize("change,status", [
    (dict(z=None), NULL), (dict(out=None), NULL), (dict(dt=2), DTYPE), (dict(odt=2), DTYPE), (dict(B=0), BATCH), (dict(B=2**31), BATCH),
    (dict(B=2**30, V=5000, rs=5000, os=5000, mw=157), BATCH), (dict(V=0), VOCAB), (dict(V=2**31), VOCAB), (dict(rs=99), STRIDE), (dict(os=99), STRIDE),
    (dict(hi=None), HISTORY), (dict(ho=None), HISTORY), (dict(P=None), NULL), (dict(bi=None), BIAS), (dict(bv=None), BIAS), (dict(bo=None), BIAS),
    (dict(bi=None, bv=None), BIAS), (dict(m=None), MASK), (dict(mr=None, ms=3), MASK), (dict(ms=0), MASK), (dict(ms=-1), MASK), (dict(mw=3), STRIDE),
    (dict(z=1), MISALIGNED), (dict(P=2), MISALIGNED), (dict(hi=2), MISALIGNED), (dict(ho=4), MISALIGNED), (dict(bi=1), MISALIGNED),
    (dict(bv=2), MISALIGNED), (dict(bo=4), MISALIGNED), (dict(m=2), MISALIGNED), (dict(mr=1), MISALIGNED), (dict(out=1), MISALIGNED),
    (dict(odt=F32, out=2), MISALIGNED), (dict(st=2), MISALIGNED), (dict(out=0, odt=F32), OVERLAP), (dict(out=0, os=104), OVERLAP),
    (dict(out=2), OVERLAP), (dict(out=798), OVERLAP), (dict(out=100, rs=120, os=120), OVERLAP),
])
def test_adjust_logits(arcs, change, status):
    a = {**ADJUST, **change}
    assert arcs.library().arcs_adjust_logits(p(a["z"]), a["dt"], a["B"], a["V"], a["rs"], p(a["P"]), p(a["hi"]), p(a["ho"]), p(a["bi"]),
                                             p(a["bv"]), p(a["bo"]), p(a["m"]), a["ms"], a["mw"], p(a["mr"]), p(a["out"]), a["odt"],
                                             a["os"], p(a["st"]), None) == status


def records(arcs, *rows):
    r = np.zeros(len(rows), arcs.TENSOR_DTYPE)
    for i, row in enumerate(rows):
        r[i] = row
    return r


def test_gradient_plans(arcs):
    lib = arcs.library()
    plan_of = lib.arcs_gradient_plan
    good = records(arcs, (BASE, BASE, 10000, BF16, BF16), (0, 0, 0, F32, F32), (BASE + 32768, 0, 5, F32, BF16))
    size = lib.arcs_gradient_plan_bytes(good.ctypes.data, 3)
    assert size == 4 * 32  # three pieces of the first tensor, one of the last
    plan = np.zeros(size, np.uint8)
    assert plan_of(good.ctypes.data, 3, plan.ctypes.data, size) == 0
    words = plan.view(np.uint64).reshape(4, 4)
    counts = plan.view(np.int32).reshape(4, 8)
    assert words[:, 0].tolist() == [BASE, BASE + 8192, BASE + 16384, BASE + 32768] and words[3, 1] == 0
    assert counts[:, 4].tolist() == [4096, 4096, 1808, 5] and counts[:, 5].tolist() == [1, 1, 1, 0] and counts[:, 6].tolist() == [1, 1, 1, 1]
    assert plan_of(good.ctypes.data, 3, plan.ctypes.data, size - 32) == PLAN
    assert plan_of(good.ctypes.data, 3, None, size) == NULL
    assert plan_of(None, 3, plan.ctypes.data, size) == NULL and plan_of(good.ctypes.data, -1, plan.ctypes.data, size) == BATCH
    assert plan_of(None, 0, None, 0) == 0
    for row, status in (((BASE, BASE, -1, BF16, BF16), PLAN), ((BASE, BASE, 2**40 + 1, BF16, BF16), PLAN), ((0, 0, 1, BF16, BF16), NULL),
                        ((BASE + 1, 0, 4, BF16, BF16), MISALIGNED), ((BASE + 2, 0, 4, F32, F32), MISALIGNED), ((BASE, BASE + 2, 4, BF16, F32), MISALIGNED),
                        ((BASE, BASE, 4, BF16, F32), OVERLAP), ((BASE, BASE, 4, 2, BF16), DTYPE), ((BASE, BASE, 4, BF16, 5), DTYPE)):
        bad = records(arcs, row)
        assert plan_of(bad.ctypes.data, 1, plan.ctypes.data, size) == status
        assert lib.arcs_gradient_plan_bytes(bad.ctypes.data, 1) == 0


@pytest.mark.parametrize("change,status", [
    (dict(plan=None), NULL), (dict(norm=None), NULL), (dict(size=33), PLAN), (dict(plan=4), MISALIGNED), (dict(norm=2), MISALIGNED),
    (dict(more=-1), SMALL), (dict(at=None), NULL), (dict(at=8), MISALIGNED),
])
def test_gradient_calls(arcs, change, status):
    lib = arcs.library()
    a = {**dict(plan=0, size=96, norm=0, at=0, more=0), **change}
    need = lib.arcs_gradient_workspace_bytes(a["size"]) + a["more"]
    assert lib.arcs_gradient_norm(p(a["plan"]), a["size"], p(a["norm"]), p(a["at"]), need, None) == status
    assert lib.arcs_clip_gradients(p(a["plan"]), a["size"], 1.0, p(a["norm"]), p(a["at"]), need, None) == status


def test_max_norm(arcs):
    for bad in (-1.0, float("nan"), -float("inf")):
        assert arcs.library().arcs_clip_gradients(p(), 96, bad, p(), p(), 4096, None) == NORM


def test_binding_checks_tensors_first(arcs):
    """Shape, type and device mistakes raise before the library is called."""
    torch = pytest.importorskip("torch")
    h, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        arcs.linear(h, w)  # host tensors
    with pytest.raises(ValueError):
        arcs.linear_backward(h, w, torch.zeros(2, 8))
    with pytest.raises(ValueError):
        arcs.adjust_logits(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        arcs.TensorList([torch.zeros(4)])
