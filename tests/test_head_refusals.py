"""The head's entry points refuse bad host arguments before launching anything
(no GPU needed: the addresses below are never dereferenced)."""

import ctypes
import re

import pytest

from _util import HEADER, ensure_built, header_functions


@pytest.fixture(scope="module")
def arcs():
    return ensure_built()


BF16, F32 = 0, 1
NULL, DTYPE, BATCH, VOCAB, STRIDE, SMALL, MISALIGNED, HIDDEN, GROUP = -1, -5, -2, -3, -4, -6, -8, -15, -16
_buf = (ctypes.c_uint8 * 4096)()
BASE = (ctypes.addressof(_buf) + 255) // 256 * 256


def p(off=0):
    return ctypes.c_void_p(BASE + off)


def test_declared_and_described(arcs):
    for name in ("arcs_w4_logits", "arcs_linear_cross_entropy", "arcs_linear_cross_entropy_backward",
                 "arcs_linear_cross_entropy_workspace_bytes"):
        assert name in header_functions() and hasattr(arcs.library(), name)
    for code in (arcs.ERR_BAD_HIDDEN, arcs.ERR_BAD_GROUP, arcs.ROW_BAD_TARGET):
        assert arcs.status_string(code) != "unknown status"
    src = open(HEADER).read()
    defs = {k: int(v) for k, v in re.findall(r"#define (ARCS_[A-Z0-9_]+) (\d+)", src)}
    assert defs["ARCS_MAX_HIDDEN"] == arcs.MAX_HIDDEN


W4 = dict(hidden=0, B=4, D=256, hs=256, q=0, V=100, qs=128, sc=0, sdt=BF16, ss=2, z=0, zs=2, g=128, out=0, odt=BF16,
          ls=100, ws=0, more=0)


@pytest.mark.parametrize("change,status", [
    (dict(hidden=None), NULL), (dict(q=None), NULL), (dict(sc=None), NULL), (dict(out=None), NULL),
    (dict(sdt=2), DTYPE), (dict(odt=-1), DTYPE), (dict(B=0), BATCH), (dict(B=-1), BATCH), (dict(B=2**31), BATCH), (dict(B=2**20, V=2**17, ls=2**17), BATCH),
    (dict(V=0), VOCAB), (dict(V=2**31), VOCAB), (dict(D=0, hs=0), HIDDEN), (dict(D=65664, hs=65664, qs=32832), HIDDEN),
    (dict(g=0), GROUP), (dict(g=16), GROUP), (dict(g=256), GROUP), (dict(g=-32), GROUP), (dict(D=192, g=128), GROUP),
    (dict(D=250), GROUP), (dict(hs=255), STRIDE), (dict(qs=127), STRIDE), (dict(ss=1), STRIDE), (dict(zs=1), STRIDE),
    (dict(ls=99), STRIDE), (dict(qs=2**21 + 16), STRIDE), (dict(ss=2**21 + 1), STRIDE), (dict(hidden=8), MISALIGNED), (dict(hs=260), MISALIGNED), (dict(q=4), MISALIGNED),
    (dict(qs=136), MISALIGNED), (dict(sc=1), MISALIGNED), (dict(sdt=F32, sc=2), MISALIGNED), (dict(out=1), MISALIGNED),
    (dict(odt=F32, out=2), MISALIGNED), (dict(B=40, ws=None), NULL), (dict(B=40, ws=16), MISALIGNED),
    (dict(B=40, more=-1), SMALL),
])
def test_w4_logits(arcs, change, status):
    a = {**W4, **change}
    at = {k: None if a[k] is None else p(a[k]) for k in ("hidden", "q", "sc", "z", "out", "ws")}
    need = arcs.w4_logits_workspace_bytes(a["B"], a["D"], a["g"])
    assert arcs.library().arcs_w4_logits(at["hidden"], a["B"], a["D"], a["hs"], at["q"], a["V"], a["qs"], at["sc"],
                                         a["sdt"], a["ss"], at["z"], a["zs"], a["g"], at["out"], a["odt"], a["ls"],
                                         at["ws"], need + a["more"], None) == status


CE = dict(h=0, hs=64, w=0, ws=64, dt=BF16, N=4, V=100, D=64, t=0, T=0, loss=0, lse=0, st=0, ws_at=0, ws_bytes=None,
          g=0, dh=0, dw=0)
SHARED = [
    (dict(h=None), NULL), (dict(w=None), NULL), (dict(t=None), NULL), (dict(lse=None), NULL), (dict(ws_at=None), NULL),
    (dict(dt=2), DTYPE), (dict(N=0), BATCH), (dict(N=-5), BATCH), (dict(N=2**31), BATCH), (dict(N=2**23 + 1), BATCH),
    (dict(N=2**21, V=2**21), BATCH), (dict(V=0), VOCAB), (dict(V=2**31), VOCAB), (dict(D=0), HIDDEN),
    (dict(D=65537, hs=65537, ws=65537), HIDDEN), (dict(hs=63), STRIDE), (dict(ws=63), STRIDE), (dict(h=1), MISALIGNED),
    (dict(w=1), MISALIGNED), (dict(dt=F32, h=2), MISALIGNED), (dict(t=2), MISALIGNED), (dict(T=2), MISALIGNED),
    (dict(lse=2), MISALIGNED), (dict(ws_at=128), MISALIGNED), (dict(ws_bytes=-1), SMALL), (dict(ws_bytes=0), SMALL),
]


def call(arcs, change, backward):
    lib = arcs.library()
    a = {**CE, **change}
    at = {k: None if a[k] is None else p(a[k]) for k in ("h", "w", "t", "T", "loss", "lse", "st", "ws_at", "g", "dh", "dw")}
    need = lib.arcs_linear_cross_entropy_workspace_bytes(a["N"], a["V"], a["D"], a["dt"], int(backward))
    size = need if a["ws_bytes"] is None else max(0, need + a["ws_bytes"]) if a["ws_bytes"] else 0
    head = (at["h"], a["hs"], at["w"], a["ws"], a["dt"], a["N"], a["V"], a["D"], at["t"], -100, at["T"])
    if backward:
        return lib.arcs_linear_cross_entropy_backward(*head, at["lse"], at["g"], at["dh"], at["dw"], at["ws_at"], size, None)
    return lib.arcs_linear_cross_entropy(*head, at["loss"], at["lse"], at["st"], at["ws_at"], size, None)


@pytest.mark.parametrize("change,status", SHARED + [(dict(loss=None), NULL), (dict(loss=2), MISALIGNED),
                                                    (dict(st=2), MISALIGNED)])
def test_cross_entropy(arcs, change, status):
    assert call(arcs, change, False) == status


@pytest.mark.parametrize("change,status", SHARED + [(dict(g=None), NULL), (dict(dh=None, dw=None), NULL),
                                                    (dict(g=2), MISALIGNED), (dict(dh=1), MISALIGNED),
                                                    (dict(dw=1), MISALIGNED)])
def test_cross_entropy_backward(arcs, change, status):
    assert call(arcs, change, True) == status


def test_workspace_sizes(arcs):
    w4 = arcs.w4_logits_workspace_bytes
    assert w4(16, 4096, 128) == 0 and w4(17, 4096, 128) >= 32 * 4096 * 2 and w4(300, 96, 32) >= 384 * 96 * 2
    assert w4(0, 128, 32) == 0 and w4(64, 128, 48) == 0 and w4(64, 0, 32) == 0
    need = arcs.linear_cross_entropy_workspace_bytes
    assert need(4096, 129280, 4096, BF16) >= 256 and need(1, 1, 1, F32, True) >= 256
    for bad in ((0, 10, 10, 0), (10, 0, 10, 0), (10, 10, 0, 0), (10, 10, 65537, 0), (10, 10, 10, 7), (2**23 + 1, 10, 10, 0)):
        assert need(*bad) == 0 and need(*bad, True) == 0
    # a piece of the vocabulary, not all of it: far below the logits' size
    assert need(8192, 262144, 4096, BF16, True) < 8192 * 262144 * 2 // 4


def test_binding_checks_tensors_first(arcs):
    """Shape, type and device mistakes raise before the library is called."""
    torch = pytest.importorskip("torch")
    h, w, t = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        arcs.linear_cross_entropy(h, w, t)  # host tensors
    with pytest.raises(ValueError):
        arcs.w4_logits(h, torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2), 32)
