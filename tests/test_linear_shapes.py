"""The rule that chooses the linear layer's tiles, and the sizes by which the tests reach each of them (no GPU needed)."""

import ctypes
import os
import re
import subprocess

import pytest

from _util import ROOT
from linear_tile_sizes import TILES

CSRC = os.path.join(ROOT, "decode_step_token_row_amd", "csrc")
MODES = ["forward", "dhidden", "dweight"]


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    """linear_shape, compiled for the host."""
    at = tmp_path_factory.mktemp("shape")
    source = at / "shape.cpp"
    source.write_text('#include "linear_shape.hpp"\n'
                      'extern "C" void shape(int mode, int64_t M, int64_t N, int64_t K, int bf16, int32_t* out) {\n'
                      "  const arcs::LinearShape s = arcs::linear_shape(mode, M, N, K, bf16 != 0);\n"
                      "  out[0] = s.columns, out[1] = s.rows, out[2] = s.workers;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(source), "-o", str(at / "shape.so")], check=True)
    lib = ctypes.CDLL(str(at / "shape.so"))
    lib.shape.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_void_p]

    def call(mode, dtype, N, V, D):
        each = 8 if dtype == "bf16" else 4
        M, n, K = {"forward": (V, N, (D + each - 1) // each * each), "dhidden": (D, N, V), "dweight": (D, V, N)}[mode]
        out = (ctypes.c_int32 * 3)()
        lib.shape(MODES.index(mode), M, n, K, dtype == "bf16", out)
        tiles = -(-M // out[0]) * -(-n // out[1])
        return tuple(out), tiles, -(-K // (64 if dtype == "bf16" else 32))

    return call


def built():
    """(product, type, columns, rows) of every tile kernel that the sources instantiate, and how many
    of its workgroups the card's 256 compute units hold by their LDS."""
    kinds = {}
    for mode in MODES:
        for dtype in ("bf16", "f32"):
            text = open(os.path.join(CSRC, f"linear_{mode}_{dtype}.hip")).read()
            for wm, wn, mt, nt, deep in re.findall(r"launch_linear_tile<\w+, \w+, (\d), (\d), (\d), (\d), (\d)>", text):
                columns, rows, waves = int(wm) * int(mt) * 32, int(wn) * int(nt) * 32, int(wm) * int(wn)
                lds = int(deep) * (columns + rows) * 128 + waves * 4096
                kinds[mode, dtype, columns, rows] = 256 * (163840 // lds)
    return kinds


@pytest.mark.parametrize("case", TILES, ids=lambda c: "-".join(map(str, c)))
def test_the_sizes_take_their_tiles(shape, case):
    mode, dtype, N, V, D, columns, rows, workers, more = case
    got, tiles, steps = shape(mode, dtype, N, V, D)
    assert got == (columns, rows, workers) and steps >= 4
    assert more == (workers == 0 and tiles > built()[mode, dtype, columns, rows])


def test_the_sizes_reach_every_tile_kernel():
    kinds = built()
    assert len(kinds) == 19
    whole = {c[:2] + c[5:7] for c in TILES if c[7] == 0}
    shared = {c[:2] + c[5:7] for c in TILES if c[7] > 0}
    assert whole == shared == set(kinds)


def test_only_built_tiles_are_chosen(shape):
    kinds = built()
    for mode in MODES:
        for dtype in ("bf16", "f32"):
            for N in (17, 33, 70, 200, 1000, 5000, 40000, 2**22):
                for V in (1, 9, 100, 1000, 9000, 130000, 2**21 - 8):
                    for D in (1, 50, 300, 2000, 9000, 65536):
                        if N * V <= 2**40:
                            (columns, rows, workers), tiles, _ = shape(mode, dtype, N, V, D)
                            assert (mode, dtype, columns, rows) in kinds and workers in (0, 128, 256, 512)
                            assert workers == 0 or tiles <= 400
