"""The recurrence's workgroups take no tile outside a pass, whatever the counter in
the workspace holds (csrc/tile_place.h, compiled for the host)."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_recurrent_sequence_shortconv_amd", "csrc")


@pytest.fixture(scope="module")
def place(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("tile_place")
    (at / "place.cpp").write_text(
        '#include "tile_place.h"\n'
        'extern "C" void place(unsigned id, int tiles, int slices, int* out) {\n'
        '  const prism::TilePlace p = prism::tile_place(id, tiles, slices);\n'
        '  out[0] = p.turn;\n  out[1] = p.slice;\n}\n')
    lib = str(at / "place.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(at / "place.cpp"), "-o", lib],
                   check=True, timeout=120)
    f = ctypes.CDLL(lib).place
    f.argtypes = [ctypes.c_uint, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int * 2)]

    def call(id, tiles, slices):
        out = (ctypes.c_int * 2)()
        f(id, tiles, slices, ctypes.byref(out))
        return out[0], out[1]
    return call


@pytest.mark.parametrize("tiles,slices", [(1, 1), (1, 7), (128, 16), (409, 3), (1 << 22, 1), (1, 1 << 22), (2047, 2048)])
def test_every_workgroup_its_own_tile(place, tiles, slices):
    n = tiles * slices
    ids = range(n) if n < 10000 else [0, 1, slices - 1, slices % n, n // 2, n - slices, n - 1]
    got = [place(i, tiles, slices) for i in ids]
    assert got == [(i // slices, i % slices) for i in ids]
    assert all(0 <= t < tiles and 0 <= s < slices for t, s in got)


@pytest.mark.parametrize("tiles,slices", [(1, 1), (128, 16), (1 << 22, 1), (1, 1 << 22), (2047, 2048)])
def test_numbers_of_no_workgroup(place, tiles, slices):
    """Past the last one, and words that are floats, negative ones among them."""
    n = tiles * slices
    for id in (n, n + 1, 0x7fffffff, 0x80000000, 0x80000001, 0xbf800000, 0xffffffff, 0xffffffff - slices):
        assert place(id, tiles, slices)[0] == -1
