"""The rule that picks the tile of an MXFP4 product (csrc/mx_tiles.h), compiled for the host: what its comment names is what it
picks."""
import ctypes as C
import os
import subprocess

import pytest

from test_gpu_mxfp4_tiles import SIZES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_tile_interleaved_rans_amd", "csrc")
CUS = 256


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    """(M, N, K) -> (rows, columns, K groups) of the tile."""
    d = tmp_path_factory.mktemp("mx_tiles")
    (d / "rule.cpp").write_text("""#include "mx_tiles.h"
extern "C" int count() { return ep::kMxTileCount; }
extern "C" void tile(long M, long N, long K, long cus, int* t) {
    const ep::MxTile& p = ep::kMxTiles[ep::mx_tile(M, N, K, cus)];
    t[0] = p.bm, t[1] = p.bn, t[2] = p.ks;
}
""")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(d / "rule.cpp"), "-o", str(d / "rule.so")],
                   check=True)
    rule = C.CDLL(str(d / "rule.so"))
    rule.tile.argtypes = [C.c_long] * 4 + [C.POINTER(C.c_int)]

    def pick(M, N, K):
        t = (C.c_int * 3)()
        rule.tile(M, N, K, CUS, t)
        return tuple(t)

    pick.count = rule.count()
    return pick


@pytest.mark.parametrize("M,N,K,want", [
    (4096, 8192, 8192, (256, 256, 1)), (1024, 11520, 3840, (256, 192, 1)), (512, 8192, 8192, (128, 128, 1)), (333, 5003, 3968, (128, 64, 1)),
    (256, 4096, 4096, (64, 64, 1)), (64, 4096, 4096, (32, 32, 2)), (64, 8192, 8192, (64, 64, 1)),
    (27, 12148, 10112, (64, 64, 1)), (1, 11520, 3840, (16, 32, 2)), (1, 4096, 16384, (16, 32, 4))])
def test_named_examples(tile, M, N, K, want):
    assert tile(M, N, K) == want


@pytest.mark.parametrize("M,N,K,want", [
    (16, 8192, 8192, (16, 32, 2)), (16, 4096, 16384, (16, 32, 4)), (24, 4096, 16384, (16, 32, 4)), (16, 3840, 10240, (16, 32, 4)),
    (24, 3840, 10240, (16, 32, 4)), (24, 8192, 8192, (32, 32, 2)), (64, 4096, 16384, (32, 32, 2)), (1024, 8192, 8192, (256, 128, 1))])
def test_fastest_measured(tile, M, N, K, want):
    """Products of the fit whose picked tile is the fastest of the nine that there are."""
    assert tile(M, N, K) == want


def test_sizes_reach_every_tile(tile):
    """The sizes of the GPU test take the tiles they stand for, leave none out, end inside a tile in both directions and turn its
    ring (four stages at most) more than once."""
    for want, M, N, K in SIZES:
        assert tile(M, N, K) == want, (M, N, K)
        assert M % want[0] and N % want[1] and K % 256 == 128 and -(-K // (256 * want[2])) > 4
    assert len({s[0] for s in SIZES}) == tile.count
