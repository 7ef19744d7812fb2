"""How far the copies of an adapter's A reach, on the CPU.

Where A[g] is stored inputs x outputs, the tiles that take x . A[g] copy its rows in chunks of 16 bytes
for every whole K tile but the last (which K or the rank's end cuts: it goes through registers, element by element).
A chunk that the rank cuts brings what lies behind it, so the matrix has to go on for that long.
csrc/narrow.hpp says how many of the rows those copies and that last tile take; it is compiled here as it is.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tile_scheduled_dense_amd", "csrc")
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


@pytest.fixture(scope="module")
def ring_rows(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    at = tmp_path_factory.mktemp("narrow")
    (at / "narrow.cpp").write_text('#include "narrow.hpp"\nextern "C" int ring_rows(int K, int width, int tile_k, int chunk) '
                                   "{ return tg::ring_rows(K, width, tile_k, chunk); }\n")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(at / "narrow.cpp"), "-o",
                    str(at / "narrow.so")], check=True)
    return ctypes.CDLL(str(at / "narrow.so")).ring_rows


def reach(rows, rank, dt):
    """One past the last element that the ring's copies bring of `rows` rows of `rank` elements."""
    chunk, tile_k = 16 // BYTES[dt], 64 // BYTES[dt]
    tiles = -(-rows // tile_k)
    copied = tiles if rows % tile_k == 0 and rank % chunk == 0 else tiles - 1
    return (copied * tile_k - 1) * rank + -(-rank // chunk) * chunk if copied > 0 else 0


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_copies_of_an_adapters_rows_end_inside_it(ring_rows, dt):
    chunk, tile_k = 16 // BYTES[dt], 64 // BYTES[dt]
    for rank in range(1, 140):
        for K in [*range(0, 200), 1024, 1025, 1030, 6200, 6241]:
            taken = ring_rows(K, rank, tile_k, chunk)
            assert reach(taken, rank, dt) <= K * rank, (rank, K)
            # what is left is one tile, and only a narrow rank leaves any
            assert 0 <= K - taken < tile_k
            assert taken == K or rank < 4


def test_the_ring_alone_would_pass_the_end():
    """The ranks and remainders of K that the rule is for."""
    past = {dt: {(rank, K % (64 // BYTES[dt])) for rank in range(1, 9) for K in range(40, 140) if reach(K, rank, dt) > K * rank}
            for dt in BYTES}
    assert past["bf16"] == past["f16"] == {(1, n) for n in range(1, 7)} | {(2, 1), (2, 2), (3, 1)}
    assert past["f32"] == {(1, 1), (1, 2)}
