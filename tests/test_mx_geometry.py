"""Launch geometry of the MX products (csrc/mx_geometry.h, the header the
library compiles): shares of a split tile and the tiles of the CTA-pair
kernel, over every split and every token count that matters."""
import ctypes
import os
import subprocess

import pytest

from mx_cases import PAIRS, SPLIT

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def geo(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("mx_geo") / "libmx_geo.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                    f"-I{os.path.join(ROOT, 'quantized_matmul_q4_gb300', 'csrc')}",
                    os.path.join(ROOT, "tests", "mx_geometry_shim.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def test_rows_of_a_split_tile(geo):
    for S in range(1, 9):
        first = [geo.mx_geo_first_row(s, S) for s in range(S + 1)]
        assert first[0] == 0 and first[S] == 128
        assert all(b > a and (b - a) % 4 == 0 for a, b in zip(first, first[1:]))


def test_split_gives_every_cta_work(geo):
    for sms in (1, 132, 148, 152):
        for tiles in (1, 2, 3, 32, 54, 86, 151, 152, 153, 400, 100000):
            for stages in (1, 2, 3, 4, 5, 16, 17, 43, 86, 256, 512):
                for tokens in (1, 16, 64, 128):
                    for bits in (4, 8):
                        S = geo.mx_geo_split(tiles, 1, tokens, stages, bits, sms)
                        assert 1 <= S <= 8 and S <= max(1, stages // 2)
    # One token through 4096 x 4096: all eight; many tiles: none.
    assert geo.mx_geo_split(32, 1, 1, 32, 8, 152) == 8
    assert geo.mx_geo_split(100000, 1, 128, 32, 8, 152) == 1


def test_pairs_take_the_large_products(geo):
    for bits in (4, 8):
        stages = 4096 * bits // 1024
        for T in range(1, 17):
            assert not geo.mx_geo_use_pairs(T, 11008, stages, bits, 152)
        assert geo.mx_geo_use_pairs(8192, 11008, stages, bits, 152)
        # The split form's grid has its token tiles in y: never 65536 of them.
        for T in (128 * 65535 + 1, 2 ** 31 - 1):
            for N in (1, 129, 11008):
                assert geo.mx_geo_use_pairs(T, N, 1, bits, 152)


def test_pair_tiles(geo):
    for N, stages, bits, sms in ((11008, 16, 4, 152), (4096, 32, 8, 152), (129, 1, 4, 152), (1, 512, 8, 1)):
        for T in list(range(1, 1200)) + [4095, 4096, 4097, 8191, 8192, 100000, 0x7FFFFE00]:
            out = (ctypes.c_int * 4)()
            geo.mx_geo_pairs(T, N, stages, bits, sms, out)
            tok, tok_tiles, row_tiles, x_tiles = out
            assert tok % 32 == 0 and 32 <= tok <= 256 and row_tiles == -(-N // 256)
            assert (tok_tiles - 1) * tok < T <= tok_tiles * tok     # every tile has a token, every token a tile
            starts = {(i * tok) % 128 for i in range(min(tok_tiles, 8))}
            assert all((s + tok + 127) // 128 <= x_tiles <= 3 for s in starts)
            # Blocks of 32 tokens that a tile's scales are shifted by: with a
            # shift eight columns are taken from three scale tiles, twelve words.
            assert all(s // 32 + tok // 32 <= 12 for s in starts)
            # Tiles with two blocks of K a stage have room for two scale tiles.
            assert tok > 128 or x_tiles <= 2


def test_the_product_tests_reach_every_form(geo):
    def stages(K, bits):
        return -(-(-(-K // 128) * 128) // (256 if bits == 4 else 128))

    for bits in (4, 8):
        tiles, splits = set(), set()
        for T, K, N in PAIRS:
            assert geo.mx_geo_use_pairs(T, N, stages(K, bits), bits, 152)
            out = (ctypes.c_int * 4)()
            geo.mx_geo_pairs(T, N, stages(K, bits), bits, 152, out)
            tiles.add(out[0])
        for T, K, N in SPLIT:
            assert not geo.mx_geo_use_pairs(T, N, stages(K, bits), bits, 152)
            splits.add(geo.mx_geo_split(-(-N // 128), -(-T // 128), T, stages(K, bits), bits, 152))
        assert {64, 96, 128, 160, 192, 224, 256} <= tiles
        assert {1, 3, 4, 8} <= splits and splits & {5, 6, 7}
