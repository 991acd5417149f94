"""The choice of tiles for products of 8-bit integers, compiled for the host: which cases of the GPU tests
take which of them."""
import os
import subprocess

import int8_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def chosen(tmp_path, asked):
    exe = str(tmp_path / "int8_tiles")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "combine_moe_layout_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "int8_tiles.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], input="\n".join("%d %d %d %d" % a for a in asked), capture_output=True, text=True,
                       timeout=60, check=True)
    return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]


def test_cases_take_the_tiles_they_are_for(tmp_path):
    for glu in (0, 1):
        got = chosen(tmp_path, [(1, T, N >> glu, glu) for T, _, N, _, _ in cases.LINEAR])
        assert got == [(0, h, 256) for *_, h, _ in cases.LINEAR]
        got = chosen(tmp_path, [(E, T * k, N >> glu, glu) for T, k, E, _, _, N, _ in cases.EXPERTS])
        assert got == [(0, h, 256) for *_, h in cases.EXPERTS]
    blocks = [cases.row_blocks(T, h) for T, _, _, h, _ in cases.LINEAR]
    assert blocks == [b for *_, b in cases.LINEAR]
    assert set.union(*blocks) == set(range(1, 9))
    # stages of 128 channels: with and without a part at the end, an even and an odd number of whole ones
    whole = {(K // 128 % 2, K % 128 > 0) for _, K, *_ in cases.LINEAR}
    assert whole >= {(0, True), (1, False), (1, True), (0, False)}


def test_every_kind_of_tile_is_chosen(tmp_path):
    asked = [(1, T, N, glu) for T in (1, 16, 17, 32, 33, 100, 200, 256, 300, 512, 640, 1000, 1200, 2300, 4000)
             for N in (64, 4096, 8192) for glu in (0, 1)] + [(256, T, 512, 1) for T in (1024, 8192, 65536)]
    got = set(chosen(tmp_path, asked))
    assert {t for t in got if not t[0]} == {(0, 64, 128), (0, 128, 128), (0, 128, 256), (0, 192, 256), (0, 256, 256)}
    assert {t[1:] for t in got if t[0]} >= {(16, 16), (16, 32), (32, 16), (32, 32), (64, 16), (64, 32), (64, 64)}
