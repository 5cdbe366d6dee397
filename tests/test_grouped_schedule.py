"""How an expert's rows are dealt to row tiles (csrc/schedule.h), compiled for
the CPU: every count of rows below 2^31 gives tiles that cover the rows once."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "group_limited_routing_router_amd", "csrc")
TOP = (1 << 31) - 1


@pytest.fixture(scope="module")
def schedule(tmp_path_factory):
    d = tmp_path_factory.mktemp("schedule")
    src, lib = d / "schedule.cpp", d / "schedule.so"
    src.write_text('#include "schedule.h"\n'
                   'extern "C" int row_tiles_of(int n, int bm) { return moe::row_tiles_of(n, bm); }\n'
                   'extern "C" int rows_per_tile(int n, int tiles, int gran) {\n'
                   '    return moe::rows_per_tile(n, tiles, gran);\n}\n')
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-shared", "-fPIC", "-I", CSRC, "-o", str(lib), str(src)],
                   check=True)
    return ctypes.CDLL(str(lib))


@pytest.mark.parametrize("bm,gran", [(32, 1), (64, 1), (128, 64), (256, 64), (256, 128)])
def test_rows_of_tiles(schedule, bm, gran):
    counts = set(range(0, 3 * bm + 2))
    for near in (1 << 20, 1 << 30, 2_130_000_000, 2_140_000_000, TOP - 40000, TOP):
        counts |= {n for n in range(near - 300, near + 301) if n <= TOP}
    for n in sorted(counts):
        tiles = schedule.row_tiles_of(n, bm)
        assert tiles == -(-n // bm), (n, tiles)
        if tiles == 0:
            continue
        per = schedule.rows_per_tile(n, tiles, gran)
        share = -(-n // tiles)
        assert per == -(-share // gran) * gran and per <= bm, (n, tiles, per)
        last = n - (tiles - 1) * per
        assert (1 <= last <= per) if gran > 1 else last <= per, (n, tiles, per)


def test_no_rows(schedule):
    assert schedule.row_tiles_of(0, 128) == 0 and schedule.row_tiles_of(-5, 128) == 0


def test_stages_of_the_weight_gradient(schedule):
    """Its stages are 32 positions: the count holds up to the last position."""
    for n in (1, 31, 32, 33, TOP - 31, TOP - 30, TOP):
        assert schedule.row_tiles_of(n, 32) == (n + 31) // 32
    src = open(os.path.join(CSRC, "gemm_wgrad.h")).read()
    assert "c.nk = row_tiles_of(c.red, SR);" in src
