"""How paged decode cuts its work, in the library's own arithmetic
(csrc/paged_runs.cuh compiled for the host): the runs of a call's tiles and the
ranges of its shared rows, up to the largest totals that a call may have."""
import bisect
import ctypes
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
TILE = 64  # rows

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("runs") / "libruns.so")
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-o", so,
                          os.path.join(HERE, "c", "paged_runs.cc")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    lib = ctypes.CDLL(so)
    i = ctypes.c_int
    lib.runs_of_call.argtypes = [i, ctypes.c_longlong, i, i, ctypes.c_void_p]
    for f in (lib.runs_begin, lib.runs_at, lib.runs_place):
        f.argtypes = [i, ctypes.c_longlong, i, i, i]
    return lib


class Runs:
    def __init__(self, lib, total, units, grid, claim):
        got = (ctypes.c_int * 2)()
        lib.runs_of_call(total, units, grid, claim, got)
        self.runs, self.waves = got
        args = (total, units, grid, claim)
        self.of = lambda x: lib.runs_at(*args, x)
        self.place = lambda j: lib.runs_place(*args, j)
        self.begin = [lib.runs_begin(*args, c) for c in range(self.runs + 1)]


def _check(r, total, units, grid, claim, rng):
    assert r.waves in (1, 3) and (r.waves == 1 or claim) and r.runs <= r.waves * grid
    assert r.begin[0] == 0 and r.begin[-1] == total
    # a run is worth three tiles at least: one behind a unit's cost of two
    assert min(b - a for a, b in zip(r.begin, r.begin[1:])) >= 3
    assert sorted(r.place(j) for j in range(r.runs)) == list(range(r.runs))
    if r.waves == 1:
        assert r.begin == [c * total // r.runs for c in range(r.runs + 1)]
    else:  # the long run of every stretch first, then all second ones, then all third ones
        assert [r.place(j) for j in range(grid)] == [3 * g for g in range(grid)]
        # a stretch's runs begin at 0, 208 and 240 of its 256 parts, in whole numbers of any size
        step = total // grid * 256 + total % grid * 256 // grid  # of a part, in 65536ths
        assert r.begin[:-1] == [(g * 256 + w) * step >> 16 for g in range(grid) for w in (0, 208, 240)]
    probe = {0, total - 1, *(x for b in rng.sample(r.begin, min(40, len(r.begin))) for x in (b - 1, b, b + 1)),
             *(rng.randrange(total) for _ in range(40))}
    for x in probe:
        if 0 <= x < total:
            assert r.of(x) == bisect.bisect_right(r.begin, x) - 1, x


@pytest.mark.parametrize("claim", [0, 1])
def test_runs_cover_every_total_once(lib, claim):
    rng = random.Random(2)
    for _ in range(150):
        grid, units = rng.choice([1, 5, 148, 296, 320]), rng.choice([1, 2, 40, 512, 2000, 100000])
        low = 3 * units
        total = min((1 << 31) - 1, low + int(2 ** rng.uniform(0, 31)))
        _check(Runs(lib, total, units, grid, claim), total, units, grid, claim, rng)


@pytest.mark.parametrize("claim", [0, 1])
@pytest.mark.parametrize("grid", [1, 2, 295, 296, 320])
def test_largest_totals(lib, grid, claim):
    """The largest totals that a call may have: 2^31 - 1 and what lies below, where 32 bits are full."""
    rng = random.Random(grid)
    for total in ((1 << 31) - 1, (1 << 31) - 2, (1 << 31) - 127, (1 << 30) + 1, 3 * (1 << 29) + 7):
        for units in (1, grid, 127, 1 << 20):
            _check(Runs(lib, total, units, grid, claim), total, units, grid, claim, rng)


@pytest.mark.parametrize("claim", [0, 1])
def test_every_tile_is_in_one_run_of_the_library(lib, claim):
    """The walk that paged_kernel makes over its runs, on the library's runs:
    every tile once, every part in one slot, every cut's parts those of its runs."""
    rng, cost2 = random.Random(7), lib.unit_cost()
    for _ in range(60):
        B, Hkv = rng.choice([1, 2, 3, 7, 64, 129]), rng.choice([1, 2, 3, 8])
        most = rng.choice([1, 64, 65, 300, 5000, 40000])
        tiles = [max(1, -(-rng.choice([0, 1, most, rng.randint(0, most)]) // TILE)) for _ in range(B)]
        unit = [t for t in tiles for _ in range(Hkv)]
        front = [0]
        for t in unit:
            front.append(front[-1] + t + cost2)
        total, grid = front[-1], rng.choice([296, 5])
        r = Runs(lib, total, B * Hkv, grid, claim)
        seen, slots, cuts = [0] * len(unit), {}, []
        for c in range(r.runs):
            t0, t1 = r.begin[c], r.begin[c + 1]
            u = bisect.bisect_right(front, t0) - 1
            off = t0 - front[u]
            tile, left = max(0, off - cost2), t1 - t0 - max(0, cost2 - off)
            assert left > 0
            while left > 0:
                n = min(unit[u] - tile, left)
                assert seen[u] == tile  # in order, none twice, none left out
                seen[u] += n
                begins, ends = tile == 0, tile + n == unit[u]
                if not (begins and ends):
                    assert slots.setdefault(2 * c + begins, u) == u
                if begins and not ends:
                    cuts.append((u, c, r.of(t1 + unit[u] - tile - n - 1)))
                left -= n + cost2
                tile, u = 0, u + 1
        assert seen == unit
        parts = {}
        for u, first, last in cuts:
            assert first < last < r.runs
            parts.update({s: u for s in [2 * first + 1] + [2 * c for c in range(first + 1, last + 1)]})
        assert parts == slots


def test_ranges_of_shared_rows(lib):
    """Each tile lies in the range that says so, no range is empty, none longer than the mean rounded up."""
    for tiles in list(range(1, 70)) + [1000, 1 << 23]:
        for n in sorted({1, 2, 3, 7, min(lib.max_ranges(), tiles)}):
            if n > tiles:
                continue
            at = [lib.begin_of_range(s, tiles, n) for s in range(n + 1)]
            assert at[0] == 0 and at[-1] == tiles and all(0 < b - a <= -(-tiles // n) for a, b in zip(at, at[1:]))
            for t in range(tiles) if tiles < 2000 else (0, 1, at[1] - 1, at[-2], tiles - 1):
                s = lib.range_of_tile(t, tiles, n)
                assert at[s] <= t < at[s + 1]
