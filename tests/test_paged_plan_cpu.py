"""Who computes what in the paged 8-bit attention, from the kernel's own plan
compiled for the host: every tile of every unit belongs to one CTA, CTAs beyond
the shares get nothing, and the CTAs that a split unit's parts are merged from
are those that hold tiles of it."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE = 128


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan_on_host.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                    "-I", os.path.join(ROOT, "grouped_query_decode_gb300", "csrc"), "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
                    os.path.join(ROOT, "tests", "plan_on_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    i32, i64, vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p
    lib.plan_case.argtypes = [i32] * 6 + [vp, i32, i32, vp, i32, vp]
    lib.plan_owner.argtypes = [i64, i32, i64]
    return lib


def rows_of(R):
    return 8 if R <= 8 else 16 if R <= 16 else 32


def unit_tiles(lens, sq, H, G, tmax):
    """Tiles of entry (b, row tile), from the causal rule."""
    R = H // G * sq
    RP = rows_of(R)
    tiles = []
    for T in np.clip(lens, 0, tmax):
        for rt in range(-(-R // RP)):
            last = min(R, (rt + 1) * RP) - 1
            keys = T if R <= RP else max(0, T - sq + last // (H // G) + 1)    # one row tile reads the whole cache
            tiles.append(-(-int(keys) // TILE))
    return tiles


def check(plan, lens, sq, H, G, page, most, sms=152, any_size=False):
    lens = np.ascontiguousarray(lens, dtype=np.int32)
    want = unit_tiles(lens, sq, H, G, most * page)
    cap = G * (len(want) + 1) * 2 + 2 * sms + sum(want) * G
    out, grid = np.zeros((cap, 8), np.int64), ctypes.c_int()
    n = plan.plan_case(len(lens), sq, H, G, page, most, lens.ctypes.data, sms, int(any_size), out.ctypes.data, cap,
                       ctypes.byref(grid))
    assert n >= 0, "threads disagree" if n == -1 else "more segments than units and CTAs"
    seen = {}
    for cta, entry, g, i0, i1, tiles, c0, shared in out[:n].tolist():
        assert 0 <= entry < len(want) and 0 <= g < G and 0 <= i0 < i1 <= tiles == want[entry]
        seen.setdefault((entry, g), []).append((i0, i1, cta, c0, shared))
    units = [(e, g) for e in range(len(want)) if want[e] for g in range(G)]
    assert sorted(seen) == units
    for (entry, g), parts in seen.items():
        parts.sort()
        assert [p[0] for p in parts] == [0] + [p[1] for p in parts[:-1]] and parts[-1][1] == want[entry], (entry, g, parts)
        ctas = [p[2] for p in parts]
        assert ctas == list(range(ctas[0], ctas[0] + len(ctas)))
        assert all((c0, k) == (ctas[0], len(ctas)) for *_, c0, k in parts), (entry, g, parts)


@pytest.mark.parametrize("empty", range(8))
@pytest.mark.parametrize("sq,H,G", [(1, 32, 8), (1, 16, 1), (1, 64, 2), (4, 16, 2), (9, 8, 2)], ids=str)
def test_an_empty_sequence_anywhere(plan, empty, sq, H, G):
    """Tables wider than the lengths, so that the grid has CTAs without a share."""
    lens = np.full(16, 1024)
    lens[empty] = 0
    check(plan, lens, sq, H, G, 64, 64)
    lens[[8, 9, 15]] = [0, 1, 4000]
    check(plan, lens, sq, H, G, 64, 64)


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(plan, seed):
    rng = np.random.default_rng(seed)
    G = int(rng.choice([1, 2, 3, 8]))
    H, sq = G * int(rng.choice([1, 4, 5, 8, 16, 32])), int(rng.choice([1, 1, 1, 2, 4, 11]))
    B = int(rng.choice([1, 2, 5, 16, 60, 128, 129, 200, 500]))
    top = int(rng.choice([3, 200, 1500, 9000]))
    lens = rng.integers(-2, top, B)
    lens[rng.random(B) < rng.choice([0.0, 0.3, 0.9])] = 0
    if rng.random() < 0.25:
        lens[:] = top
    page = int(rng.choice([16, 64, 256]))
    check(plan, lens, sq, H, G, page, -(-top // page) * int(rng.choice([1, 1, 3])), sms=int(rng.choice([1, 7, 20, 152])),
          any_size=rng.random() < 0.2)


def test_nothing_to_do(plan):
    check(plan, [0] * 5, 1, 8, 2, 64, 8)
    check(plan, [0] * 300, 1, 8, 2, 64, 8)


def test_owner_of_a_tile_past_32_bits(plan):
    """The CTA of a tile, ((t + 1) * ctas - 1) // total, whatever needs 64 bits:
    the product, the number of tiles, both or neither."""
    rng = np.random.default_rng(5)
    totals = [1, 7, 152, (1 << 32) - 1, 1 << 32, (1 << 32) + 1, 3 << 32, 1 << 40]
    totals += [int(x) for x in rng.integers(1 << 28, 1 << 45, 30)]
    for total in totals:
        for ctas in (1, 2, 151, 152):
            if ctas > total:
                continue
            for t in [0, 1, total // 2, total - 1, *(int(x) for x in rng.integers(0, total, 20))]:
                t = min(t, total - 1)
                assert plan.plan_owner(total, ctas, t) == ((t + 1) * ctas - 1) // total, (total, ctas, t)
