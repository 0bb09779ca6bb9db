"""The line on which a packed batch's units lie, with the plan's own numbers for both
head sizes: parts have the least tiles that the plan states, and what a CTA takes of
the line is its share, up to what cutting at whole tiles moves."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIELDS = ("cta", "seq", "g", "row0", "a", "b", "pos0", "pos_last", "key0", "j0", "tiles_a", "tiles_b", "slot", "first",
          "parts", "counter", "valid")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("line") / "ragged_line.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "grouped_query_decode_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "ragged_line_on_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.ragged_parts.restype = ctypes.c_longlong
    lib.ragged_parts.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int] * 5 + [ctypes.c_void_p, ctypes.c_longlong]
    lib.ragged_line.argtypes = [ctypes.c_int] * 6 + [ctypes.c_void_p]
    lib.ragged_ctas.argtypes = [ctypes.c_longlong, ctypes.c_int]
    return lib


def line(lib, n, T, tq, G, D, pr):
    out = np.zeros(7, dtype=np.int64)
    lib.ragged_line(n, T, tq, G, D, pr, out.ctypes.data)
    return dict(zip(("start", "length", "head", "part", "share", "eighths", "pad"), (int(v) for v in out)))


def check(lib, seqs, heads, G, D, grid=152):
    tq = 128 // heads
    n, T = (np.array([s[i] for s in seqs], dtype=np.int32) for i in (0, 1))
    start = (np.cumsum(n) - n).astype(np.int32)
    most = int(sum(-(-int(x) // (2 * tq)) for x in n)) * G + 2 * grid + 10
    out = np.zeros((most, 17), dtype=np.int32)
    got = lib.ragged_parts(*(x.ctypes.data for x in (start, n, T)), len(seqs), tq, G, D, grid, out.ctypes.data, most)
    assert got >= 0
    total = sum(line(lib, a, b, tq, G, D, 0)["head"] for a, b in seqs if a) * G
    ctas = lib.ragged_ctas(total, grid)
    load, longest = np.zeros(grid), 0
    for row in out[:got]:
        u = dict(zip(FIELDS, (int(v) for v in row)))
        s = seqs[u["seq"]]
        at = line(lib, *s, tq, G, D, (u["row0"] - int(start[u["seq"]])) // (2 * tq))
        tiles, end = max(u["tiles_a"], u["tiles_b"]), u["j0"] + max(u["tiles_a"], u["tiles_b"])
        whole = 0 if u["pos_last"] < 0 else u["pos_last"] // 128 + 1
        if u["parts"] > 1:
            assert tiles >= at["part"], u
        key = at["eighths"] / 8 if u["b"] == 0 else 1.0
        load[u["cta"]] += (at["length"] if end == whole else end * 128 * key) - u["j0"] * 128 * key
        longest = max(longest, at["length"])
    assert abs(load.sum() - total) < 1e-6 * total + 1e-3
    # A share's two ends move by the least part at most, and the later one by the unit's
    # pad and its last tile's fraction too; keys of single row tiles are counted by 410 / 256 for 8 / 5.
    p = line(lib, 1, 1, tq, G, D, 0)
    slack = 2 * p["part"] * 128 + p["pad"] + 128 + (longest * 0.002 if p["eighths"] == 5 else 0)
    assert load.max() <= total / ctas + 1 + slack, (load.max(), total / ctas, slack)
    assert (load[ctas:] == 0).all()
    return load[:ctas], total / ctas


@pytest.mark.parametrize("D", [64, 128])
def test_least_part_and_share(lib, D):
    p = line(lib, 1, 1, 32, 8, D, 0)
    assert p["part"] == 4 and p["share"] == 512 and lib.ragged_ctas(512 * 9 + 511, 152) == 9
    assert lib.ragged_ctas(1, 152) == 1 and lib.ragged_ctas(1 << 40, 152) == 152


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [1, 3, 4, 8, 32, 128])
@pytest.mark.parametrize("G", [1, 2, 8])
def test_shares(lib, heads, G, D):
    rng = np.random.default_rng(heads * 100 + G * 10 + D)
    for _ in range(4):
        B = int(rng.integers(1, 40))
        T = np.exp(rng.uniform(0, np.log(6000), B)).astype(int)
        n = np.where(rng.random(B) < 0.4, 1, np.minimum(T, np.exp(rng.uniform(0, np.log(1500), B)).astype(int)))
        n = np.where(rng.random(B) < 0.1, 0, n)
        n[0] = max(n[0], 1)
        check(lib, list(zip(n.tolist(), T.tolist())), heads, G, D, grid=int(rng.choice([152, 7, 1])))
        check(lib, [(int(x), int(x)) for x in T], heads, G, D)


@pytest.mark.parametrize("D", [64, 128])
def test_long_batches_are_shared_out_evenly(lib, D):
    for seqs, heads, G in (([(1, 5000)] * 64, 4, 8), ([(3000, 3000)], 4, 8), ([(1, 100000)], 8, 8),
                           ([(100, 8000), (1, 300)] * 20, 4, 4), ([(1, (1 << 31) - 200)] * 3, 4, 2)):
        load, share = check(lib, seqs, heads, G, D)
        assert (load > 0).sum() >= 140
