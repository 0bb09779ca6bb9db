"""Who computes what in the attention of packed batches, from the kernel's own
plan compiled for the host: every key tile that a row tile sees belongs to one
part, parts of a unit have slots and CTAs that the merge finds, and shares are
about equal."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIELDS = ("cta", "seq", "g", "row0", "a", "b", "pos0", "pos_last", "key0", "j0", "tiles_a", "tiles_b", "slot", "first",
          "parts", "counter", "valid")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "ragged_plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "grouped_query_decode_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "ragged_plan_on_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.ragged_parts.restype = ctypes.c_longlong
    lib.ragged_parts.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int] * 5 + [ctypes.c_void_p, ctypes.c_longlong]
    return lib


def parts_of(plan, seqs, heads, G, grid=152, D=128):
    n, T = (np.array([s[i] for s in seqs], dtype=np.int32) for i in (0, 1))
    start = (np.cumsum(n) - n).astype(np.int32)
    tq = 128 // heads
    most = int(sum(-(-int(x) // (2 * tq)) for x in n)) * G + 2 * grid + 10
    out = np.zeros((most, 17), dtype=np.int32)
    got = plan.ragged_parts(*(x.ctypes.data for x in (start, n, T)), len(seqs), tq, G, D, grid, out.ctypes.data, most)
    assert got >= 0, got
    return [dict(zip(FIELDS, (int(v) for v in row))) for row in out[:got]], start, tq


def check(plan, seqs, heads, G, grid=152):
    """Both head sizes; the load with D 128."""
    one(plan, seqs, heads, G, grid, 64)
    return one(plan, seqs, heads, G, grid, 128)


def one(plan, seqs, heads, G, grid, D):
    parts, start, tq = parts_of(plan, seqs, heads, G, grid, D)
    units = {}
    for u in parts:
        assert u["valid"] == 1
        units.setdefault((u["seq"], u["g"], u["row0"]), []).append(u)
    load = np.zeros(grid)
    for b, (n, T) in enumerate(seqs):
        for g in range(G):
            for pr in range(-(-n // (2 * tq))):
                row0 = int(start[b]) + pr * 2 * tq
                got = units.pop((b, g, row0))
                left = n - pr * 2 * tq
                tokens = [min(left, tq), min(max(left - tq, 0), tq)]
                pos0 = T - n + pr * 2 * tq
                see = [max(0, pos0 + sum(tokens[:x + 1])) if tokens[x] else 0 for x in (0, 1)]      # keys of the last row
                want = [-(-s // 128) for s in see]
                slots = []
                at = 0
                for k, u in enumerate(got):
                    assert (u["a"], u["b"]) == tuple(tokens) and u["pos0"] == pos0 and u["key0"] == start[b]
                    assert u["pos_last"] == pos0 + sum(tokens) - 1
                    assert u["j0"] == at and u["cta"] == got[0]["cta"] + k
                    at += max(u["tiles_a"], u["tiles_b"])
                    assert u["tiles_a"] == max(0, min(want[0], at) - u["j0"])
                    assert u["tiles_b"] == max(0, min(want[1], at) - u["j0"])
                    load[u["cta"]] += max(u["tiles_a"], u["tiles_b"]) * (128 if tokens[1] else 80) + 256
                    assert u["parts"] == len(got) and u["first"] == got[0]["cta"]
                    if len(got) == 1:
                        assert u["slot"] == -1
                    else:
                        assert max(u["tiles_a"], u["tiles_b"]) >= 2
                        # where the merge looks for it
                        assert u["slot"] == (u["counter"] if k == 0 else 2 * u["cta"]) and u["slot"] // 2 == u["cta"]
                    slots.append(u["slot"])
                assert at == max(want) and len({u["counter"] for u in got}) == 1
    assert not units
    used = [u["slot"] for u in parts if u["slot"] >= 0]
    counters = [u["counter"] for u in parts if u["slot"] >= 0 and u["first"] == u["cta"]]
    assert len(set(used)) == len(used) and len(set(counters)) == len(counters)
    return load


@pytest.mark.parametrize("heads", [1, 3, 4, 8, 32, 128])
@pytest.mark.parametrize("G", [1, 2, 8])
def test_batches(plan, heads, G):
    rng = np.random.default_rng(heads * 10 + G)
    check(plan, [(1, 1)], heads, G)
    check(plan, [(0, 0), (0, 100)], heads, G)
    check(plan, [(1, 100000)], heads, G)
    check(plan, [(5, 3), (4, 0), (1, 0), (2, 2)], heads, G)
    for _ in range(12):
        B = int(rng.integers(1, 40))
        T = np.exp(rng.uniform(0, np.log(6000), B)).astype(int)
        n = np.where(rng.random(B) < 0.4, 1, np.minimum(T, np.exp(rng.uniform(0, np.log(1500), B)).astype(int)))
        n = np.where(rng.random(B) < 0.1, 0, n)
        check(plan, list(zip(n.tolist(), T.tolist())), heads, G, grid=int(rng.choice([152, 7, 1])))
        check(plan, [(int(x), int(x)) for x in T], heads, G)


def test_shares_are_about_equal(plan):
    for seqs, heads, G in (([(1, 5000)] * 64, 4, 8), ([(3000, 3000)], 4, 8), ([(1, 100000)], 8, 8),
                           ([(100, 8000), (1, 300)] * 20, 4, 4)):
        load = check(plan, seqs, heads, G)
        assert (load > 0).sum() >= 140 and load.max() <= 1.3 * load.mean() + 512


def test_largest_sizes(plan):
    """Lengths near 2^31 and positions far along the line."""
    check(plan, [(1, (1 << 31) - 200)], 4, 2)
    check(plan, [(1, (1 << 31) - 200)] * 50, 1, 16)
