"""Page management on the GPU, equal to the model's in every integer and byte."""
import numpy as np
import pytest
import torch

import grouped_query_decode_gb300 as gq
import paged_fp8_model as model

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class State:
    """Rows with pages as a serving loop leaves them, some of them shared."""

    def __init__(self, seed, B, most, ps, num, share=True, reserved=True):
        self.rng = rng = np.random.default_rng(seed)
        self.ps, self.num = ps, num
        self.table = np.full((B, most), -1, np.int32)
        self.refs = np.zeros(num, np.int32)
        self.lens = np.zeros(B, np.int32)
        ids = list(rng.permutation(num))
        for b in range(B):
            if share and b and rng.random() < 0.4:
                s = rng.integers(0, b)
                full = int(self.lens[s]) // ps
                self.table[b, :full] = self.table[s, :full]
                self.lens[b] = full * ps + (rng.integers(0, ps) if full < most else 0)
            else:
                full = 0
                self.lens[b] = rng.integers(0, most * ps + 1)
            for j in range(full, -(-int(self.lens[b]) // ps)):
                if not ids:
                    self.lens[b] = j * ps
                    break
                self.table[b, j] = ids.pop()
            n = -(-int(self.lens[b]) // ps)
            if reserved and n < most and ids and rng.random() < 0.3:
                self.table[b, n] = ids.pop()
            for e in self.table[b]:
                if e >= 0:
                    self.refs[e] += 1

    def pools(self, kinds=("codes", "scale", "odd")):
        shapes = {"codes": ((3, self.num, 2, self.ps, 64), np.uint8), "scale": ((2, self.num, 2, 1), np.float32),
                  "odd": ((1, self.num, 37), np.uint8), "bf16": ((2, self.num, 1, self.ps, 64), np.int16),
                  "big": ((1, self.num, 9001), np.uint8)}
        out = []
        for k in kinds:
            shape, t = shapes[k]
            x = self.rng.integers(0, 120, shape)
            out.append(x.astype(t))
        return out


def moved(pools, pairs):
    out = [x.copy() for x in pools]
    for x, was in zip(out, pools):
        for a, b in pairs:
            x[:, b] = was[:, a]
    return out


SIZES = [(1, 1, 16, 4), (6, 5, 16, 64), (33, 9, 32, 500), (64, 40, 16, 3000), (300, 3, 128, 1200), (5, 2100, 16, 9000)]


@pytest.mark.parametrize("B,most,ps,num", SIZES, ids=str)
@pytest.mark.parametrize("seed", range(3))
def test_reserve(seed, B, most, ps, num):
    s = State(seed, B, most, ps, num, reserved=False)
    lens = np.minimum(s.lens + s.rng.integers(0, 3 * ps, B), most * ps).astype(np.int32)
    if seed == 2:
        lens[:] = most * ps + 5        # clamped; more than there is
    want = model.reserve(s.table, lens, s.refs, ps)
    t, r, c = dev(s.table), dev(s.refs), torch.zeros(2, dtype=torch.int32, device="cuda")
    gq.gqa_pages_reserve(t, dev(lens), r, ps, c)
    assert c.tolist() == want[2]
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(r.cpu().numpy(), want[1])


def test_reserve_for_the_longest_sequences():
    """715827 pages of 3000 tokens: the last page ends past 2^31 tokens."""
    most, ps, num = 715827, 3000, 50
    t = torch.full((1, most), -1, dtype=torch.int32, device="cuda")
    r, c = torch.zeros(num, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    gq.gqa_pages_reserve(t, dev(np.array([2 ** 31 - 1], np.int32)), r, ps, c)
    assert c.tolist() == [most, num] and bool((t == -1).all()) and not bool(r.any())


@pytest.mark.parametrize("B,most,ps,num", SIZES, ids=str)
@pytest.mark.parametrize("seed", range(4))
def test_fork(seed, B, most, ps, num):
    s = State(10 + seed, B, most, ps, num)
    src = s.rng.integers(-1, B + (seed == 1), B).astype(np.int32)
    if seed == 2:
        src[:] = src[0] if B > 1 else 0         # every row goes on from one
    if seed == 3:
        src = s.rng.permutation(B).astype(np.int32)
    pools = s.pools()
    want_t, want_l, want_r, counts, pairs = model.fork(src, s.table, s.lens, s.refs, ps)
    d = [dev(x) for x in pools]
    t, l, r = dev(s.table), dev(s.lens), dev(s.refs)
    outs = [torch.full_like(x, -77) for x in (t, l, r)]
    c = torch.zeros(2, dtype=torch.int32, device="cuda")
    for rep in range(2):                        # the inputs stay: a second call does the same
        gq.gqa_pages_fork(d, dev(src), t, l, r, ps, *outs, c, page_dim=1)
        assert c.tolist() == counts
        for got, want in zip(outs, (want_t, want_l, want_r)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(t.cpu().numpy(), s.table) and np.array_equal(r.cpu().numpy(), s.refs)
        for got, want in zip(d, moved(pools, pairs)):
            assert np.array_equal(got.cpu().numpy(), want)


def test_fork_without_enough_free_pages_changes_nothing():
    ps, num = 16, 9
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7]], np.int32)
    lens, refs = np.array([20, 20, 20, 20], np.int32), np.array([1] * 8 + [0], np.int32)
    src = np.array([0, 0, 0, 1], np.int32)
    t, l, r = dev(table), dev(lens), dev(refs)
    outs = [torch.zeros_like(x) for x in (t, l, r)]
    c = torch.zeros(2, dtype=torch.int32, device="cuda")
    pool = torch.arange(num, device="cuda").view(num, 1).float()
    gq.gqa_pages_fork([pool], dev(src), t, l, r, ps, *outs, c)
    assert c.tolist() == [2, 1]
    for got, was in zip(outs, (table, lens, refs)):
        assert np.array_equal(got.cpu().numpy(), was)
    assert pool.flatten().tolist() == list(range(num))


@pytest.mark.parametrize("B,most,ps,num", SIZES, ids=str)
def test_free(B, most, ps, num):
    s = State(30, B, most, ps, num)
    done = s.rng.random(B) < 0.5
    want = model.free(done, s.table, s.lens, s.refs)
    for mask in (dev(done), dev(done.astype(np.uint8) * 7)):
        t, l, r = dev(s.table), dev(s.lens), dev(s.refs)
        for rep in range(2):                    # an empty row stays empty
            gq.gqa_pages_free(mask, t, l, r)
            for got, w in zip((t, l, r), want):
                assert np.array_equal(got.cpu().numpy(), w)


def test_free_does_not_take_counts_below_zero():
    t, l = dev(np.array([[0, 1], [0, 1]], np.int32)), dev(np.array([20, 20], np.int32))
    r = dev(np.array([1, 2, 5], np.int32))
    gq.gqa_pages_free(dev(np.array([True, True])), t, l, r)
    assert r.tolist() == [0, 0, 5] and t.flatten().tolist() == [-1] * 4 and l.tolist() == [0, 0]


@pytest.mark.parametrize("B,most,ps,num", SIZES, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(in_place, B, most, ps, num):
    s = State(40, B, most, ps, num)
    pools = s.pools(("codes", "odd", "bf16") if num < 5000 else ("scale", "odd"))
    want_t, want_r, counts, pairs = model.compact(s.table, s.refs)
    d, t, r = [dev(x) for x in pools], dev(s.table), dev(s.refs)
    t2, r2 = (t, r) if in_place else (torch.full_like(t, -9), torch.full_like(r, -9))
    c = torch.zeros(2, dtype=torch.int32, device="cuda")
    gq.gqa_pages_compact(d, t, r, t2, r2, c, page_dim=1)
    assert c.tolist() == counts
    assert np.array_equal(t2.cpu().numpy(), want_t) and np.array_equal(r2.cpu().numpy(), want_r)
    for got, want in zip(d, moved(pools, pairs)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("live", ["none", "all"])
def test_compact_of_an_empty_and_a_full_pool(live):
    num = 100
    refs = np.full(num, 2 if live == "all" else 0, np.int32)
    table = (np.arange(num) if live == "all" else np.full(num, -1)).astype(np.int32).reshape(4, 25)
    pool = torch.arange(num, device="cuda").float().view(num, 1)
    t, r, c = dev(table), dev(refs), torch.zeros(2, dtype=torch.int32, device="cuda")
    gq.gqa_pages_compact([pool], t, r, t, r, c)
    assert c.tolist() == [0, num if live == "all" else 0]
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert pool.flatten().tolist() == list(range(num))


@pytest.mark.parametrize("n", [0, 1, 7, 300])
def test_copy(n):
    s = State(50, 4, 4, 16, 1000)
    pools = s.pools(("codes", "scale", "odd", "bf16", "big"))
    order = s.rng.permutation(1000)
    src, dst = order[:n].astype(np.int32), order[n:2 * n].astype(np.int32)
    if n > 5:
        src[2], dst[4] = -1, 1000               # skipped pairs
    pairs = [(a, b) for a, b in zip(src, dst) if 0 <= a < 1000 and 0 <= b < 1000]
    d = [dev(x) for x in pools]
    gq.gqa_pages_copy(d, dev(src), dev(dst), 1000, page_dim=1)
    for got, want in zip(d, moved(pools, pairs)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_copy_of_pools_at_odd_addresses_and_of_many_pools():
    buf = torch.randint(0, 100, (64 * 33 + 64,), dtype=torch.uint8, device="cuda")
    pools = [buf[k:k + 10 * 33].view(10, 33) for k in (1,)] + [torch.rand(10, 3, device="cuda") for _ in range(63)]
    src, dst = dev(np.array([1, 9], np.int32)), dev(np.array([0, 4], np.int32))
    want = [p.clone() for p in pools]
    for w in want:
        w[0], w[4] = w[1].clone(), w[9].clone()
    gq.gqa_pages_copy(pools, src, dst, 10)
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    with pytest.raises(gq.GQADecodeError) as e:
        gq.gqa_pages_copy(pools + pools[:1], src, dst, 10)
    assert e.value.status == gq.GQA_ERR_UNSUPPORTED


def test_page_past_2_31_bytes():
    num, size = 40, 1 << 26
    pool = torch.zeros(num, size, dtype=torch.uint8, device="cuda")
    pool[39] = 7
    pool[38, -1] = 3
    gq.gqa_pages_copy([pool], dev(np.array([39, 38], np.int32)), dev(np.array([1, 35], np.int32)), num)
    assert bool((pool[1] == 7).all()) and int(pool[35].sum()) == 3 and int(pool[35, -1]) == 3
    assert int(pool[0].sum()) == 0 and int(pool[2].sum()) == 0


def test_a_serving_loop_of_every_call_in_a_graph():
    """reserve, append, attend, fork, free and compact as one captured step,
    replayed with new tokens; the state follows the models, and the attention
    the oracle over what the models hold."""
    import math

    import oracle
    B, H, G, D, ps, most, num = 6, 8, 2, 64, 16, 8, 60
    rng = np.random.default_rng(60)
    nb = 1
    codes = [np.full((num, G, ps, D), model.NAN_CODE, np.uint8) for _ in range(2)]
    scales = [np.full((num, G, nb), np.nan, np.float32) for _ in range(2)]
    table, lens, refs = np.full((B, most), -1, np.int32), np.zeros(B, np.int32), np.zeros(num, np.int32)
    lens[:4] = [30, 16, 7, 45]
    i32 = dict(dtype=torch.int32, device="cuda")
    d = dict(k=dev(codes[0]), v=dev(codes[1]), ks=dev(scales[0]), vs=dev(scales[1]), table=dev(table), refs=dev(refs),
             lens=dev(lens), table2=torch.zeros(B, most, **i32), lens2=torch.zeros(B, **i32),
             refs2=torch.zeros(num, **i32), counts=torch.zeros(3, 2, **i32), src=torch.zeros(B, **i32),
             done=torch.zeros(B, dtype=torch.bool, device="cuda"))
    new = [torch.zeros(B, 1, G, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    sm = 1 / math.sqrt(D)
    pools = [d["k"], d["v"], d["ks"], d["vs"]]

    # the prompts
    prompt = [rng.standard_normal((B, 45, G, D)) for _ in range(2)]
    prompt = [torch.from_numpy(x).to(torch.bfloat16) for x in prompt]
    gq.gqa_pages_reserve(d["table"], d["lens"], d["refs"], ps, d["counts"][0])
    gq.gqa_append_paged_fp8(prompt[0].cuda(), prompt[1].cuda(), *pools, d["table"], d["lens"])
    table, refs, _ = model.reserve(table, lens, refs, ps)
    for c, s, x in zip(codes, scales, prompt):
        model.append(c, s, x.double().numpy(), table, lens)

    def step():
        gq.gqa_pages_fork(pools, d["src"], d["table"], d["lens"], d["refs"], ps, d["table2"], d["lens2"], d["refs2"],
                          d["counts"][0])
        gq.gqa_pages_free(d["done"], d["table2"], d["lens2"], d["refs2"])
        gq.gqa_pages_compact(pools, d["table2"], d["refs2"], d["table"], d["refs"], d["counts"][1])
        d["lens"].copy_(torch.where(d["lens2"] > 0, d["lens2"] + 1, d["lens2"]))
        gq.gqa_pages_reserve(d["table"], d["lens"], d["refs"], ps, d["counts"][2])
        gq.gqa_append_paged_fp8(new[0], new[1], *pools, d["table"], d["lens"])
        gq.gqa_decode_paged_fp8(q, *pools, d["table"], d["lens"], sm, out)

    saved = {k: x.clone() for k, x in d.items()}
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):       # every kernel is loaded before the capture
        side.wait_stream(torch.cuda.current_stream())
        step()
    torch.cuda.synchronize()
    for k, x in saved.items():
        d[k].copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for it in range(12):
        src = rng.integers(-1 if it % 3 == 2 else 0, B, B).astype(np.int32)
        done = rng.random(B) < (0.2 if it % 4 == 3 else 0.0)
        x = [torch.from_numpy(rng.standard_normal((B, 1, G, D)) * 2.0 ** (it % 3)).to(torch.bfloat16) for _ in range(2)]
        qh = torch.from_numpy(rng.standard_normal((B, 1, H, D))).to(torch.bfloat16)
        d["src"].copy_(dev(src))
        d["done"].copy_(dev(done))
        new[0].copy_(x[0])
        new[1].copy_(x[1])
        q.copy_(qh)
        graph.replay()
        torch.cuda.synchronize()
        assert gq.gqa_decode_check_error() == gq.GQA_OK
        table, lens, refs, c0, pairs = model.fork(src, table, lens, refs, ps)
        codes, scales = (moved([y[None] for y in z], pairs) for z in (codes, scales))
        codes, scales = [y[0] for y in codes], [y[0] for y in scales]
        table, lens, refs = model.free(done, table, lens, refs)
        table, refs, c1, pairs = model.compact(table, refs)
        codes, scales = (moved([y[None] for y in z], pairs) for z in (codes, scales))
        codes, scales = [y[0] for y in codes], [y[0] for y in scales]
        lens = np.where(lens > 0, lens + 1, lens).astype(np.int32)
        table, refs, c2 = model.reserve(table, lens, refs, ps)
        for c, s, y in zip(codes, scales, x):
            model.append(c, s, y.double().numpy(), table, lens)
        assert d["counts"].tolist() == [c0, c1, c2], it
        for name, want in (("table", table), ("lens", lens), ("refs", refs), ("ks", scales[0]), ("vs", scales[1])):
            got = d[name].cpu().numpy()
            assert np.array_equal(got, want, equal_nan=got.dtype == np.float32), (it, name)
        assert np.array_equal(d["k"].cpu().numpy() & 127 != 0, codes[0] & 127 != 0)
        k, v = (model.logical(model.page_values(c, s), table, lens, most * ps) for c, s in zip(codes, scales))
        ref, ref_lse = oracle.get().gqa_decode_kv(qh.view(torch.int16).numpy().view(np.uint16), k, v, lens, sm)
        vmax = np.nanmax(np.abs(v)) if (lens > 0).any() else 0.0
        err = np.abs(out.float().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * vmax).all(), (it, err.max())


@pytest.mark.parametrize("num", [262144, 262145, 300001])
def test_pools_of_many_pages(num):
    """More pages than the planning kernel's warps keep in one mask a lane."""
    s = State(70, 40, 6, 16, num)
    some = s.rng.choice(num, num // 2, replace=False)       # pages that holders outside the table count
    s.refs[some] += 1
    pool = s.rng.integers(0, 2 ** 31, (num, 1)).astype(np.int32)
    lens = np.full(40, 6 * 16, np.int32)
    want = model.reserve(s.table, lens, s.refs, 16)
    t, r, c = dev(s.table), dev(s.refs), torch.zeros(2, dtype=torch.int32, device="cuda")
    gq.gqa_pages_reserve(t, dev(lens), r, 16, c)
    assert c.tolist() == want[2]
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(r.cpu().numpy(), want[1])

    src = s.rng.integers(0, 40, 40).astype(np.int32)
    want_t, want_l, want_r, counts, pairs = model.fork(src, s.table, s.lens, s.refs, 16)
    d, t, l, r = dev(pool), dev(s.table), dev(s.lens), dev(s.refs)
    outs = [torch.full_like(x, -77) for x in (t, l, r)]
    gq.gqa_pages_fork([d], dev(src), t, l, r, 16, *outs, c)
    assert c.tolist() == counts
    for got, w in zip(outs, (want_t, want_l, want_r)):
        assert np.array_equal(got.cpu().numpy(), w)
    after = moved([pool[None]], pairs)[0][0]
    assert np.array_equal(d.cpu().numpy(), after)

    want_t, want_r, counts, pairs = model.compact(s.table, s.refs)
    d, t, r = dev(pool), dev(s.table), dev(s.refs)
    gq.gqa_pages_compact([d], t, r, t, r, c)
    assert c.tolist() == counts
    assert np.array_equal(t.cpu().numpy(), want_t) and np.array_equal(r.cpu().numpy(), want_r)
    assert np.array_equal(d.cpu().numpy(), moved([pool[None]], pairs)[0][0])


@pytest.mark.parametrize("B,most", [(3, 200), (700, 70), (8192, 3)])
def test_reserve_fills_holes(B, most):
    """Missing entries anywhere in a row, rows without any, entries outside the pool."""
    rng = np.random.default_rng(71)
    ps, num = 16, B * most + 7
    table = rng.permutation(num)[:B * most].reshape(B, most).astype(np.int32)
    holes = rng.random((B, most)) < rng.choice([0.0, 0.02, 0.7], (B, 1))
    refs = np.zeros(num, np.int32)
    refs[table[~holes]] = 1
    table[holes] = rng.choice([-1, -5, num, 2 ** 31 - 1], holes.sum())
    lens = rng.integers(0, most * ps + 1, B).astype(np.int32)
    want = model.reserve(table, lens, refs, ps)
    t, r, c = dev(table), dev(refs), torch.zeros(2, dtype=torch.int32, device="cuda")
    gq.gqa_pages_reserve(t, dev(lens), r, ps, c)
    assert c.tolist() == want[2]
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(r.cpu().numpy(), want[1])


def test_a_forked_copy_is_held_whatever_its_free_page_counted():
    """Counts below 0 are free pages too: the copies that take them count 1, and
    no later reservation hands them out again."""
    table = np.array([[0, 1], [0, 2], [-1, -1]], np.int32)
    lens, refs = np.array([20, 20, 0], np.int32), np.array([2, 1, 1, -3, -1, 0, 1, -7], np.int32)
    src = np.array([0, 0, 0], np.int32)
    t, l, r = dev(table), dev(lens), dev(refs)
    outs = [torch.zeros_like(x) for x in (t, l, r)]
    c = torch.zeros(2, dtype=torch.int32, device="cuda")
    gq.gqa_pages_fork([], dev(src), t, l, r, 16, *outs, c)
    assert c.tolist() == [2, 4]
    assert outs[0].tolist() == [[0, 1], [0, 3], [0, 4]] and outs[1].tolist() == [20, 20, 20]
    assert outs[2].tolist() == [3, 1, 0, 1, 1, 0, 1, -7]
    outs[1].copy_(dev(np.array([33, 20, 20], np.int32)))       # clamped to two pages: nothing to reserve
    gq.gqa_pages_reserve(outs[0], outs[1], outs[2], 16, c)
    assert c.tolist() == [0, 3]


def test_host_threads_fork_and_compact_on_one_stream():
    """Three threads on one stream, each with its own table and pool: forks,
    compactions, reservations and attention whose launches come in between each
    other's, results as those of the models."""
    import threading
    n, reps, ps = 3, 60, 16
    cases, errors = [], []
    for i in range(n):
        B, most, num = [(6, 5, 64), (33, 9, 500), (64, 40, 3000)][i]
        s = State(80 + i, B, most, ps, num)
        src = s.rng.integers(0, B, B).astype(np.int32)
        pool = s.pools(("scale",))[0]
        cases.append((s, src, pool, model.fork(src, s.table, s.lens, s.refs, ps)))
    q = torch.ones(4, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    pages, scale = torch.full((4, 2, ps, 64), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(4, 2, 1, device="cuda")
    short, some = dev(np.arange(4, dtype=np.int32)[:, None]), dev(np.full(4, ps, np.int32))
    data = [(dev(src), dev(s.table), dev(s.lens), dev(s.refs), [dev(pool) for _ in range(reps)]) for s, src, pool, _ in cases]
    torch.cuda.synchronize()
    start = threading.Barrier(n)

    def work(i):
        try:
            s, src, pool, (want_t, want_l, want_r, counts, pairs) = cases[i]
            d_src, t, l, r, pools = data[i]
            outs = [[torch.full_like(x, -77) for x in (t, l, r)] for _ in range(reps)]
            after = [[torch.full_like(x, -77) for x in (t, r)] for _ in range(reps)]
            c = [torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2 * reps)]
            o = torch.empty_like(q)
            start.wait(60)
            for k in range(reps):
                gq.gqa_pages_fork([pools[k]], d_src, t, l, r, ps, *outs[k], c[2 * k], page_dim=1)
                gq.gqa_decode_paged_fp8(q, pages, pages, scale, scale, short, some, 0.1, o)
                gq.gqa_pages_compact([pools[k]], outs[k][0], outs[k][2], *after[k], c[2 * k + 1], page_dim=1)
            torch.cuda.synchronize()
            moved_once = moved([pool], pairs)[0]
            final_t, final_r, final_c, final_pairs = model.compact(want_t, want_r)
            want_pool = moved([moved_once], final_pairs)[0]
            for k in range(reps):
                assert c[2 * k].tolist() == counts and c[2 * k + 1].tolist() == final_c, k
                for got, want in zip(outs[k] + after[k] + [pools[k]], (want_t, want_l, want_r, final_t, final_r, want_pool)):
                    assert np.array_equal(got.cpu().numpy(), want), k
            assert bool((o == 1).all())
        except Exception as e:                    # a thread's failure is the test's
            errors.append((i, repr(e)[:500]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors and not any(t.is_alive() for t in threads), errors
