"""Attention of packed batches (gqa_prefill_packed, gqa_prefill_paged) against a
float64 model with derived bounds: head groups of 1 to 128, both head sizes,
sequences without new tokens, without keys and with fewer keys than new tokens,
page sizes below and above a tile, NaN and infinities in masked places, views of
fused projections, padded batches, captured graphs and streams that overlap."""
import math
import threading

import pytest
import torch

import grouped_query_decode_gb300 as gq
import ragged_model as model
from gpu_helpers import env

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
I32 = torch.int32


def normal(shape, g, spread=1.0):
    return (torch.randn(*shape, generator=g) * spread).to(BF)


class Batch:
    """A packed batch on the CPU and the device; page 0 of sequences is drawn from
    one shuffled pool whose other entries, and slots past the lengths, hold NaN."""

    def __init__(self, H, G, D, seqs, page=0, behind=0, seed=0, fill=math.nan, spread=1.0):
        g = torch.Generator().manual_seed(1000 + seed)
        self.H, self.G, self.D, self.seqs, self.page = H, G, D, seqs, page
        news = [n for n, _ in seqs]
        self.N = sum(news) + behind
        self.cu = torch.tensor([0] + news).cumsum(0).to(I32)
        self.scale = 1 / math.sqrt(D)
        self.q = normal((self.N, H, D), g, spread)
        self.q[sum(news):] = fill
        if page == 0:
            self.k, self.v = (normal((self.N, G, D), g) for _ in range(2))
            for x in (self.k, self.v):
                x[sum(news):] = fill
        else:
            need = [-(-T // page) for _, T in seqs]
            num = sum(need) + 2
            order = torch.randperm(num, generator=g, dtype=I32)
            self.table = torch.full((len(seqs), max(need + [1])), -1, dtype=I32)
            self.pages = [torch.full((num, G, page, D), fill, dtype=BF) for _ in range(2)]
            self.held, at = [], 0
            for b, (_, T) in enumerate(seqs):
                self.table[b, :need[b]] = order[at:at + need[b]]
                at += need[b]
                kv = [normal((T, G, D), g) for _ in range(2)]
                self.held.append(kv)
                t = torch.arange(T)
                for pool, x in zip(self.pages, kv):
                    pool[self.table[b].long()[t // page], :, t % page] = x
            self.lens = torch.tensor([T for _, T in seqs], dtype=I32)

    def device(self):
        self.dq = self.q.cuda()
        self.out = torch.full((self.N, self.H, self.D), 7.0, dtype=BF, device="cuda")
        self.lse = torch.full((self.N, self.H), 7.0, device="cuda")
        self.dcu = self.cu.cuda()
        if self.page:
            self.dp = [p.cuda() for p in self.pages]
            self.dt, self.dl = self.table.cuda(), self.lens.cuda()
        else:
            self.dk, self.dv = self.k.cuda(), self.v.cuda()
        return self

    def call(self, **kw):
        if self.page:
            gq.gqa_prefill_paged(self.dq, *self.dp, self.dt, self.dcu, self.dl, self.scale, self.out, self.lse, **kw)
        else:
            gq.gqa_prefill_packed(self.dq, self.dk, self.dv, self.dcu, self.scale, self.out, self.lse, **kw)

    def run(self, **kw):
        self.device()
        self.call(**kw)
        torch.cuda.synchronize()
        assert gq.gqa_decode_check_error() == gq.GQA_OK
        return self

    def kv(self, b):
        if self.page:
            return self.held[b]
        i, j = int(self.cu[b]), int(self.cu[b + 1])
        return self.k[i:j], self.v[i:j]

    def check(self, what=""):
        for b, (n, T) in enumerate(self.seqs):
            i = int(self.cu[b])
            want = model.attention(self.q[i:i + n], *self.kv(b), n, T, self.scale)
            model.check_rows(self.out[i:i + n], self.lse[i:i + n], want, f"{what} sequence {b}: {n} of {T}")
        end = int(self.cu[-1])
        assert (self.out[end:].float() == 7).all() and (self.lse[end:] == 7).all(), "rows behind the last sequence"
        return self


# ------------------------------------------------------------------ packed

PACKED = [  # H, G, D, lengths, rows behind the last
    (8, 2, 64, [1], 0),
    (8, 2, 128, [17, 1, 0, 40], 3),
    (4, 4, 128, [300, 129, 128, 127], 0),            # a KV head for every head
    (6, 2, 64, [200, 77, 43, 42], 0),                # three heads: 42 tokens fill 126 of 128 rows
    (32, 1, 128, [130, 4, 5], 1),                    # 32 heads: four tokens a tile
    (128, 1, 64, [9, 2], 0),                         # a token a tile
    (127, 1, 64, [6], 0),
    (10, 2, 128, [260, 1, 25], 0),
    (7, 1, 64, [333], 2),
    (24, 3, 128, [64, 65, 500], 0),
    (16, 2, 64, [1000, 3], 0),
    (2, 1, 128, [700, 701], 0),
    (1, 1, 64, [257, 255], 0),
    (64, 64, 64, [33, 1], 0),
]


@pytest.mark.parametrize("H,G,D,lens,behind", PACKED, ids=lambda x: str(x))
def test_packed(H, G, D, lens, behind):
    Batch(H, G, D, [(n, n) for n in lens], behind=behind, seed=H + D).run().check()


def test_packed_many_sequences():
    r = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 12, (700,), generator=r).tolist()
    Batch(4, 2, 64, [(n, n) for n in lens], behind=2, seed=6).run().check()
    Batch(4, 2, 128, [(0, 0)] * 300 + [(3, 3)] + [(0, 0)] * 900 + [(150, 150)] + [(0, 0)] * 5, seed=7).run().check()


@pytest.mark.parametrize("D", [64, 128])
def test_packed_views_of_a_fused_projection(D):
    H, G, lens = 8, 2, [70, 131, 9]
    b = Batch(H, G, D, [(n, n) for n in lens], seed=8).device()
    x = torch.cat([b.q, b.k, b.v], 1).cuda()
    b.dq, b.dk, b.dv = x[:, :H], x[:, H:H + G], x[:, H + G:]
    b.call()
    b.check()
    wide = torch.full((b.N, H + 5, D), math.nan, dtype=BF, device="cuda")      # another stride, not of 16 rows
    wide[:, 1:1 + H] = b.q.cuda()
    first = b.out.clone()
    b.dq = wide[:, 1:1 + H]
    b.call()
    assert torch.equal(first, b.out)


def test_sharp_softmax_and_rising_maxima():
    """Scores that grow along the sequence move the running maximum in every tile."""
    for D, H, G in ((128, 4, 1), (64, 4, 4)):
        b = Batch(H, G, D, [(640, 640), (300, 300)], seed=9)
        ramp = torch.linspace(0.2, 6.0, b.N)[:, None, None]
        b.k = (b.k.float() * ramp).to(BF)
        b.scale = 0.5
        b.run().check("ramp")
        b.k = b.k.flip(0).contiguous()
        b.run().check("falling")


def test_lse_is_optional_and_repeats_are_equal():
    b = Batch(8, 2, 128, [(500, 500), (77, 77), (1, 1)], seed=10).run().check()
    out, lse = b.out.clone(), b.lse.clone()
    for _ in range(5):
        b.out.fill_(3)
        b.call()
        assert torch.equal(out, b.out) and torch.equal(lse, b.lse)
    b.lse = None
    b.out.fill_(3)
    b.call()
    assert torch.equal(out, b.out)


# ------------------------------------------------------------------- paged

PAGED = [  # H, G, D, (new, all) tokens, page
    (8, 2, 128, [(1, 1), (1, 100), (1, 4000), (1, 128), (1, 129)], 16),
    (8, 2, 64, [(1, 5000)], 32),
    (32, 8, 64, [(64, 1000), (1, 77), (0, 50), (5, 5), (130, 600)], 64),
    (4, 4, 128, [(200, 900), (1, 300), (128, 128)], 128),
    (6, 2, 128, [(50, 333), (43, 43), (1, 2000)], 256),
    (16, 1, 64, [(7, 1024), (9, 500), (1, 1)], 1024),
    (128, 1, 128, [(3, 300), (1, 2500)], 16),
    (5, 1, 128, [(26, 1000), (1, 999)], 32),
    (8, 2, 128, [(5, 3), (4, 0), (300, 200), (1, 0), (2, 2)], 16),       # rows that see nothing
    (2, 2, 64, [(257, 700), (255, 256)], 16),
    (64, 8, 128, [(4, 20000), (4, 513)], 64),
]


@pytest.mark.parametrize("H,G,D,seqs,page", PAGED, ids=lambda x: str(x))
def test_paged(H, G, D, seqs, page):
    Batch(H, G, D, seqs, page=page, behind=len(seqs) % 3, seed=H + D + page).run().check()


def test_paged_serving_batches():
    """Many single tokens beside chunks: units of unlike lengths, shared out over all CTAs."""
    r = torch.Generator().manual_seed(3)
    for D, G, page in ((128, 2, 16), (64, 4, 64)):
        seqs = []
        for b in range(90):
            T = int(torch.randint(1, 3000, (1,), generator=r))
            n = 1 if b % 7 else min(T, int(torch.randint(1, 400, (1,), generator=r)))
            seqs.append((n, T))
        Batch(4 * G, G, D, seqs, page=page, behind=5, seed=11).run().check()


@pytest.mark.parametrize("D,H,G,B,every", [(64, 32, 32, 128, 5), (128, 8, 2, 1000, 9), (128, 16, 16, 100, 100), (64, 4, 4, 700, 701)])
def test_padded_batches(D, H, G, B, every):
    """A batch padded with tokens of sequences without a key: runs of units in which there
    is nothing to do, far longer than the list that hands units on."""
    seqs = [(1, 300 + b) if (b + 1) % every == 0 else (1 + b % 3, 0) for b in range(B)]
    Batch(H, G, D, seqs, page=32, behind=2, seed=64).run().check()


def test_units_that_take_longer_than_a_wait():
    """Units of 12 million keys, one to a CTA (their pages are one page, again and again), take
    longer than a wait for a step is given here, 10 ms. Keys of zero: out is the mean
    of equal values, lse the logarithm of the number of keys."""
    H, G, D, page, pages = 128, 1, 64, 65536, 192
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N, T = 2 * sms, page * pages
    k = torch.zeros(1, G, page, D, dtype=BF, device="cuda")
    v = (2.0 ** (torch.arange(D, device="cuda") % 7 - 3)).to(BF).expand_as(k).contiguous()
    q = normal((N, H, D), torch.Generator().manual_seed(65)).cuda()
    table = torch.zeros(1, pages, dtype=I32, device="cuda")
    cu, lens = torch.tensor([0, N], dtype=I32, device="cuda"), torch.tensor([T], dtype=I32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(N, H, device="cuda")
    with env(GQA_DECODE_DEBUG_TIMEOUT_MS=10):
        gq.gqa_prefill_paged(q, k, v, table, cu, lens, 0.125, out, lse)
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    assert torch.equal(out, v[0, 0, 0].expand_as(out))
    want = torch.log(torch.arange(T - N + 1, T + 1, dtype=torch.float64))
    # log2 and the product, 2^-23 each of at most 23.6 and 16.4
    assert (lse.double().cpu() - want[:, None]).abs().max() < 1e-5


def test_paged_unusable_entries_and_clamped_lengths():
    """Entries outside the pool read as zeros; lengths are cut to the table's."""
    b = Batch(8, 2, 64, [(3, 100), (1, 60), (4, 64)], page=16, seed=12, fill=2.0)
    b.table[0, 1], b.table[0, 4], b.table[1, 0] = -7, 1 << 30, b.pages[0].shape[0]
    for x in b.held[0]:
        x[16:32], x[64:80] = 0, 0
    for x in b.held[1]:
        x[:16] = 0
    b.run().check("entries")
    b = Batch(8, 2, 64, [(3, 112), (2, 64)], page=16, seed=13)          # 7 pages
    b.device()
    b.dl = torch.tensor([100000, 64], dtype=I32, device="cuda")
    b.call()
    b.check("clamped")
    b.dl = torch.tensor([-5, 64], dtype=I32, device="cuda")
    b.seqs = [(3, 0), (2, 64)]
    b.held[0] = [x[:0] for x in b.held[0]]
    b.call()
    b.check("negative")


def test_malformed_offsets_stay_inside():
    """cu past the rows or descending: what is defined is right, nothing outside is touched."""
    b = Batch(4, 2, 64, [(10, 10), (20, 20), (5, 5)], behind=4, seed=14).device()
    b.dcu = torch.tensor([0, 10, 30, 1000], dtype=I32, device="cuda")     # the last takes all rows to N
    b.k[35:], b.v[35:], b.q[35:] = 1.0, 1.0, 1.0
    b.dq, b.dk, b.dv = b.q.cuda(), b.k.cuda(), b.v.cuda()
    b.call()
    b.seqs, b.cu = [(10, 10), (20, 20), (9, 9)], torch.tensor([0, 10, 30, 39], dtype=I32)
    b.check()
    b.dcu = torch.tensor([5, 3, -8, 1 << 30], dtype=I32, device="cuda")
    b.call()
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK


@pytest.mark.parametrize("D", [64, 128])
def test_units_in_many_parts(D):
    """Few tokens with many heads behind a long context: one unit over nearly all CTAs,
    whose parts are merged a few rows at a time; and one with a part of its own per head."""
    Batch(32, 1, D, [(8, 60000)], page=256, seed=60).run().check()
    Batch(8, 2, D, [(1, 40000), (1, 3)], page=64, seed=61).run().check()
    Batch(16, 1, D, [(13, 9000), (16, 700)], page=32, seed=62).run().check()


def test_outputs_on_16_bytes():
    """Outputs need no more than the 16 bytes that the header asks for; lse none but its own."""
    b = Batch(8, 2, 64, [(130, 130), (5, 5)], seed=63).device()
    buf = torch.full((b.out.numel() + 16,), 7.0, dtype=BF, device="cuda")
    lse = torch.full((b.lse.numel() + 1,), 7.0, device="cuda")
    b.out, b.lse = buf[8:8 + b.out.numel()].view(b.out.shape), lse[1:].view(b.lse.shape)
    b.call()
    b.check()
    assert (buf[:8].float() == 7).all() and (buf[-8:].float() == 7).all() and lse[0] == 7


def test_scores_without_any_key_left():
    """Rows whose every visible key scores -inf weigh nothing: out 0, lse -inf, as rows that see nothing."""
    b = Batch(4, 1, 64, [(40, 40)], seed=64)
    b.q = b.q.abs() + 0.5
    b.k[:3] = -math.inf
    b.run()
    assert (b.out[:3].float() == 0).all() and torch.isneginf(b.lse[:3]).all()
    assert torch.isfinite(b.out[3:].float()).all()


# -------------------------------------------------- NaN and masked positions

@pytest.mark.parametrize("D,H,G", [(128, 8, 2), (64, 2, 2), (64, 3, 1)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite(D, H, G, value):
    """V at position t reaches the rows that see t, in its column alone; rows before t not at all."""
    b = Batch(H, G, D, [(300, 300), (200, 200)], seed=15)
    for t, c in ((70, 3), (71, D - 1), (299, 0), (128, 8)):
        b.v[t, 0, c] = value
    b.run().check()
    p = Batch(H, G, D, [(140, 400), (1, 300)], page=16, seed=16)
    for t, c in ((10, 5), (300, 3), (399, 7)):
        p.held[0][1][t, 0, c] = value
        p.pages[1][int(p.table[0, t // 16]), 0, t % 16, c] = value
    p.run().check()


def test_keys_that_are_nan():
    b = Batch(8, 2, 128, [(300, 300), (40, 40)], seed=17)
    b.k[130, 1, 5] = math.nan
    b.run()
    out, lse = b.out.float().cpu(), b.lse.cpu()
    assert torch.isfinite(out[:130]).all() and torch.isfinite(out[:, :4]).all() and torch.isfinite(out[300:]).all()
    assert torch.isnan(out[130:300, 4:]).all() and torch.isnan(lse[130:300, 4:]).all()


def test_queries_of_other_rows_do_not_matter():
    b = Batch(8, 2, 64, [(100, 100), (60, 60)], seed=18).run().check()
    out = b.out.clone()
    b.q[33], b.q[120, 5] = math.nan, math.inf
    b.device()
    b.call()
    same = torch.ones(160, 8, dtype=torch.bool)
    same[33], same[120, 5] = False, False
    assert torch.equal(b.out[same.cuda()], out[same.cuda()])
    assert not torch.isfinite(b.out[33].float()).any()


def test_tokens_far_into_a_pool_past_32_bits():
    """Element offsets past 2^31: pages at the end of a pool of 2.2e9 elements."""
    G, page, D = 8, 256, 128
    num = (1 << 31) // (G * page * D) + 40
    b = Batch(16, G, D, [(3, 1000), (1, 700)], page=page, seed=19)
    pools = [torch.full((num, G, page, D), math.nan, dtype=BF, device="cuda") for _ in range(2)]
    b.device()
    shift = num - b.pages[0].shape[0]
    for pool, small in zip(pools, b.dp):
        pool[shift:] = small
    b.dp, b.dt = pools, torch.where(b.dt >= 0, b.dt + shift, b.dt)
    b.call()
    b.check()


# ----------------------------------------------------- workspaces and streams

def test_workspace_of_the_caller():
    b = Batch(8, 2, 128, [(3, 5000), (200, 900)], page=64, seed=20).run().check()
    out = b.out.clone()
    need = gq.gqa_prefill_ragged_workspace_bytes(b.N, 2, 8, 2, 128)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    b.out.zero_()
    b.call(workspace=ws[:need])
    assert torch.equal(out, b.out) and (ws[need:] == 0xA5).all()
    for bad in (ws[:need - 1], ws[16:16 + need]):
        with pytest.raises(gq.GQADecodeError) as e:
            b.call(workspace=bad)
        assert e.value.status == gq.GQA_ERR_WORKSPACE


def test_graphs_replayed_with_other_lengths():
    """The plan is made on the device: a replay takes new lengths, and two graphs overlap."""
    a = Batch(8, 2, 128, [(1, 3000), (60, 500), (3, 64)], page=16, seed=21).run()
    b = Batch(8, 2, 64, [(300, 300), (5, 5)], seed=22).run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for x, s in zip((a, b), streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            x.call()
        graphs.append(graph)
    for _ in range(4):
        for x in (a, b):
            x.out.fill_(7)
            x.lse.fill_(7)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()
    c = Batch(8, 2, 64, [(12, 12), (290, 290), ], behind=3, seed=23)
    for mine, other in ((b.dq, c.q), (b.dk, c.k), (b.dv, c.v), (b.dcu, c.cu)):
        mine.copy_(other)
    b.out.fill_(7)
    b.lse.fill_(7)
    torch.cuda.synchronize()
    graphs[1].replay()
    torch.cuda.synchronize()
    c.out, c.lse = b.out, b.lse
    c.check("other lengths")


def test_streams_that_overlap():
    batches = [Batch(8, 2, 128, [(1, 2000 + 300 * i), (30, 400)], page=32, seed=30 + i).device() for i in range(4)]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                b.call()
    torch.cuda.synchronize()
    for b in batches:
        b.check()
    b.out.fill_(7)
    torch.cuda.synchronize()
    b.call(stream=streams[0])
    torch.cuda.synchronize()
    b.check()


def test_host_threads_on_one_stream():
    """Threads that share a stream share no workspace."""
    batches = [Batch(8, 2, 128, [(3, 4000 + 500 * i), (40, 300)], page=32, seed=70 + i).device() for i in range(4)]
    torch.cuda.synchronize()
    stream, failed = torch.cuda.Stream(), []

    def work(b):
        try:
            with torch.cuda.stream(stream):
                for _ in range(20):
                    b.call()
        except Exception as e:          # noqa: BLE001 (reported below)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(b,)) for b in batches]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for b in batches:
        b.check()


def test_no_tokens():
    e = torch.empty(0, 8, 64, dtype=BF, device="cuda")
    k = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    cu = torch.zeros(3, dtype=I32, device="cuda")
    gq.gqa_prefill_packed(e, k, k, cu, 0.1, e.clone())
    b = Batch(8, 2, 64, [(0, 50), (0, 0)], page=16, behind=6, seed=24).run()
    b.check()


# ------------------------------------------------------------ a serving step

@pytest.mark.parametrize("interleaved", [False, True])
def test_a_serving_loop(interleaved):
    """Reserve, append with rotation, attention, over steps of prompts and single
    tokens, against the model over what a plain cache holds."""
    H, G, D, page, num = 8, 2, 64, 16, 120
    g = torch.Generator().manual_seed(40)
    rope = gq.gqa_rope_init(D, dims=48, interleaved=interleaved, base=500000.0, scaling="bands", factor=8.0,
                            original=64.0, low=1.0, high=4.0)
    f, gain = model.frequencies(48, 500000.0, "bands", 8.0, 64.0, 1.0, 4.0)
    B = 3
    pages = [torch.full((num, G, page, D), math.nan, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.full((B, 40), -1, dtype=I32, device="cuda")
    refs, counts = torch.zeros(num, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")
    lens = [0] * B
    held = [[torch.empty(0, G, D, dtype=BF)] * 2 for _ in range(B)]
    for news in ([70, 0, 5], [1, 130, 1], [1, 1, 1], [1, 1, 40], [9, 1, 1]):
        n_all = sum(news)
        cu = torch.tensor([0] + news).cumsum(0).to(I32)
        lens = [T + n for T, n in zip(lens, news)]
        x = normal((n_all, H + 2 * G, D), g)
        dx, dl, dcu = x.cuda(), torch.tensor(lens, dtype=I32, device="cuda"), cu.cuda()
        q = torch.empty(n_all, H, D, dtype=BF, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(n_all, H, device="cuda")
        gq.gqa_pages_reserve(table, dl, refs, page, counts)
        gq.gqa_append_paged(dx[:, H:H + G], dx[:, H + G:], *pages, table, dcu, dl, rope=rope, q=dx[:, :H], q_out=q)
        gq.gqa_prefill_paged(q, *pages, table, dcu, dl, 0.125, out, lse)
        torch.cuda.synchronize()
        assert gq.gqa_decode_check_error() == gq.GQA_OK
        t = table.cpu().long()
        pos = torch.cat([torch.arange(T - n, T) for n, T in zip(news, lens)])
        want_q = model.rotate(x[:, :H], pos, f, gain, interleaved)
        assert ((q.double().cpu() - want_q[0]).abs() <= model.rotate_bound(*want_q)).all()
        for b, (n, T) in enumerate(zip(news, lens)):
            i, at = int(cu[b]), torch.arange(T)
            k, v = (p.cpu()[t[b, at // page], :, at % page] for p in pages)
            held[b][1] = torch.cat([held[b][1], x[i:i + n, H + G:]])
            assert torch.equal(v, held[b][1])
            assert torch.equal(k[:T - n], held[b][0])                    # older keys as they were
            want_k = model.rotate(x[i:i + n, H:H + G], torch.arange(T - n, T), f, gain, interleaved)
            assert ((k[T - n:].double() - want_k[0]).abs() <= model.rotate_bound(*want_k)).all()
            held[b][0] = k
            model.check_rows(out[i:i + n], lse[i:i + n], model.attention(q.cpu()[i:i + n], k, v, n, T, 0.125))


def test_a_captured_serving_step():
    """Reserve, append and attention in one graph, replayed as the lengths grow."""
    H, G, D, page, num, B = 4, 1, 128, 16, 60, 2
    g = torch.Generator().manual_seed(41)
    rope = gq.gqa_rope_init(D)
    f, gain = model.frequencies(D, 10000.0)
    pages = [torch.zeros(num, G, page, D, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.full((B, 20), -1, dtype=I32, device="cuda")
    refs, counts = torch.zeros(num, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")
    x = torch.zeros(8, H + 2 * G, D, dtype=BF, device="cuda")
    q, out = torch.zeros(8, H, D, dtype=BF, device="cuda"), torch.zeros(8, H, D, dtype=BF, device="cuda")
    cu, lens = torch.zeros(B + 1, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")

    def step():
        gq.gqa_pages_reserve(table, lens, refs, page, counts)
        gq.gqa_append_paged(x[:, H:H + G], x[:, H + G:], *pages, table, cu, lens, rope=rope, q=x[:, :H], q_out=q)
        gq.gqa_prefill_paged(q, *pages, table, cu, lens, 0.1, out)

    step()                                           # no tokens: nothing grows
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    T = [0, 0]
    for news in ([5, 3], [1, 1], [1, 7], [0, 8], [4, 1]):
        T = [a + n for a, n in zip(T, news)]
        x.copy_(normal(tuple(x.shape), g))
        cu.copy_(torch.tensor([0] + news).cumsum(0))
        lens.copy_(torch.tensor(T))
        graph.replay()
        torch.cuda.synchronize()
        first = 0
        for b, n in enumerate(news):
            at = torch.arange(T[b])
            k, v = (p.cpu()[table.cpu().long()[b, at // page], :, at % page] for p in pages)
            want = model.rotate(x.cpu()[first:first + n, H:H + G], at[T[b] - n:], f, gain)
            assert ((k[T[b] - n:].double() - want[0]).abs() <= model.rotate_bound(*want)).all()
            model.check_rows(out[first:first + n], None, model.attention(q.cpu()[first:first + n], k, v, n, T[b], 0.1))
            first += n


# ------------------------------------------------------- bounded waits

def test_a_tile_that_never_comes():
    """A load that is left out ends in a status, not in a hang, and leaves the
    workspace so that the same call is right afterwards."""
    b = Batch(8, 2, 128, [(1, 3000), (200, 900)], page=64, seed=50).run().check()
    with env(GQA_DECODE_DEBUG_SKIP_TILE=0, GQA_DECODE_DEBUG_TIMEOUT_MS=50, GQA_DECODE_DEBUG_EPOCH=77):
        b.call()
        assert gq.gqa_decode_check_error() == gq.GQA_ERR_DEVICE_TIMEOUT
    with env(GQA_DECODE_DEBUG_EPOCH=77):
        for _ in range(2):
            b.out.fill_(7)
            b.lse.fill_(7)
            b.call()
            torch.cuda.synchronize()
            assert gq.gqa_decode_check_error() == gq.GQA_OK
            b.check()
