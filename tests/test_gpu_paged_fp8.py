"""Attention over the paged 8-bit cache on the GPU, against the float64 oracle
over the values the pages hold. Everything the call must not use holds NaN:
pages of no sequence, rows past a length, and their blocks' scales.

Bounds (arithmetic, for N(0,1)-sized values; vmax = max |v| that a row sees):
  scores: fp32 sums of D <= 128 products, error at most D 2^-24 sum|q k| scale
      <= 2^-14 for |scores| of a few units: taken as 2^-13, in natural units;
  out: output rounding 2^-8 |out|; probabilities rounded to fp16, 2^-11 vmax,
      or by at most 2^-24 of the largest one each, T 2^-24 vmax; the scores'
      error twice (numerator and sum), 2^-12 vmax;
  lse: the scores' error, fp32 sums of T terms T 2^-24, and its own rounding.
"""
import math

import numpy as np
import pytest
import torch

import grouped_query_decode_gb300 as gq
import oracle
import paged_fp8_model as model
import synthetic as syn
from gpu_helpers import _CANARY_BF16, _CANARY_F32, _PAD, bf16_to_f64, env, to_device_bf16

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed, B, sq, H, G, D, page, lens, most=None, spread=1.0, extra=3, scale_spread=0):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        self.most = most or max(1, -(-int(self.lens.max()) // page))
        need = [-(-min(max(int(t), 0), self.most * page) // page) for t in self.lens]
        num = sum(need) + extra
        order = rng.permutation(num).astype(np.int32)
        self.table = np.full((B, self.most), -1, np.int32)
        self.shape = (B, sq, H, G, D, page)
        self.q = syn.normal_bf16(seed, syn.STREAM_Q, (B, sq, H, D))
        self.sm = 1 / math.sqrt(D)
        nb = model.blocks_of(page)
        self.codes, self.scales = [], []
        for _ in range(2):
            s = (0.5 + rng.random((num, G, nb))) / 100 * spread
            s = (s * np.exp2(rng.integers(-scale_spread, scale_spread + 1, s.shape))).astype(np.float32)
            c = model.nearest_codes(np.clip(rng.standard_normal((num, G, page, D)) * 80, -448, 448))
            self.codes.append(c)
            self.scales.append(s)
        at, size = 0, model.block_tokens(page)
        used = np.zeros((num, page), bool)
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
            T = min(max(int(self.lens[b]), 0), self.most * page)
            for j in range(n):
                used[self.table[b, j], :max(0, min(page, T - j * page))] = True
        for c, s in zip(self.codes, self.scales):
            c.transpose(0, 2, 1, 3)[~used] = model.NAN_CODE
            live = used.reshape(num, nb, size).any(2)
            s.transpose(0, 2, 1)[~live] = np.nan

    def reference(self):
        B, sq, H, G, D, page = self.shape
        tmax = self.most * page
        with np.errstate(invalid="ignore"):
            k, v = (model.logical(model.page_values(c, s), self.table, self.lens, tmax)
                    for c, s in zip(self.codes, self.scales))
        lens = np.clip(self.lens, 0, tmax)
        out, lse = oracle.get().gqa_decode_kv(self.q, k, v, lens, self.sm, threads=8)
        self.vmax = np.zeros((B, 1, H, 1))
        for b in range(B):
            if lens[b]:
                top = np.abs(v[b, :, :lens[b]]).max((1, 2))
                self.vmax[b, 0, :, 0] = np.repeat(top, H // G)
        return out, lse

    def device(self):
        d = [to_device_bf16(self.q)]
        d += [torch.from_numpy(x).cuda() for x in (*self.codes, *self.scales)]
        d += [torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda()]
        return d


def guarded(shape, dtype, canary):
    n = math.prod(shape)
    buf = torch.empty(n + 2 * _PAD, dtype=dtype, device="cuda")
    buf.view(torch.int16 if dtype == torch.bfloat16 else torch.int32).fill_(canary)
    return buf, buf[_PAD:_PAD + n].view(shape)


F32_CANARY = int(np.float32(_CANARY_F32).view(np.int32))
BF_CANARY = int(np.uint16(_CANARY_BF16).view(np.int16))


def run(case, dev=None, with_lse=True, **kw):
    B, sq, H, G, D, page = case.shape
    dev = dev or case.device()
    obuf, out = guarded((B, sq, H, D), torch.bfloat16, BF_CANARY)
    lbuf, lse = guarded((B, sq, H), torch.float32, F32_CANARY)
    gq.gqa_decode_paged_fp8(*dev, case.sm, out, lse if with_lse else None, **kw)
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    for buf, c in ((obuf.view(torch.int16), BF_CANARY), (lbuf.view(torch.int32), F32_CANARY)):
        assert (buf[:_PAD] == c).all() and (buf[-_PAD:] == c).all(), "guard words"
    if not with_lse:
        assert (lbuf.view(torch.int32) == F32_CANARY).all()
    return bf16_to_f64(out), lse.cpu().numpy().astype(np.float64)


def check(case, out, lse, ref=None, what=""):
    ref_out, ref_lse = ref or case.reference()
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty), what
    assert (out[empty] == 0).all(), what
    T = max(1, int(np.clip(case.lens, 0, None).max()))
    assert np.isfinite(out).all(), what
    bound = 2.0 ** -8 * np.abs(ref_out) + (2.0 ** -11 + 2.0 ** -12 + T * 2.0 ** -24) * case.vmax
    excess = np.abs(out - ref_out) - bound
    assert excess.max() <= 0, (what, excess.max(), np.abs(out - ref_out).max())
    lerr = np.abs(lse[~empty] - ref_lse[~empty])
    lbound = 2.0 ** -13 + T * 2.0 ** -24 + 2.0 ** -23 * np.abs(ref_lse[~empty])
    assert (lerr <= lbound).all(), (what, lerr.max())


LENS = [1, 15, 64, 65, 127, 128, 129, 200, 511, 512, 0]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G,sq", [(8, 8, 1), (32, 8, 1), (16, 2, 1), (24, 2, 1), (32, 1, 1), (64, 8, 4), (6, 2, 3)],
                         ids=str)
def test_matches_the_oracle(H, G, sq, D, page):
    c = Case(100 + H + sq + D + page, len(LENS), sq, H, G, D, page, LENS)
    check(c, *run(c))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G,sq,T", [(32, 8, 64, 300), (8, 2, 130, 257), (40, 1, 1, 300), (32, 1, 7, 140), (4, 4, 129, 129)],
                         ids=str)
def test_many_rows(H, G, sq, T, D):
    """More than 32 rows per KV head: prompt chunks and wide groups."""
    c = Case(300 + H + sq + D, 2, sq, H, G, D, 64, [T, max(1, T // 3)], most=5)
    check(c, *run(c))


@pytest.mark.parametrize("page,D,T", [(16, 128, 20000), (64, 64, 33333), (256, 128, 8192)])
def test_long_and_split(page, D, T):
    """One sequence split over every SM, next to a short one."""
    c = Case(400 + page, 2, 1, 16, 2, D, page, [T, 130])
    check(c, *run(c))


@pytest.mark.parametrize("B,H,G,T,page", [(16, 32, 8, 1100, 64), (5, 16, 16, 1500, 32), (64, 16, 1, 1030, 16), (38, 8, 8, 300, 64),
                                          (128, 4, 2, 130, 16), (129, 4, 2, 130, 16), (400, 2, 1, 100, 32)], ids=str)
def test_equal_lengths(B, H, G, T, page):
    """Batches of one length, whose grid leaves SMs idle so that no unit is cut
    unevenly; and batches on each side of the per-warp plan's size."""
    c = Case(450 + B, B, 1, H, G, 128, page, [T] * B)
    check(c, *run(c))


@pytest.mark.parametrize("lens", [[1], [2], [3], [128], [127, 1, 0, 300]])
@pytest.mark.parametrize("sq", [1, 4])
def test_short_sequences_and_rows_without_a_key(lens, sq):
    c = Case(500 + sq, len(lens), sq, 16, 4, 128, 16, lens)
    check(c, *run(c))


def test_lengths_are_clamped():
    c = Case(510, 3, 1, 8, 2, 64, 16, [500, -3, 17], most=4)
    check(c, *run(c))


@pytest.mark.parametrize("H,sq", [(8, 1), (32, 1)])
def test_table_for_almost_2_31_tokens(H, sq):
    """Two sequences in the largest pages and the widest table: sizes whose
    plan does not fit 32 bits, for few sequences."""
    c = Case(515, 2, sq, H, 1, 64, 65536, [3000, 500], extra=0)
    ref = c.reference()
    d = c.device()
    d[5] = torch.full((2, 32000), -1, dtype=torch.int32, device="cuda")
    d[5][:, :1] = torch.from_numpy(c.table)
    check(c, *run(c, d), ref)


def test_many_sequences():
    lens = np.random.default_rng(1).integers(0, 90, 700)
    c = Case(520, 700, 1, 4, 2, 64, 32, lens)
    check(c, *run(c))


@pytest.mark.parametrize("B", [90, 420])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G,sq", [(8, 2, 1), (32, 2, 1), (64, 2, 1), (8, 2, 8), (24, 2, 6)], ids=str)
def test_many_units_of_unlike_lengths(H, G, sq, D, B):
    """Many units to a CTA, of one tile to several, whole and cut: lengths of
    zero, of whole tiles, and a few long ones among short ones."""
    rng = np.random.default_rng(540 + H + sq + D + B)
    lens = rng.choice([0, 1, 127, 128, 129, 256, 300, 900], B, p=[.1, .1, .1, .2, .15, .15, .15, .05])
    lens[::7] = rng.integers(0, 700, lens[::7].size)
    c = Case(540 + H + sq + D + B, B, sq, H, G, D, 64, lens)
    check(c, *run(c))


def test_lse_is_optional():
    c = Case(530, 2, 1, 8, 2, 128, 64, [200, 77])
    ref = c.reference()
    out, _ = run(c, with_lse=False)
    check(c, out, ref[1], ref)


@pytest.mark.parametrize("page", [16, 64, 128])
def test_entries_outside_the_pool_read_as_zeros(page):
    c = Case(540 + page, 2, 1, 16, 4, 128, page, [300, 200])
    c.table[0, 1] = c.codes[0].shape[0] + 7
    c.table[1, 0] = -1
    c.table[0, 0] = np.iinfo(np.int32).min
    check(c, *run(c))


def test_scales_of_unlike_size():
    """Neighbouring blocks' scales up to 2^16 apart, in K within 2^4."""
    c = Case(550, 3, 2, 16, 2, 128, 16, [900, 333, 64])
    rng = np.random.default_rng(3)
    c.scales[0] *= np.exp2(rng.integers(-2, 2, c.scales[0].shape)).astype(np.float32) / 4
    c.scales[1] *= np.exp2(rng.integers(-8, 9, c.scales[1].shape)).astype(np.float32)
    check(c, *run(c))


def test_zero_scales():
    c = Case(560, 2, 1, 8, 2, 64, 16, [200, 100])
    rng = np.random.default_rng(4)
    for s in c.scales:
        s[rng.random(s.shape) < 0.4] = 0
    check(c, *run(c))
    for s in c.scales:
        s[...] = 0
    out, lse = run(c)
    assert (out == 0).all()
    check(c, out, lse)


def test_large_and_tiny_queries():
    """Rows of unlike magnitude in one group, and a zero row; the softmax scale
    brings the scores back to a few units."""
    c = Case(570, 1, 1, 16, 2, 128, 64, [400])
    q = torch.from_numpy(c.q.view(np.int16)).view(torch.bfloat16).float()
    q *= torch.exp2(torch.arange(16).float() - 15).view(1, 1, 16, 1)
    q[0, 0, 3] = 0
    c.q = (q * 2.0 ** 30).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    c.sm = 2.0 ** -30 / math.sqrt(128)
    check(c, *run(c))


def test_one_key_above_the_rest_and_a_long_tail():
    """The first key holds half of the weight, 40000 equal keys the other
    half: what each of them adds is 2^-17 of the first."""
    T, D, page = 40000, 128, 64
    c = Case(580, 1, 1, 2, 2, D, page, [T])
    for x in range(2):
        c.scales[x][...] = 1.0
    c.codes[0][...] = 0
    c.codes[1] &= 0x7F          # positive values: the tail does not average out
    p0 = int(c.table[0, 0])
    c.codes[0][p0, :, 0, 0] = model.nearest_codes(np.array(16.0))
    c.q[...] = 0
    c.q[..., 0] = int(torch.tensor([1.0]).to(torch.bfloat16).view(torch.int16))
    c.sm = math.log(T) / 16
    check(c, *run(c))


def test_positive_and_negative_softmax_scales():
    for sm in (0.0, -0.09, 1.5):
        c = Case(590, 2, 2, 8, 2, 64, 32, [150, 40])
        c.sm = sm
        out, lse = run(c)
        ref = c.reference()
        if sm == 1.5:       # scores of up to ~60: their error grows with them
            assert np.abs(out - ref[0]).max() <= 2.0 ** -6 * c.vmax.max()
        else:
            check(c, out, lse, ref)


def test_nan_reaches_the_rows_that_see_it_and_no_other():
    B, sq, H, G, D, page = 2, 4, 8, 2, 128, 16
    base = Case(600, B, sq, H, G, D, page, [200, 90])
    ref = run(base)
    for which in (0, 1):                    # K, V
        for pos in (50, 197, 198, 199):     # visible to all rows; the new tokens 1, 2, 3
            c = Case(600, B, sq, H, G, D, page, [200, 90])
            c.codes[which][c.table[0, pos // page], 1, pos % page, 7] = 0xFF
            out, lse = run(c)
            sees = np.zeros((B, sq, H), bool)
            sees[0, [s for s in range(sq) if 200 - sq + s >= pos], H // G:] = True
            assert np.isnan(out[sees]).any(axis=-1).all(), (which, pos)
            assert np.array_equal(out[~sees], ref[0][~sees]) and np.array_equal(lse[~sees], ref[1][~sees])


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_non_finite_queries_poison_their_own_row(bad):
    base = Case(610, 1, 2, 8, 2, 64, 16, [100])
    ref = run(base)
    c = Case(610, 1, 2, 8, 2, 64, 16, [100])
    c.q[0, 1, 5, 9] = int(torch.tensor([bad]).to(torch.bfloat16).view(torch.int16)) & 0xFFFF
    out, lse = run(c)
    assert np.isnan(out[0, 1, 5]).all() and np.isnan(lse[0, 1, 5])
    keep = np.ones((1, 2, 8), bool)
    keep[0, 1, 5] = False
    assert np.array_equal(out[keep], ref[0][keep]) and np.array_equal(lse[keep], ref[1][keep])


def test_matches_the_contiguous_fp8_cache():
    """The same codes and scales in 64-token pages and in one contiguous cache."""
    B, H, G, D, T = 2, 16, 4, 128, 512
    c = Case(620, B, 1, H, G, D, 64, [T, T])
    dev = c.device()
    out, lse = run(c, dev)
    t = dev[5].long()
    k, v = (x[t].transpose(1, 2).reshape(B, G, T, D).contiguous() for x in dev[1:3])
    ks, vs = (x[t][..., 0].transpose(1, 2).contiguous() for x in dev[3:5])
    o2 = torch.empty(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    l2 = torch.empty(B, 1, H, dtype=torch.float32, device="cuda")
    gq.gqa_decode_fp8(dev[0], k, v, ks, vs, dev[6], c.sm, o2, l2)
    check(c, bf16_to_f64(o2), l2.cpu().numpy().astype(np.float64))
    assert np.abs(out - bf16_to_f64(o2)).max() <= 2.0 ** -7 * np.abs(out).max() + 2.0 ** -10 * c.vmax.max()


def test_two_calls_agree_bit_for_bit():
    c = Case(630, 3, 4, 64, 8, 128, 64, [3000, 700, 45])
    dev = c.device()
    a, b = run(c, dev), run(c, dev)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_streams_graphs_and_dirty_workspaces():
    """Two graphs with their own memory, replayed at once on two streams with
    new lengths and queries; and a caller's workspace full of canary bytes."""
    cases = [Case(640 + i, 3, 1, 32, 8, 128, 64, [2000, 1500 - 99 * i, 40]) for i in range(2)]
    devs = [c.device() for c in cases]
    refs = [run(c, d) for c, d in zip(cases, devs)]
    outs, graphs = [], []
    for c, d in zip(cases, devs):
        B, sq, H, G, D, page = c.shape
        o = torch.zeros(B, sq, H, D, dtype=torch.bfloat16, device="cuda")
        l = torch.zeros(B, sq, H, dtype=torch.float32, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gq.gqa_decode_paged_fp8(*d, c.sm, o, l)
        outs.append((o, l))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        for o, l in outs:
            o.zero_()
            l.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for (o, l), ref in zip(outs, refs):
            assert np.array_equal(bf16_to_f64(o), ref[0])
            assert np.array_equal(l.cpu().numpy(), ref[1].astype(np.float32))
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    n = gq.gqa_decode_paged_fp8_workspace_bytes(3, 1, 32, 8, 128, 64, cases[1].most)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    got = run(cases[1], devs[1], workspace=ws)
    assert np.array_equal(got[0], refs[1][0])
    short = torch.empty(n - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(gq.GQADecodeError) as e:
        run(cases[1], devs[1], workspace=short)
    assert e.value.status == gq.GQA_ERR_WORKSPACE


def test_kept_workspaces_grow_and_are_released():
    """Calls on one stream share a workspace that grows; releasing it, and calls
    with streams as arguments, change no result."""
    small = Case(645, 1, 1, 8, 2, 64, 16, [40])
    large = Case(646, 4, 4, 64, 8, 128, 64, [3000, 2500, 17, 900])
    devs = [small.device(), large.device()]
    refs = [run(small, devs[0]), run(large, devs[1])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for rep in range(3):
        gq.gqa_decode_release_workspace()
        for c, d, ref in zip((small, large, small), (devs[0], devs[1], devs[0]), (refs[0], refs[1], refs[0])):
            for kw in ({}, dict(stream=side), dict(stream=side.cuda_stream)):
                got = run(c, d, **kw)
                assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
        with torch.cuda.stream(side):
            got = run(large, devs[1])
        assert np.array_equal(got[0], refs[1][0])


def test_replay_with_new_lengths_and_pages():
    c = Case(650, 2, 2, 16, 2, 64, 16, [400, 400])
    d = c.device()
    B, sq, H, G, D, page = c.shape
    o = torch.zeros(B, sq, H, D, dtype=torch.bfloat16, device="cuda")
    l = torch.zeros(B, sq, H, dtype=torch.float32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gq.gqa_decode_paged_fp8(*d, c.sm, o, l)
    for lens in ([400, 400], [1, 399], [0, 64], [130, 0], [400, 16]):
        c.lens = np.array(lens, np.int32)
        c.table = c.table[::-1].copy()
        d[6].copy_(torch.from_numpy(c.lens))
        d[5].copy_(torch.from_numpy(c.table))
        g.replay()
        torch.cuda.synchronize()
        check(c, bf16_to_f64(o), l.cpu().numpy().astype(np.float64), what=str(lens))


def test_an_expired_wait_is_reported_and_the_context_survives():
    c = Case(660, 2, 1, 16, 2, 128, 64, [2000, 900])
    d = c.device()
    ref = run(c, d)
    B, sq, H, G, D, page = c.shape
    o = torch.empty(B, sq, H, D, dtype=torch.bfloat16, device="cuda")
    with env(GQA_DECODE_DEBUG_TIMEOUT_MS=200, GQA_DECODE_DEBUG_SKIP_TILE=0):
        gq.gqa_decode_paged_fp8(*d, c.sm, o)
        assert gq.gqa_decode_check_error() == gq.GQA_ERR_DEVICE_TIMEOUT
    for _ in range(2):
        got = run(c, d)
        assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])


def test_host_threads_with_a_stream_each():
    """Four threads, attention and page management at once, each on its own
    stream and so with its own kept workspace, results as without the others."""
    import threading
    cases = [Case(670 + i, 3, 1 + i, 16, 2, 64 if i % 2 else 128, 32, [1500 - 300 * i, 77, 640]) for i in range(4)]
    refs, wrong = [run(c) for c in cases], []

    def work(i):
        try:
            c = cases[i]
            B, sq, H, G, D, page = c.shape
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                d = c.device()
                o = [torch.empty(B, sq, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
                lse = torch.empty(B, sq, H, device="cuda")
                table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
                refs_, counts = torch.zeros(200, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
                done = torch.ones(B, dtype=torch.bool, device="cuda")
                for x in o:
                    lens = torch.full((B,), 16 * (5 + i), dtype=torch.int32, device="cuda")
                    gq.gqa_pages_reserve(table, lens, refs_, 16, counts)
                    gq.gqa_decode_paged_fp8(*d, c.sm, x, lse)
                    gq.gqa_pages_free(done, table, lens, refs_)
                stream.synchronize()
                same = all(np.array_equal(bf16_to_f64(x), refs[i][0]) for x in o)
                if not (same and counts.tolist() == [B * (5 + i), 200] and not bool(refs_.any()) and bool((table == -1).all())):
                    wrong.append(i)
        except Exception as e:                    # a thread's failure is the test's
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong and not any(t.is_alive() for t in threads), wrong


@pytest.mark.parametrize("H,G,sq,D", [(64, 2, 1, 128), (8, 1, 4, 64), (32, 2, 1, 128)], ids=str)
def test_an_expired_wait_with_more_rows_and_units(H, G, sq, D):
    """16 and 32 rows, CTAs with parts of several units: the call ends, says so,
    and leaves a workspace that the next calls use as if nothing had been."""
    c = Case(661, 8, sq, H, G, D, 64, [3000, 1000, 129, 2500, 1, 700, 2048, 1500])
    d = c.device()
    n = gq.gqa_decode_paged_fp8_workspace_bytes(8, sq, H, G, D, 64, c.most)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ref = run(c, d, workspace=ws)
    check(c, *ref)
    o = torch.empty(c.shape[0], sq, H, D, dtype=torch.bfloat16, device="cuda")
    for tile in (0, 3):
        with env(GQA_DECODE_DEBUG_TIMEOUT_MS=200, GQA_DECODE_DEBUG_SKIP_TILE=tile):
            gq.gqa_decode_paged_fp8(*d, c.sm, o, workspace=ws)
            assert gq.gqa_decode_check_error() == gq.GQA_ERR_DEVICE_TIMEOUT
        for _ in range(2):
            got = run(c, d, workspace=ws)
            assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])


def test_page_pool_past_2_31_codes():
    """A pool of more than 2^31 codes: the last pages' bytes and scales."""
    G, D, page = 8, 128, 64
    num = (1 << 31) // (G * D * page) + 5
    c = Case(670, 1, 1, 16, G, D, page, [600])
    dev = c.device()
    n = c.codes[0].shape[0]
    for i, shape in ((1, (num, G, page, D)), (2, (num, G, page, D))):
        big = torch.full(shape, model.NAN_CODE, dtype=torch.uint8, device="cuda")
        big[num - n:] = dev[i]
        dev[i] = big
    for i in (3, 4):
        big = torch.full((num, G, 1), float("nan"), device="cuda")
        big[num - n:] = dev[i]
        dev[i] = big
    dev[5] = torch.where(dev[5] >= 0, dev[5] + (num - n), dev[5])
    check(c, *run(c, dev))


@pytest.mark.parametrize("H,G,sq", [(32, 8, 1), (64, 2, 1), (8, 2, 9)], ids=str)
@pytest.mark.parametrize("empty", [1, 3])
def test_an_empty_sequence_before_many_units(empty, H, G, sq):
    """A freed row among 16, tables wider than the lengths: the CTAs without a
    share do nothing, and so repeated calls agree bit for bit."""
    lens = [1024] * 16
    lens[empty] = 0
    lens[9:12] = [700, 1, 2000]
    c = Case(700 + empty + sq, 16, sq, H, G, 128, 64, lens, most=64)
    dev = c.device()
    first = run(c, dev)
    check(c, *first)
    for rep in range(30):
        again = run(c, dev)
        assert np.array_equal(again[0], first[0]) and np.array_equal(again[1], first[1]), rep


@pytest.mark.parametrize("H,G", [(8, 8), (64, 4)], ids=str)
def test_an_expired_wait_writes_no_row_that_is_not_its_own(H, G):
    """A CTA whose wait expires in its first unit ends its other units without
    their queries: what shared memory held for them, rows of an earlier and
    larger call, is no place to write to."""
    B, T, D = 320 // G, 1024, 64
    large = Case(720, 3 * B, 1, H, G, D, 64, [130] * (3 * B))
    small = Case(721, B, 1, H, G, D, 64, [T] * B)
    ds, dl = small.device(), large.device()
    buf = torch.zeros(3 * B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(3 * B, 1, H, device="cuda")
    gq.gqa_decode_paged_fp8(*ds, small.sm, buf[:B], lse[:B])
    torch.cuda.synchronize()
    ref = buf[:B].clone()
    for rep in range(3):
        gq.gqa_decode_paged_fp8(*dl, large.sm, buf, lse)
        torch.cuda.synchronize()
        buf.view(torch.int16).fill_(BF_CANARY)
        lse.view(torch.int32).fill_(F32_CANARY)
        with env(GQA_DECODE_DEBUG_TIMEOUT_MS=200, GQA_DECODE_DEBUG_SKIP_TILE=0):
            gq.gqa_decode_paged_fp8(*ds, small.sm, buf[:B], lse[:B])
            assert gq.gqa_decode_check_error() == gq.GQA_ERR_DEVICE_TIMEOUT
        assert bool((buf[B:].view(torch.int16) == BF_CANARY).all()) and bool((lse[B:].view(torch.int32) == F32_CANARY).all())
    gq.gqa_decode_paged_fp8(*ds, small.sm, buf[:B], lse[:B])
    assert torch.equal(buf[:B], ref)
    assert gq.gqa_decode_check_error() == gq.GQA_OK


# Small weights. A key's weight, p times its block's V scale, is rounded to fp16
# with the largest such product of the unit at 2^11 or a little above: by at
# most 2^-11 of itself, or 2^-25, which is 2^-35 448 S a key, with S the largest
# |v_scale| of the unit's blocks and the row's largest p at 1 or above:
#   |out - exact| <= 2^-8 |out| + 2^-11 sum(p |v|) / l + n 2^-35 448 S / l
# and the scores' error, 2^-13 in natural units, on numerator and sum.

def weighted(pool_k, pool_v, pages, q, sm):
    """Exact out of one row over `pages` (repeats allowed) of values [num, page, D];
    also sum(p |v|) / l, and l with the largest p at 1."""
    count = np.bincount(pages, minlength=len(pool_k)).astype(np.float64)
    x = pool_k @ q * sm
    m = x[count > 0].max()
    w = np.exp(x - m) * count[:, None]
    l = w.sum()
    return (w.reshape(-1) @ pool_v.reshape(-1, pool_v.shape[-1]) / l,
            w.reshape(-1) @ np.abs(pool_v).reshape(-1, pool_v.shape[-1]) / l, l)


def run_weighted(codes, scales, pages, q, sm, H=2, page=64, B=1):
    """B equal sequences over `pages`, one KV head, H equal query rows; what comes
    out and how far it may be off."""
    D, T = codes[0].shape[-1], len(pages) * page
    d = [torch.from_numpy(x[:, None]).cuda() for x in (*codes, *scales)]
    qs = torch.from_numpy(q).to(torch.bfloat16)
    assert np.array_equal(qs.double().numpy(), q)
    out = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    gq.gqa_decode_paged_fp8(qs.cuda().expand(B, 1, H, D).contiguous(), *d,
                            torch.from_numpy(np.asarray(pages, np.int32)).cuda().expand(B, -1).contiguous(),
                            torch.full((B,), T, dtype=torch.int32, device="cuda"), sm, out)
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    k, v = (model.page_values(c[:, None], s[:, None])[:, 0] for c, s in zip(codes, scales))
    want, spread, l = weighted(k, v, pages, q, sm)
    S = np.abs(scales[1][np.unique(pages)]).max()
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + T * 2.0 ** -35 * 448 * S / l
    return out.double().cpu().numpy()[:, 0], want, bound


@pytest.mark.parametrize("T,rest", [(1 << 17, 0.5), (1 << 17, 0.1), (1 << 17, 0.01), (1 << 20, 0.1), (1 << 20, 0.01)])
@pytest.mark.parametrize("H", [2, 12, 32])
@pytest.mark.parametrize("B", [1, 304])
def test_a_sink_and_a_long_tail(B, H, T, rest):
    """A first key with most of the weight and a value of zero, the rest of the
    weight spread over a long context whose values have one sign: split over the
    SMs, each part with its own reference, and with whole sequences to an SM."""
    rng = np.random.default_rng(T % 977 + H)
    page, D, n = 64, 64, 40
    codes = [np.zeros((n, page, D), np.uint8), model.nearest_codes(rng.uniform(40, 200, (n, page, D)))]
    codes[0][..., 0] = model.nearest_codes(rng.uniform(-1, 1, (n, page)))
    codes[0][0, 0, 0], codes[1][0, 0] = model.nearest_codes(np.array(16.0)), 0
    scales = [np.ones((n, 1), np.float32), np.full((n, 1), 0.75 / 64, np.float32)]
    pages = np.concatenate([[0], 1 + np.arange(T // page - 1) % (n - 1)])
    q = np.zeros(D)
    q[0] = 1.0
    got, want, bound = run_weighted(codes, scales, pages, q, math.log(T / rest) / 16, H, B=B)
    assert (np.abs(got - want) <= bound).all(), (np.abs(got / want - 1).max(), (np.abs(got - want) / bound).max())


@pytest.mark.parametrize("ratio", [16, 20, 24, 26])
def test_values_far_below_the_largest_scale(ratio):
    """Equal weights; the values of a page with a large scale are zeros, those of
    the others 2^-ratio of its scale."""
    rng = np.random.default_rng(ratio)
    page, D, n = 64, 128, 12
    codes = [np.zeros((n, page, D), np.uint8), model.nearest_codes(rng.uniform(100, 448, (n, page, D)))]
    scales = [np.ones((n, 1), np.float32), np.exp2(-ratio + rng.uniform(-0.5, 0.5, (n, 1))).astype(np.float32)]
    codes[1][0], scales[1][0] = 0, 1.0
    for pages in (np.arange(n), np.arange(n)[::-1], np.concatenate([np.zeros(1, int), 1 + np.arange(400) % (n - 1)])):
        got, want, bound = run_weighted(codes, scales, pages, np.zeros(D), 1.0)
        assert (np.abs(got - want) <= bound).all(), (np.abs(got / want - 1).max(), (np.abs(got - want) / bound).max())


@pytest.mark.parametrize("e", [-126, -110, -90, -75, -61, 59])
@pytest.mark.parametrize("D,H", [(64, 2), (128, 12), (128, 32)])
def test_the_smallest_and_the_largest_scales(D, H, e):
    """V scales from the smallest that the append makes, 2^-126, to 2^60: in one
    tile, in both groups' tiles, and in parts of several CTAs."""
    rng = np.random.default_rng(e + 200 + D)
    page, n = 64, 20
    codes = [model.nearest_codes(rng.standard_normal((n, page, D))), model.nearest_codes(rng.uniform(100, 448, (n, page, D)))]
    scales = [np.ones((n, 1), np.float32) / 8, np.full((n, 1), 2.0 ** e, np.float32)]
    for count in (1, 5, n, 60):
        got, want, bound = run_weighted(codes, scales, np.arange(count) % n, np.round(rng.standard_normal(D) * 2) / 2,
                                        1 / math.sqrt(D), H)
        assert (np.abs(got - want) <= bound).all(), (count, np.abs(got / want - 1).max())
