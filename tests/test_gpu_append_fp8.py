"""The quantising append on the GPU: codes and scales bit for bit as the
model's, and nothing else in the pool touched."""
import numpy as np
import pytest
import torch

import grouped_query_decode_gb300 as gq
import oracle
import paged_fp8_model as model

pytestmark = pytest.mark.gpu


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


class Pool:
    def __init__(self, seed, B, G, D, page, most, extra=3):
        self.rng = np.random.default_rng(seed)
        num = B * most + extra
        self.codes = [self.rng.integers(0, 256, (num, G, page, D)).astype(np.uint8) for _ in range(2)]
        for c in self.codes:
            c[(c & 127) == 127] ^= 1          # NaN codes only where a test puts them
        self.scales = [np.exp2(self.rng.integers(-8, -3, (num, G, model.blocks_of(page)))).astype(np.float32)
                       for _ in range(2)]
        self.table = self.rng.permutation(num)[:B * most].reshape(B, most).astype(np.int32)
        self.dev = [torch.from_numpy(x.copy()).cuda() for x in (*self.codes, *self.scales, self.table)]

    def tokens(self, B, sq, G, D, sizes=(-3, 4)):
        x = self.rng.standard_normal((B, sq, G, D)) * np.exp2(self.rng.integers(*sizes, (B, sq, G, 1)))
        return bf16(x)

    def append(self, k, v, lens):
        lens = np.asarray(lens, np.int32)
        gq.gqa_append_paged_fp8(k.cuda(), v.cuda(), *self.dev, torch.from_numpy(lens).cuda())
        torch.cuda.synchronize()
        for c, s, x in zip(self.codes, self.scales, (k, v)):
            with np.errstate(invalid="ignore"):
                model.append(c, s, x.double().numpy(), self.table, lens)

    def check(self, what=""):
        for i, (c, s) in enumerate(zip(self.codes, self.scales)):
            got, gs = self.dev[i].cpu().numpy(), self.dev[2 + i].cpu().numpy()
            assert np.array_equal(gs.view(np.uint32), s.view(np.uint32)), (what, i, "scales")
            nan = (c & 127) == 127
            assert np.array_equal((got & 127) == 127, nan), (what, i, "NaN codes")
            # a code of zero keeps or loses its sign with the value that underflows
            zero = (c & 127) == 0
            assert np.array_equal(got[~nan & ~zero], c[~nan & ~zero]), (what, i, "codes")
            assert ((got & 127)[zero] == 0).all(), (what, i, "zeros")


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sq", [1, 2, 5, 8, 9, 17, 64, 100])
def test_matches_the_model(sq, D, page):
    B, G = 5, 3
    most = -(-300 // page)
    p = Pool(10 + sq + D + page, B, G, D, page, most)
    lens = [sq, sq + 1, 128 + sq, max(1, sq // 2), min(300, 190 + sq)]
    p.append(p.tokens(B, sq, G, D), p.tokens(B, sq, G, D), lens)
    p.check()


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64)])
def test_token_by_token(D, page):
    """Sixty decode steps: scales that grow, requantised codes, new pages."""
    B, G = 3, 2
    p = Pool(50 + D, B, G, D, page, -(-100 // page))
    for t in range(1, 61):
        size = (-6 + t // 12, -4 + t // 12)
        p.append(p.tokens(B, 1, G, D, size), p.tokens(B, 1, G, D, size), [t, t + 7, t + 39])
        if t % 10 == 0:
            p.check(f"token {t}")
    p.check()


def test_lengths_below_the_new_tokens_zero_and_clamped():
    p = Pool(60, 5, 2, 64, 16, 4)
    p.append(p.tokens(5, 6, 2, 64), p.tokens(5, 6, 2, 64), [0, -4, 3, 1000, 64])
    p.check()


def test_entries_outside_the_pool_are_skipped():
    p = Pool(70, 3, 2, 128, 16, 6)
    num = p.codes[0].shape[0]
    p.table[0, 1], p.table[1, 3], p.table[2, 0] = -1, num, np.iinfo(np.int32).min
    p.dev[4].copy_(torch.from_numpy(p.table))
    p.append(p.tokens(3, 40, 2, 128), p.tokens(3, 40, 2, 128), [45, 90, 40])
    p.check()


def test_ties_zeros_subnormals_and_the_largest_values():
    B, G, D, page = 4, 1, 64, 16
    p = Pool(80, B, G, D, page, 2)
    x = np.zeros((B, 4, G, D), np.float32)
    x[0, 0, 0, 0] = 448.0                                        # scale 2 (31/16 * 2^8 = 496 below)
    x[0, 1, 0] = np.ldexp(1 + (2 * np.arange(D) % 16 + 1) / 16, np.arange(D) % 15 - 6)
    x[0, 2, 0] = (np.arange(D) + 0.5) * 2.0 ** -10               # subnormal codes and their ties
    x[1, 3, 0, 5] = 3.3e38                                       # beside zeros
    x[2] = 1e-39                                                 # below every scale but 2^-126
    x[3, :, 0] = -np.abs(p.rng.standard_normal((4, D)))
    p.append(bf16(x), bf16(-x), [4, 4, 4, 20])
    p.check()
    assert p.scales[0][p.table[0, 0], 0, 0] == 2.0


def test_zero_blocks_then_values():
    """A block of zeros has scale 0 and takes any scale later."""
    p = Pool(90, 1, 2, 64, 16, 1)
    z = bf16(np.zeros((1, 1, 2, 64)))
    for t in range(1, 4):
        p.append(z, z, [t])
    assert (p.scales[0][p.table[0, 0]] == 0).all()
    p.append(p.tokens(1, 1, 2, 64), z, [4])
    p.append(z, p.tokens(1, 1, 2, 64), [5])
    p.check()


def test_nan_and_infinities_become_nan_codes_and_leave_the_scale():
    p = Pool(100, 2, 2, 128, 16, 2)
    k = p.tokens(2, 3, 2, 128)
    k[0, 1, 0, 5], k[0, 1, 0, 6], k[1, 2, 1, 0] = float("nan"), float("inf"), float("-inf")
    k[1, 0, 0] = float("inf")
    p.append(k, p.tokens(2, 3, 2, 128), [3, 20])
    p.check()
    assert np.isfinite(p.scales[0]).all()
    assert ((p.codes[0][p.table[0, 0], 0, 1, 5:7] & 127) == 127).all()


def test_scales_that_are_no_powers_of_two():
    """A pool quantised elsewhere (scale = max/448): kept while it fits."""
    p = Pool(110, 4, 2, 64, 64, 2)
    for i, s in enumerate(p.scales):
        s *= (1 + 0.9 * p.rng.random(s.shape)).astype(np.float32)
        p.dev[2 + i].copy_(torch.from_numpy(s))
    sizes = (-8, 3)
    p.append(p.tokens(4, 2, 2, 64, sizes), p.tokens(4, 2, 2, 64, sizes), [30, 70, 90, 128])
    # x / scale rounds in fp32 before e4m3: one code apart at most, where x is
    # within fp32's rounding of a tie.
    for i, (c, s) in enumerate(zip(p.codes, p.scales)):
        got = p.dev[i].cpu().numpy()
        assert np.array_equal(p.dev[2 + i].cpu().numpy(), s)
        off = got != c
        a, b = oracle.e4m3_to_f64(got[off]), oracle.e4m3_to_f64(c[off])
        assert off.mean() < 1e-3 and (np.abs(a - b) <= np.maximum(np.abs(b) / 8, 2.0 ** -9)).all()


def test_a_held_scale_that_is_not_positive_counts_as_zero():
    p = Pool(111, 4, 2, 64, 64, 2)
    for i, s in enumerate(p.scales):
        odd = torch.from_numpy(s.copy())
        odd[p.table[1, 0]], odd[p.table[2, 0]], odd[p.table[3, 0]] = -0.5, float("nan"), -0.0
        p.dev[2 + i].copy_(odd)
        s[p.table[1:, 0]] = 0.0
    p.append(p.tokens(4, 3, 2, 64), p.tokens(4, 3, 2, 64), [10, 10, 33, 64])
    p.check()


@pytest.mark.parametrize("sq", [1, 20, 200])
def test_positions_up_to_almost_2_31(sq):
    """The last tokens of the widest table in the largest pages: as the last
    tokens of a table of one page."""
    page, most = 65536, 32000
    x = [bf16(np.random.default_rng(112 + i).standard_normal((1, sq, 1, 64))).cuda() for i in range(2)]
    got = []
    for n in (1, most):
        pool = [torch.zeros(2, 1, page, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scale = [torch.full((2, 1, 1024), 2.0 ** -9, device="cuda") for _ in range(2)]
        table = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
        table[0, -1] = 1
        lens = torch.tensor([n * page - 5], dtype=torch.int32, device="cuda")
        gq.gqa_append_paged_fp8(*x, *pool, *scale, table, lens)
        got.append(pool + scale)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert all(bool(p[1, 0, page - 5 - sq:page - 5].any(1).all()) and not bool(p[1, 0, page - 5:].any()) for p in got[1][:2])


def test_append_then_attend_serves_the_values(monkeypatch):
    """A prompt, then tokens one by one, through the public calls alone: the
    attention is the oracle's over the values the model quantised."""
    import math
    B, H, G, D, page, most = 2, 8, 2, 128, 16, 6
    p = Pool(120, B, G, D, page, most)
    rng = np.random.default_rng(6)
    q_all = bf16(rng.standard_normal((6, B, 5, H, D)))
    lens = np.array([40, 23], np.int32)
    sm = 1 / math.sqrt(D)
    for step in range(4):
        sq = 5 if step == 0 else 1
        lens = lens + (0 if step == 0 else 1)
        p.append(p.tokens(B, 40 if step == 0 else 1, G, D, (-1, 2)), p.tokens(B, 40 if step == 0 else 1, G, D, (-1, 2)),
                 lens)
        q = q_all[step, :, :sq].contiguous()
        out = torch.empty(B, sq, H, D, dtype=torch.bfloat16, device="cuda")
        gq.gqa_decode_paged_fp8(q.cuda(), *p.dev, torch.from_numpy(lens.astype(np.int32)).cuda(), sm, out)
        torch.cuda.synchronize()
        k, v = (model.logical(model.page_values(c, s), p.table, lens, most * page)
                for c, s in zip(p.codes, p.scales))
        ref, _ = oracle.get().gqa_decode_kv(q.view(torch.int16).numpy().view(np.uint16), k, v, lens, sm)
        vmax = np.nanmax(np.abs(v))
        assert np.abs(out.float().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -10 * vmax


NOT_FINITE = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("sq", [1, 5, 20])
@pytest.mark.parametrize("held", ["none", "zeros", "not positive"])
@pytest.mark.parametrize("beside", ["alone", "zeros"])
def test_nan_and_infinities_in_blocks_without_a_scale(beside, held, sq):
    """No finite element above 0 and no scale held: the block's scale is 0, and
    NaN and infinities are NaN codes all the same, so attention says NaN."""
    B, G, D, page = 3, 2, 64, 64
    p = Pool(130 + sq, B, G, D, page, 1)
    kept = 0 if held == "none" else 7
    if kept:
        for i, s in enumerate(p.scales):
            odd = torch.from_numpy(s.copy())
            odd[p.table[:, 0]] = torch.tensor(0.0 if held == "zeros" else -0.5)
            p.dev[2 + i].copy_(odd)
            s[p.table[:, 0]] = 0.0
    k, v = torch.zeros(B, sq, G, D), torch.zeros(B, sq, G, D)
    for b in range(B):                              # sequence b: NaN, inf or -inf, in K head 0 and V head 1
        if beside == "alone":
            k[b, :, 0], v[b, :, 1] = NOT_FINITE[b], NOT_FINITE[b]
        else:
            k[b, sq // 2, 0, 3 + b], v[b, sq - 1, 1, 60 - b] = NOT_FINITE[b], NOT_FINITE[b]
    lens = [kept + sq] * B
    p.append(k.to(torch.bfloat16), v.to(torch.bfloat16), lens)
    p.check()
    at = p.table[:, 0]
    want = ~np.isfinite(k.numpy().transpose(0, 2, 1, 3))
    assert np.array_equal((p.dev[0].cpu().numpy()[at, :, kept:kept + sq] & 127) == 127, want)
    out = torch.zeros(B, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(B, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    gq.gqa_decode_paged_fp8(q, *p.dev, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1.0, out)
    assert bool(out[:, :, 0].isnan().all())                              # a NaN score: the whole row
    assert torch.equal(out[:, 0, 1].isnan().cpu(), torch.from_numpy(~np.isfinite(v.numpy()[:, :, 1])).any(1))
