"""Rotary positions (gqa_rope) and the append to bf16 pages (gqa_append_paged)
against float64 models: layouts, parts of a head, scalings, far positions,
strides, rows and pages that must stay as they are."""
import math

import pytest
import torch

import grouped_query_decode_gb300 as gq
import ragged_model as model

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
SCALINGS = {
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, scaling="linear", factor=4.0),
    "base": dict(base=10000.0, scaling="base", factor=8.0),
    "bands": dict(base=500000.0, scaling="bands", factor=8.0, original=8192.0, low=1.0, high=4.0),
    "yarn": dict(base=10000.0, scaling="yarn", factor=16.0, original=4096.0, low=1.0, high=32.0),
}


def make(D, dims, interleaved, scaling):
    rope = gq.gqa_rope_init(D, dims=dims, interleaved=interleaved, **SCALINGS[scaling])
    f, gain = model.frequencies(dims, **SCALINGS[scaling])
    return rope, f, gain


def close(got, want_size, what=""):
    want, size = want_size
    off = (got.double().cpu() - want).abs() - model.rotate_bound(want, size)
    assert (off <= 0).all(), f"{what}: off by {off.max():.3e} more than the bound"


def rows(N, heads, D, seed, dtype=BF):
    return torch.randn(N, heads, D, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("D,dims,interleaved", [
    (128, 128, False), (128, 128, True), (64, 64, False), (64, 64, True), (128, 64, False), (128, 64, True),
    (128, 32, False), (64, 16, False), (64, 2, False), (64, 2, True), (128, 6, False), (128, 6, True),
    (128, 126, False), (128, 126, True), (64, 24, False), (64, 50, True)])
def test_layouts_and_scalings(D, dims, interleaved, scaling):
    rope, f, gain = make(D, dims, interleaved, scaling)
    q, k = rows(37, 6, D, 1), rows(37, 2, D, 2)
    t = torch.randint(0, 1 << 17, (37,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    t[0] = 0
    q_out, k_out = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    gq.gqa_rope(rope, q.cuda(), k.cuda(), t.cuda(), q_out, k_out)
    close(q_out, model.rotate(q, t, f, gain, interleaved), "q")
    close(k_out, model.rotate(k, t, f, gain, interleaved), "k")
    assert torch.equal(q_out.cpu()[..., dims:], q[..., dims:])


@pytest.mark.parametrize("N,H,G,D", [(1, 1, 1, 64), (1, 32, 8, 128), (2, 5, 5, 128), (3000, 32, 8, 128),
                                     (9733, 3, 1, 64), (25000, 8, 2, 64), (700, 128, 1, 128)])
def test_sizes(N, H, G, D):
    """One token to more tokens than all CTAs take at eight a time."""
    rope, f, gain = make(D, D, False, "none")
    q, k = rows(N, H, D, 4), rows(N, G, D, 5)
    t = torch.arange(N, dtype=torch.int32)
    q_out, k_out = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    gq.gqa_rope(rope, q.cuda(), k.cuda(), t.cuda(), q_out, k_out)
    close(q_out, model.rotate(q, t, f, gain))
    close(k_out, model.rotate(k, t, f, gain))


def test_far_and_negative_positions():
    """Angles stay exact to 2^31 positions (a product in fp32 would be off by whole turns)."""
    rope, f, gain = make(64, 64, False, "none")
    t = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31), -12345], dtype=torch.int32)
    q = rows(len(t), 4, 64, 6)
    out = torch.empty_like(q).cuda()
    gq.gqa_rope(rope, q.cuda(), None, t.cuda(), out, None)
    # The model's own product t * f is off by 2^31 * 2^-53 radians at most.
    close(out, model.rotate(q, t, f, gain))


def test_one_of_both_in_place_strided_and_inverse():
    rope, f, gain = make(128, 128, True, "yarn")
    N, H, G = 65, 4, 2
    x = rows(N, H + 2 * G, 128, 7)
    t = torch.randint(0, 9000, (N,), dtype=torch.int32, generator=torch.Generator().manual_seed(8))
    d = x.cuda()
    gq.gqa_rope(rope, d[:, :H], d[:, H:H + G], t.cuda(), d[:, :H], d[:, H:H + G])      # views, in place
    close(d[:, :H], model.rotate(x[:, :H], t, f, gain, True))
    close(d[:, H:H + G], model.rotate(x[:, H:H + G], t, f, gain, True))
    assert torch.equal(d[:, H + G:].cpu(), x[:, H + G:])                               # values
    k = torch.empty(N, G, 128, dtype=BF, device="cuda")
    gq.gqa_rope(rope, None, x.cuda()[:, H:H + G], t.cuda(), None, k)
    assert torch.equal(k, d[:, H:H + G])
    back = torch.empty_like(k)
    gq.gqa_rope(rope, None, k, t.cuda(), None, back, inverse=True)
    close(back, model.rotate(k.cpu(), t, f, gain, True, inverse=True))


def test_inverse_is_the_gradient():
    """y = R x, so dL/dx = R^T dL/dy: against differences of the model along random directions."""
    rope, f, gain = make(64, 32, False, "yarn")
    x, dy, e = (rows(9, 2, 64, s) for s in (11, 12, 13))
    t = torch.arange(9, dtype=torch.int32) * 77
    dx = torch.empty_like(x).cuda()
    gq.gqa_rope(rope, dy.cuda(), None, t.cuda(), dx, None, inverse=True)
    h = 2.0 ** -10
    y = [model.rotate(x.double() + s * h * e.double(), t, f, gain)[0] for s in (1, -1)]
    slope = ((y[0] - y[1]) / (2 * h) * dy.double()).sum()
    got = (dx.double().cpu() * e.double()).sum()
    bound = (model.rotate_bound(*model.rotate(dy, t, f, gain, inverse=True)) * e.double().abs()).sum()
    assert abs(got - slope) <= bound + 1e-6
    # and every element against the transpose of the model's own matrix
    close(dx, model.rotate(dy, t, f, gain, inverse=True))


def test_nan_and_infinity_stay_in_their_pair():
    rope, f, gain = make(64, 64, False, "none")
    x = rows(4, 2, 64, 14)
    x[1, 0, 3], x[2, 1, 40] = math.nan, math.inf
    out = torch.empty_like(x).cuda()
    gq.gqa_rope(rope, x.cuda(), None, torch.arange(4, dtype=torch.int32).cuda(), out, None)
    bad = ~torch.isfinite(out.cpu())
    want = torch.zeros_like(bad)
    want[1, 0, [3, 35]] = True
    want[2, 1, [8, 40]] = True
    assert torch.equal(bad, want)


# ------------------------------------------------------------------- append

def tables(lens, page, seed, extra=3):
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(T, 0) // page) for T in lens]
    num = sum(need) + extra
    order = torch.randperm(num, generator=g, dtype=torch.int32)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, num


def appended(k_new, v_new, pages, table, news, lens, page, turn):
    """The pages after the append: bf16 copies, and where rotated keys went."""
    kp, vp = pages[0].clone(), pages[1].clone()
    keys = []
    most = table.shape[1] * page
    first = 0
    for b, n in enumerate(news):
        T = min(max(lens[b], 0), most)
        for s in range(n):
            t = T - n + s
            if t >= 0 and 0 <= table[b, t // page] < kp.shape[0]:
                p = int(table[b, t // page])
                keys.append((p, t % page, first + s, t))
                vp[p, :, t % page] = v_new[first + s]
                if not turn:
                    kp[p, :, t % page] = k_new[first + s]
        first += n
    return kp, vp, keys


CASES = [  # H, G, D, page, (new, length) of each sequence, rows behind the last
    (8, 2, 128, 16, [(1, 1), (1, 40), (1, 17), (1, 16)], 0),
    (6, 3, 64, 32, [(50, 50), (0, 10), (7, 100), (33, 65)], 5),
    (4, 4, 128, 64, [(200, 333)], 1),
    (32, 8, 64, 16, [(3, 2), (5, 0), (4, 4), (2, 70)], 3),       # more new tokens than the length
    (5, 1, 128, 256, [(1, 300)] * 9 + [(0, 0)] * 40 + [(300, 513)], 0),
    (2, 1, 64, 16, [(2, 2)] * 1100, 0),                          # more sequences than 32 * 32
]


@pytest.mark.parametrize("rotated", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case, rotated):
    H, G, D, page, seqs, behind = CASES[case]
    news, lens = [n for n, _ in seqs], [T for _, T in seqs]
    N = sum(news) + behind
    table, num = tables(lens, page, 20 + case)
    cu = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    x = rows(N, H + 2 * G, D, 21 + case)
    q, k, v = x[:, :H], x[:, H:H + G], x[:, H + G:]
    pages = [rows(num * G, page, D, 22 + i).view(num, G, page, D) for i in range(2)]
    dx, dp = x.cuda(), [p.cuda() for p in pages]
    q_out = torch.full((N, H, D), 7.0, dtype=BF, device="cuda")
    rope, f, gain = make(D, D // 2, case % 2 == 1, "bands") if rotated else (None, None, None)
    gq.gqa_append_paged(dx[:, H:H + G], dx[:, H + G:], *dp, table.cuda(), cu.cuda(),
                        torch.tensor(lens, dtype=torch.int32).cuda(), rope=rope, q=dx[:, :H], q_out=q_out)
    kp, vp, keys = appended(k, v, pages, table, news, lens, page, rotated)
    assert torch.equal(dp[1].cpu(), vp)
    if rotated:
        got = dp[0].cpu()
        if keys:
            p, slot, row, t = (torch.tensor(z) for z in zip(*keys))
            close(got[p, :, slot], model.rotate(k[row], t, f, gain, case % 2 == 1), "keys")
            kp[p, :, slot] = got[p, :, slot]
        assert torch.equal(got, kp)                              # nothing else was written
        pos = torch.cat([torch.arange(n) + min(max(T, 0), table.shape[1] * page) - n for n, T in seqs] or [torch.zeros(0)])
        m = len(pos)
        close(q_out[:m], model.rotate(q[:m], pos, f, gain, case % 2 == 1), "queries")
    else:
        assert torch.equal(dp[0].cpu(), kp)
        m = sum(news)
        assert torch.equal(q_out[:m].cpu(), q[:m])
    assert (q_out[m:].float() == 7).all()                        # rows behind the last sequence


def test_append_without_queries_and_with_unusable_entries():
    """Entries outside the pool, lengths past the table, cu past the rows."""
    G, D, page = 2, 64, 16
    seqs = [(20, 40), (3, 1000), (4, 9)]
    table = torch.tensor([[2, -1, 5], [0, 9, 1], [7, 1 << 30, -5]], dtype=torch.int32)     # 6 pages
    k, v = rows(27, G, D, 31), rows(27, G, D, 32)
    pages = [torch.zeros(6, G, page, D, dtype=BF) for _ in range(2)]
    dp = [p.cuda() for p in pages]
    cu = torch.tensor([0, 20, 23, 27 + 100], dtype=torch.int32)
    lens = [T for _, T in seqs]
    gq.gqa_append_paged(k.cuda(), v.cuda(), *dp, table.cuda(), cu.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    kp, vp, _ = appended(k, v, pages, table, [20, 3, 4], lens, page, False)
    assert torch.equal(dp[0].cpu(), kp) and torch.equal(dp[1].cpu(), vp)


def test_no_tokens():
    rope, _, _ = make(64, 64, False, "none")
    e = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    gq.gqa_rope(rope, e, e, torch.empty(0, dtype=torch.int32, device="cuda"), e, e)
    p = torch.ones(2, 2, 16, 64, dtype=BF, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    gq.gqa_append_paged(e, e, p, p.clone(), torch.zeros(1, 1, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32))
    assert (p == 1).all()
