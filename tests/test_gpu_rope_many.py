"""Rotation and append of so many tokens that a CTA takes several, to which form a
call changes at 16 and 64 tokens for each SM: sequences that end inside a CTA, a last
CTA with fewer, and halves of a head that do not start on 16 bytes."""
import pytest
import torch

import grouped_query_decode_gb300 as gq
import ragged_model as model

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32
DIMS = [(64, 64, False), (64, 50, False), (64, 50, True), (64, 48, False), (128, 128, False), (128, 100, False),
        (128, 100, True), (128, 6, False)]


def many(more):
    """Tokens: `more` beyond 16 or 64 for each SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return [16 * sms - 1, 16 * sms + more, 64 * sms - 1, 64 * sms + more]


def rows(N, heads, D, seed):
    return torch.randn(N, heads, D, generator=torch.Generator().manual_seed(seed)).to(BF)


def close(got, want, what):
    off = (got.double().cpu() - want[0]).abs() - model.rotate_bound(*want)
    assert (off <= 0).all(), f"{what}: off by {off.max():.3e} more than the bound"


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("D,dims,interleaved", DIMS)
def test_rotation(D, dims, interleaved, which):
    N, H, G = many(3)[which], 3, 2
    rope = gq.gqa_rope_init(D, dims=dims, interleaved=interleaved, base=500000.0)
    f, gain = model.frequencies(dims, 500000.0)
    x = rows(N, H + 2 * G, D, 1)
    t = torch.randint(0, 1 << 17, (N,), generator=torch.Generator().manual_seed(2), dtype=I32)
    d = x.cuda()
    gq.gqa_rope(rope, d[:, :H], d[:, H:H + G], t.cuda(), d[:, :H], d[:, H:H + G])
    close(d[:, :H], model.rotate(x[:, :H], t, f, gain, interleaved), "q")
    close(d[:, H:H + G], model.rotate(x[:, H:H + G], t, f, gain, interleaved), "k")
    assert torch.equal(d[:, H + G:].cpu(), x[:, H + G:])
    assert torch.equal(d[:, :H + G, dims:].cpu(), x[:, :H + G, dims:])


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("D,dims,interleaved", DIMS + [(64, 0, False), (128, 0, False)])
def test_append(D, dims, interleaved, which):
    """dims 0: without rotation. Sequences of 0 to 6 new tokens, one of 200, some with
    more than they are long, some with an entry outside the pool, rows behind the last."""
    H, G, page = 4, 2, 16
    g = torch.Generator().manual_seed(3 + which)
    behind = 5
    left = many(3)[which] - behind - 200
    news = []
    while left > 0:
        n = min(left, int(torch.randint(0, 7, (1,), generator=g)))
        news.append(n)
        left -= n
    news.insert(len(news) // 2, 200)
    B, N = len(news), sum(news) + behind
    n = torch.tensor(news)
    T = n + torch.randint(-2, 40, (B,), generator=g)
    T = T.clamp(min=0)
    need = (T + page - 1) // page
    num, most = int(need.sum()) + 3, int(need.max())
    order = torch.randperm(num, generator=g, dtype=I32)
    table = torch.full((B, most), -1, dtype=I32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + int(need[b])]
        at += int(need[b])
    table[::37, 0] = num                                  # outside the pool
    cu = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).to(I32)
    x = rows(N, H + 2 * G, D, 4)
    pages = [rows(num * G, page, D, 5 + i).view(num, G, page, D) for i in range(2)]
    dx, dp = x.cuda(), [p.cuda() for p in pages]
    q_out = torch.full((N, H, D), 7.0, dtype=BF, device="cuda")
    rope = gq.gqa_rope_init(D, dims=dims, interleaved=interleaved) if dims else None
    f, gain = model.frequencies(dims, 10000.0)
    gq.gqa_append_paged(dx[:, H:H + G], dx[:, H + G:], *dp, table.cuda(), cu.cuda(), T.to(I32).cuda(), rope=rope,
                        q=dx[:, :H], q_out=q_out)
    b = torch.repeat_interleave(torch.arange(B), n)
    m = len(b)
    t = T[b] - n[b] + torch.arange(m) - cu[b].long()
    entry = table[b, (t.clamp(min=0) // page)].long()
    row = ((t >= 0) & (entry >= 0) & (entry < num)).nonzero()[:, 0]
    where = (entry[row], slice(None), t[row] % page)
    assert 0 < len(row) < m
    got = [p.cpu() for p in dp]
    if dims:
        close(q_out[:m], model.rotate(x[:m, :H], t, f, gain, interleaved), "queries")
        close(got[0][where], model.rotate(x[row, H:H + G], t[row], f, gain, interleaved), "keys")
    else:
        assert torch.equal(q_out[:m].cpu(), x[:m, :H]) and torch.equal(got[0][where], x[row, H:H + G])
    assert torch.equal(got[1][where], x[row, H + G:])
    assert (q_out[m:].float() == 7).all()
    for p, mine in zip(got, pages):                       # and nothing else
        mine[where] = p[where]
        assert torch.equal(p, mine)
