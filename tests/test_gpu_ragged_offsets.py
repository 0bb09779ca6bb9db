"""Offsets of packed batches (cu) that lie outside the rows, or descend: entries are
clamped to [0, N]; descending ones, which no call checks, leave everything alone that
lies in no sequence's range."""
import pytest
import torch

import grouped_query_decode_gb300 as gq
import ragged_model as model
from test_gpu_ragged import Batch

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


@pytest.mark.parametrize("cu", [[-7, 10, 30, 1000], [0, 10, 30, 35], [-(1 << 31), 10, 30, (1 << 31) - 1]])
def test_entries_outside_the_rows(cu):
    """Attention with and without pages and the append take the same rows."""
    seqs, H, G, D, page = [(10, 25), (20, 20), (5, 400)], 8, 2, 64, 16
    b = Batch(H, G, D, seqs, page=page, seed=80).device()
    b.dcu = i32(cu)
    b.call()
    b.check("pages")
    p = Batch(H, G, D, [(n, n) for n, _ in seqs], seed=81).device()
    p.dcu = i32(cu)
    p.call()
    p.check("packed")
    pages = [torch.zeros_like(x) for x in b.dp]
    gq.gqa_append_paged(p.dk, p.dv, *pages, b.dt, b.dcu, b.dl)
    want = [torch.zeros_like(x) for x in b.pages]
    at = 0
    for i, (n, T) in enumerate(seqs):
        t = torch.arange(T - n, T)
        for w, x in zip(want, (p.k, p.v)):
            w[b.table[i].long()[t // page], :, t % page] = x[at:at + n]
        at += n
    assert all(torch.equal(x.cpu(), w) for x, w in zip(pages, want))


@pytest.mark.parametrize("cu", [[5, 3, 9, 2, 12], [12, 9, 6, 3, 0], [0, 14, 4, 14, 8], [8, 8, 2, 11, 11]])
def test_descending_entries_stay_inside(cu):
    seqs, H, G, D, page = [(1, 20), (1, 33), (1, 16), (1, 60)], 8, 2, 64, 16
    N = 16
    b = Batch(H, G, D, seqs, page=page, behind=N - 4, seed=82, fill=1.0).device()
    b.dcu = i32(cu)
    b.call()
    p = Batch(H, G, D, [(N, N)], seed=83).device()
    p.dcu = i32(cu)
    p.call()
    rows, new = set(), set()
    for i, (_, T) in enumerate(seqs):
        first, end = cu[i], max(cu[i], cu[i + 1])
        rows |= set(range(first, end))
        new |= {(int(b.table[i, t // page]), t % page) for t in range(max(0, T - (end - first)), T)}
    outside = [n for n in range(N) if n not in rows]
    for x in (b, p):
        assert (x.out[outside].float() == 7).all() and (x.lse[outside] == 7).all()
    pages = [torch.full_like(x, 3.0) for x in b.dp]
    q_out = torch.full_like(p.out, 7.0)
    gq.gqa_append_paged(p.dk, p.dv, *pages, b.dt, b.dcu, b.dl, q=p.dq, q_out=q_out)
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    assert (q_out[outside].float() == 7).all()
    for x in pages:
        touched = (x.float() != 3.0).any(-1).any(1).nonzero().tolist()
        assert {tuple(t) for t in touched} <= new


def test_the_last_of_several_empty_sequences():
    """Rows belong to the sequence whose range holds them, whatever empty ones lie around it."""
    f, _ = model.frequencies(64, 10000.0)
    news, page = [0, 0, 3, 0, 0, 1, 0], 16
    cu = torch.tensor([0] + news).cumsum(0).to(I32)
    lens = [9, 0, 30, 4, 8, 17, 0]
    table = torch.arange(14, dtype=I32).view(7, 2)
    k = torch.randn(4, 1, 64, generator=torch.Generator().manual_seed(84)).to(BF)
    pages = [torch.zeros(14, 1, page, 64, dtype=BF, device="cuda") for _ in range(2)]
    gq.gqa_append_paged(k.cuda(), k.cuda(), *pages, table.cuda(), cu.cuda(), i32(lens), rope=gq.gqa_rope_init(64))
    t, b = torch.tensor([27, 28, 29, 16]), torch.tensor([2, 2, 2, 5])
    at = table[b, t // page].long()
    got = pages[0].cpu()
    want = model.rotate(k, t, f)
    assert ((got[at, :, t % page].double() - want[0]).abs() <= model.rotate_bound(*want)).all()
    got[at, :, t % page] = 0
    assert (got == 0).all() and torch.equal(pages[1].cpu()[at, :, t % page], k)
