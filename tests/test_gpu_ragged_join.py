"""What two pipelines, or the parts of a split unit, leave of a row is put together
with weights that may be zero: a NaN or an infinity in V that the row sees stays,
however far its scores lie below the row's largest, and a part that shows the row
nothing adds nothing."""
import math

import pytest
import torch

import grouped_query_decode_gb300 as gq

pytestmark = pytest.mark.gpu

BF, I32 = torch.bfloat16, torch.int32


def steps(T, D, at, high, sign=1.0):
    """Queries of ones and keys whose scores (scale 1) are 0 before `at` and `high` from there on;
    sign -1: the other way round."""
    k = torch.zeros(T, 1, D, dtype=BF)
    rows = slice(at, None) if sign > 0 else slice(None, at)
    k[rows, :, 0] = high
    return k


def run_paged(H, D, n, k, v, page=64, **kw):
    T = k.shape[0]
    pages = -(-T // page)
    pool = [torch.zeros(pages, 1, page, D, dtype=BF) for _ in range(2)]
    t = torch.arange(T)
    for p, x in zip(pool, (k, v)):
        p[t // page, :, t % page] = x
    q = torch.zeros(n, H, D, dtype=BF)
    q[..., 0] = 1
    out, lse = torch.full((n, H, D), 7.0, dtype=BF, device="cuda"), torch.full((n, H), 7.0, device="cuda")
    gq.gqa_prefill_paged(q.cuda(), pool[0].cuda(), pool[1].cuda(), torch.arange(pages, dtype=I32).cuda()[None],
                         torch.tensor([0, n], dtype=I32).cuda(), torch.tensor([T], dtype=I32).cuda(), 1.0, out, lse, **kw)
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    return out.float().cpu(), lse.cpu()


def check(out, lse, columns, rows=slice(None)):
    bad = torch.zeros(out.shape, dtype=torch.bool)
    for c in columns:
        bad[rows, :, c] = True
    assert torch.equal(~torch.isfinite(out), bad), "columns that are not finite"
    assert (out[~bad] == 1).all() and torch.isfinite(lse).all()


# Tokens, keys: one unit in both pipelines; many parts; two row tiles in many parts.
FORMS = [(1, 256), (3, 700), (1, 9000), (20, 30000)]


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("D,H", [(64, 8), (128, 8), (128, 32)])
@pytest.mark.parametrize("n,T", FORMS)
def test_values_far_below_the_largest_score(n, T, D, H, sign, value):
    """V[c] is not finite among keys that score 200 less than others: weight 0 in 32 bits."""
    at = 128 if T == 256 else T // 2
    k, v = steps(T, D, at, 200.0, sign), torch.ones(T, 1, D, dtype=BF)
    low = 5 if sign > 0 else at + 5
    v[low, 0, 3] = value
    v[low + 1, 0, D - 1] = value
    check(*run_paged(H, D, n, k, v), [3, D - 1])


@pytest.mark.parametrize("D", [64, 128])
def test_at_the_limits_of_the_last_rows(D):
    """The value sits in the last key tile, which only some rows see whole, far below the first keys' scores."""
    n, T = 6, 9000
    k, v = steps(T, D, 4000, 200.0, -1.0), torch.ones(T, 1, D, dtype=BF)
    v[T - 3, 0, 9] = math.nan
    out, lse = run_paged(8, D, n, k, v)
    check(out, lse, [9], slice(n - 3, None))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [100, 256, 9000])
def test_values_of_keys_that_score_nothing(D, T):
    """Every key of the first half scores -inf: their weight is 0 whatever the others score."""
    k, v = steps(T, D, T // 2, -math.inf, -1.0), torch.ones(T, 1, D, dtype=BF)
    v[T // 2 - 1, 0, 7] = math.nan
    check(*run_paged(8, D, 1, k, v), [7])


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing_over_a_workspace_of_nan(D):
    """Rows without a key, and a unit cut into parts whose last ones show some rows
    nothing, over a workspace full of NaN: what no part has written is not read."""
    H, n, T = 64, 40, 30
    q = torch.zeros(n, H, D, dtype=BF)
    q[..., 0] = 1
    big = 20000
    seqs = [(n, T), (3, big)]
    page = 64
    pages = [-(-x // page) for _, x in seqs]
    pool = [torch.ones(sum(pages), 1, page, D, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.full((2, max(pages)), -1, dtype=I32)
    table[0, :pages[0]] = torch.arange(pages[0])
    table[1, :pages[1]] = torch.arange(pages[0], sum(pages))
    N = n + 3
    q = torch.cat([q, q[:3]]).cuda()
    out, lse = torch.full((N, H, D), 7.0, dtype=BF, device="cuda"), torch.full((N, H), 7.0, device="cuda")
    ws = torch.full((gq.gqa_prefill_ragged_workspace_bytes(N, 2, H, 1, D),), 0xFF, dtype=torch.uint8, device="cuda")
    gq.gqa_prefill_paged(q, *pool, table.cuda(), torch.tensor([0, n, N], dtype=I32).cuda(),
                         torch.tensor([T, big], dtype=I32).cuda(), 1.0, out, lse, workspace=ws)
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    assert (out[:n - T].float() == 0).all() and torch.isneginf(lse[:n - T]).all()
    assert (out[n - T:].float() == 1).all() and torch.isfinite(lse[n - T:]).all()


@pytest.mark.parametrize("D,G", [(64, 2), (128, 1)])
def test_prompts_in_parts(D, G):
    """Whole prompts, cut into parts: a value far below the last keys' scores."""
    T, H = 3000, 4 * G
    k, v = steps(T, D, 2900, 200.0).expand(T, G, D).contiguous(), torch.ones(T, G, D, dtype=BF)
    v[40, 0, 5] = math.inf
    q = torch.zeros(T, H, D, dtype=BF)
    q[..., 0] = 1
    out = torch.full((T, H, D), 7.0, dtype=BF, device="cuda")
    gq.gqa_prefill_packed(q.cuda(), k.cuda(), v.cuda(), torch.tensor([0, T], dtype=I32).cuda(), 1.0, out)
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    want = torch.zeros(out.shape, dtype=torch.bool)
    want[40:, :4, 5] = True
    out = out.float().cpu()
    assert torch.equal(~torch.isfinite(out), want) and (out[~want] == 1).all()
