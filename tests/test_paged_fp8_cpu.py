"""The paged 8-bit cache without a GPU: the tests' own models against facts
that do not come from them, and the refusals of every entry point, which come
before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

import grouped_query_decode_gb300 as gq
import oracle
import paged_fp8_model as model


# ----------------------------------------------------------------- the models

def test_nearest_codes_agree_with_torch_and_are_idempotent():
    x = np.concatenate([np.linspace(-448, 448, 4001), np.linspace(-0.04, 0.04, 4001), [0.0, -0.0, np.nan]])
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = model.nearest_codes(x.astype(np.float32))
    assert np.array_equal(got, want)
    every = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    assert np.array_equal(model.nearest_codes(oracle.e4m3_to_f64(every)), every)


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.5, 1), (449.0, 1), (224.0, -1), (1.0, -8), (7 / 4, -8),
                                   (1.75 + 2 ** -8, -7), (1e-39, -126), (3.3e38, 120)])
def test_scale_for(top, e):
    assert model.scale_for(top) == 2.0 ** e


def test_append_one_by_one_is_append_at_once_for_normal_codes():
    """Power-of-two scales: a block filled token by token holds the codes of a
    block filled at once, wherever the code is a normal e4m3 number."""
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((1, 32, 2, 64)) * np.exp2(rng.integers(-4, 5, (1, 32, 2, 1)))).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    table = np.array([[1, 0]], dtype=np.int32)
    once, by_one = (np.full((2, 2, 16, 64), model.NAN_CODE, np.uint8) for _ in range(2))
    s1, s2 = (np.full((2, 2, 1), np.nan, np.float32) for _ in range(2))
    model.append(once, s1, x, table, [32])
    for t in range(32):
        model.append(by_one, s2, x[:, t:t + 1], table, [t + 1])
    assert np.array_equal(s1, s2)
    normal = (once & 0x78) != 0
    assert np.array_equal(once[normal], by_one[normal])
    err = np.abs(model.page_values(by_one, s2) - model.page_values(once, s1))
    assert (err <= s1.astype(np.float64)[..., None] * 2.0 ** -9).all()
    # and a value is within half a step of its code, or half a subnormal step
    vals = model.logical(model.page_values(once, s1), table, [32], 32)[0].transpose(1, 0, 2)
    bound = np.maximum(np.abs(x[0]) * 2.0 ** -4,
                       np.repeat(s1[table[0]].transpose(0, 2, 1).reshape(2, 2), 16, 0)[..., None] * 2.0 ** -10)
    assert (np.abs(vals - x[0]) <= bound).all()


def test_fork_model_keeps_the_invariants():
    """Counts equal the entries that name a page, no partly filled page is
    shared, and every row reads the tokens it went on from."""
    rng = np.random.default_rng(11)
    ps, B, num = 16, 6, 64
    table = np.full((B, 5), -1, np.int32)
    lens = np.array([0, 16, 17, 40, 64, 79], np.int32)
    refs = np.zeros(num, np.int32)
    table, refs, counts = model.reserve(table, lens, refs, ps)
    assert counts[0] == sum(-(-t // ps) for t in lens) and refs.sum() == counts[0]
    for step in range(8):
        src = rng.integers(-1, B, B).astype(np.int32)
        content = np.arange(num)
        new_table, new_lens, new_refs, counts, pairs = model.fork(src, table, lens, refs, ps)
        for a, b in pairs:
            content[b] = content[a]
        assert np.array_equal(new_refs, np.bincount(new_table[new_table >= 0], minlength=num))
        for i in range(B):
            s = src[i]
            n = -(-new_lens[i] // ps)
            assert new_lens[i] == (lens[s] if s >= 0 else 0)
            assert [content[p] for p in new_table[i, :n]] == [int(p) for p in table[s, :n]][:n]
            if new_lens[i] % ps:
                assert new_refs[new_table[i, n - 1]] == 1
        table, lens, refs = new_table, new_lens, new_refs


def test_compact_model():
    refs = np.array([0, 2, 0, 1, 0, 0, 3, 1], np.int32)
    table = np.array([[7, 1, -1], [6, 3, 9]], np.int32)
    out, r, counts, moves = model.compact(table, refs)
    assert counts == [2, 4] and moves == [(6, 0), (7, 2)]
    assert out.tolist() == [[2, 1, -1], [0, 3, 9]] and r.tolist() == [3, 2, 1, 1, 0, 0, 0, 0]


# ------------------------------------------------------------------- refusals

A = 1 << 20   # an aligned address that no call reads


def _attend(ptrs=None, scale=0.1, lse=None, shape=(1, 1, 8, 2, 64, 16, 4, 4), ws=A, ws_bytes=1 << 30):
    p = [A] * 8
    for i, x in (ptrs or {}).items():
        p[i] = x
    return gq.load().gqa_decode_paged_fp8(*p[:7], scale, p[7], lse, *shape, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ptrs={0: None}), gq.GQA_ERR_INVALID_ARG), (dict(ptrs={5: None}), gq.GQA_ERR_INVALID_ARG),
    (dict(ptrs={7: None}), gq.GQA_ERR_INVALID_ARG),
    (dict(ptrs={0: A + 8}), gq.GQA_ERR_MISALIGNED), (dict(ptrs={1: A + 4}), gq.GQA_ERR_MISALIGNED),
    (dict(ptrs={3: A + 2}), gq.GQA_ERR_MISALIGNED), (dict(lse=A + 1), gq.GQA_ERR_MISALIGNED),
    (dict(scale=math.inf), gq.GQA_ERR_INVALID_ARG), (dict(scale=math.nan), gq.GQA_ERR_INVALID_ARG),
    (dict(shape=(0, 1, 8, 2, 64, 16, 4, 4)), gq.GQA_ERR_INVALID_ARG),
    (dict(shape=(1, 0, 8, 2, 64, 16, 4, 4)), gq.GQA_ERR_INVALID_ARG),
    (dict(shape=(1, 1, 8, 3, 64, 16, 4, 4)), gq.GQA_ERR_HEAD_RATIO),
    (dict(shape=(1, 1, 8, 2, 96, 16, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1, 1, 8, 2, 64, 24, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1, 1, 8, 2, 64, 8, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1, 1, 8, 2, 64, 131072, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1, 1, 8, 2, 64, 65536, 4, 32768)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1, 1, 8, 2, 64, 16, 0, 4)), gq.GQA_ERR_INVALID_ARG),
    (dict(shape=(1, 1, 8, 2, 64, 16, 1 << 30, 4)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1 << 16, 1 << 12, 8, 2, 64, 16, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
])
def test_attention_refuses(kw, code):
    assert _attend(**kw) == code


def _append(ptrs=None, shape=(1, 1, 2, 64, 16, 4, 4)):
    p = [A] * 8
    for i, x in (ptrs or {}).items():
        p[i] = x
    return gq.load().gqa_append_paged_fp8(*p, *shape, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ptrs={0: None}), gq.GQA_ERR_INVALID_ARG), (dict(ptrs={7: None}), gq.GQA_ERR_INVALID_ARG),
    (dict(ptrs={1: A + 8}), gq.GQA_ERR_MISALIGNED), (dict(ptrs={4: A + 2}), gq.GQA_ERR_MISALIGNED),
    (dict(shape=(1, 0, 2, 64, 16, 4, 4)), gq.GQA_ERR_INVALID_ARG),
    (dict(shape=(1, 1, 2, 32, 16, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1, 1, 2, 64, 48, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1, 1, 2, 64, 65536, 4, 32768)), gq.GQA_ERR_UNSUPPORTED),
    (dict(shape=(1 << 20, 1 << 10, 16, 64, 16, 4, 4)), gq.GQA_ERR_UNSUPPORTED),
])
def test_append_refuses(kw, code):
    assert _append(**kw) == code


def _pool(base=A, page_bytes=64, layer_bytes=64 * 8, layers=1):
    arr = (gq.PagePoolT * 1)()
    arr[0].base, arr[0].page_bytes, arr[0].layer_bytes, arr[0].layers = base, page_bytes, layer_bytes, layers
    return arr


def test_pages_refuse():
    lib = gq.load()
    ok = _pool()
    INV, UNS, MIS, WS = (gq.GQA_ERR_INVALID_ARG, gq.GQA_ERR_UNSUPPORTED, gq.GQA_ERR_MISALIGNED,
                         gq.GQA_ERR_WORKSPACE)
    assert lib.gqa_pages_copy(ok, 1, A, A, -1, 8, None) == INV
    assert lib.gqa_pages_copy(ok, 1, A, A, 1, 0, None) == INV
    assert lib.gqa_pages_copy(None, 1, A, A, 1, 8, None) == INV
    assert lib.gqa_pages_copy(ok, 65, A, A, 1, 8, None) == UNS
    assert lib.gqa_pages_copy(ok, 1, None, A, 1, 8, None) == INV
    assert lib.gqa_pages_copy(ok, 1, A + 2, A, 1, 8, None) == MIS
    assert lib.gqa_pages_copy(ok, 1, None, None, 0, 8, None) == gq.GQA_OK     # nothing to do
    assert lib.gqa_pages_copy(_pool(base=None), 1, A, A, 1, 8, None) == INV
    assert lib.gqa_pages_copy(_pool(page_bytes=0), 1, A, A, 1, 8, None) == INV
    assert lib.gqa_pages_copy(_pool(layers=0), 1, A, A, 1, 8, None) == INV
    assert lib.gqa_pages_copy(_pool(layers=2, layer_bytes=64 * 8 - 1), 1, A, A, 1, 8, None) == INV

    big = 1 << 30
    assert lib.gqa_pages_reserve(None, A, A, A, 1, 4, 16, 8, A, big, None) == INV
    assert lib.gqa_pages_reserve(A, A, A, A, 0, 4, 16, 8, A, big, None) == INV
    assert lib.gqa_pages_reserve(A, A, A, A, 8193, 4, 16, 8, A, big, None) == UNS
    assert lib.gqa_pages_reserve(A, A, A, A, 1, 1 << 20, 1 << 11, 8, A, big, None) == UNS
    assert lib.gqa_pages_reserve(A, A, A, A, 1, 4, 16, (1 << 30) + 1, A, 1 << 40, None) == UNS
    assert lib.gqa_pages_reserve(A, A + 2, A, A, 1, 4, 16, 8, A, big, None) == MIS
    need = gq.gqa_pages_workspace_bytes(1, 8)
    assert lib.gqa_pages_reserve(A, A, A, A, 1, 4, 16, 8, A, need - 1, None) == WS
    assert lib.gqa_pages_reserve(A, A, A, A, 1, 4, 16, 8, A + 64, big, None) == WS
    assert lib.gqa_pages_reserve(A, A, A, A, 1, 4, 16, 8, None, big, None) == WS

    def fork(pools=ok, n=1, table=A, lens=A, refs=A, t_out=2 * A, l_out=2 * A, r_out=2 * A, B=1, num=8, ws=A):
        return lib.gqa_pages_fork(pools, n, A, table, lens, refs, t_out, l_out, r_out, A, B, 4, 16, num, ws, big, None)

    assert fork(t_out=A) == INV and fork(l_out=A) == INV and fork(r_out=A) == INV
    assert fork(t_out=None) == INV and fork(B=8193) == UNS and fork(num=0) == INV
    assert fork(t_out=2 * A + 2) == MIS and fork(ws=None) == WS and fork(pools=None) == INV
    assert lib.gqa_pages_free(None, A, A, A, 1, 4, 8, None) == INV
    assert lib.gqa_pages_free(A, A, A + 1, A, 1, 4, 8, None) == MIS
    assert lib.gqa_pages_free(A, A, A, A, 1, 0, 8, None) == INV
    assert lib.gqa_pages_compact(ok, 1, A, A, A, None, A, 1, 4, 8, A, big, None) == INV
    assert lib.gqa_pages_compact(ok, 1, A, A, A, A, A, 1, 4, 8, A, need - 1, None) == WS
    assert gq.gqa_pages_workspace_bytes(0, 8) == 0 and gq.gqa_pages_workspace_bytes(1, 0) == 0


def test_pages_refuse_arrays_that_overlap():
    """B = 4 rows of 4 entries (64 bytes), 8 pages (32 bytes)."""
    lib = gq.load()
    INV, big = gq.GQA_ERR_INVALID_ARG, 1 << 30
    at = [A * (i + 1) for i in range(9)]

    def fork(**kw):
        x = dict(src=at[0], table=at[1], lens=at[2], refs=at[3], t_out=at[4], l_out=at[5], r_out=at[6], counts=at[7],
                 ws=at[8])
        x.update(kw)
        return lib.gqa_pages_fork(_pool(), 1, x["src"], x["table"], x["lens"], x["refs"], x["t_out"], x["l_out"],
                                  x["r_out"], x["counts"], 4, 4, 16, 8, x["ws"], big, None)

    for kw in (dict(t_out=at[1] + 60), dict(t_out=at[1] - 60), dict(l_out=at[2] + 12), dict(r_out=at[3] - 28),
               dict(t_out=at[3]), dict(l_out=at[0]), dict(counts=at[4] + 8), dict(r_out=at[4] + 32),
               dict(ws=at[1]), dict(t_out=at[8] + 256)):
        assert fork(**kw) == INV, kw
    if not torch.cuda.is_available():       # ranges that only touch go on, to the missing device
        for kw in ({}, dict(t_out=at[1] + 64), dict(t_out=at[1] - 64), dict(l_out=at[2] + 16)):
            assert fork(**kw) not in (INV, gq.GQA_OK), kw
    assert lib.gqa_pages_reserve(at[0], at[1], at[0] + 60, at[2], 4, 4, 16, 8, at[3], big, None) == INV
    assert lib.gqa_pages_reserve(at[0], at[1], at[2], at[2] + 28, 4, 4, 16, 8, at[3], big, None) == INV
    assert lib.gqa_pages_free(at[0], at[1], at[2], at[1] + 32, 4, 4, 8, None) == INV
    assert lib.gqa_pages_compact(_pool(), 1, at[0], at[1], at[0] + 4, at[1], at[2], 4, 4, 8, at[3], big, None) == INV
    assert lib.gqa_pages_compact(_pool(), 1, at[0], at[1], at[0], at[1] - 4, at[2], 4, 4, 8, at[3], big, None) == INV
    assert lib.gqa_pages_compact(_pool(), 1, at[0], at[1], at[1], at[0], at[2], 4, 4, 8, at[3], big, None) == INV


def test_reserve_refuses_tables_past_2_31_entries():
    lib = gq.load()
    assert lib.gqa_pages_reserve(A, A, A, A, 8192, 1 << 18, 16, 8, A, 1 << 30, None) == gq.GQA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors_dtypes_and_shapes():
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    q = torch.zeros(1, 1, 8, 64, dtype=bf)
    pages = torch.zeros(4, 2, 16, 64, dtype=u8)
    sc = torch.zeros(4, 2, 1)
    table, lens = torch.zeros(1, 4, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_decode_paged_fp8(q, pages, pages, sc, sc, table, lens, 0.1, torch.zeros_like(q))
    with pytest.raises(TypeError, match="must be torch.bfloat16"):
        gq.gqa_decode_paged_fp8(q.half(), pages, pages, sc, sc, table, lens, 0.1, torch.zeros_like(q))
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_append_paged_fp8(q, q, pages, pages, sc, sc, table, lens)
    with pytest.raises(TypeError, match="must be torch.bfloat16"):
        gq.gqa_append_paged_fp8(q.float(), q, pages, pages, sc, sc, table, lens)
    refs, counts = torch.zeros(4, dtype=i32), torch.zeros(2, dtype=i32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_pages_reserve(table, lens, refs, 16, counts)
    with pytest.raises(TypeError, match="must be torch.int32"):
        gq.gqa_pages_reserve(table.long(), lens, refs, 16, counts)
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_pages_free(torch.zeros(1, dtype=torch.bool), table, lens, refs)
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_pages_copy([pages], lens, lens, 4)
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_pages_fork([pages], lens, table, lens, refs, 16, table, lens, refs, counts)
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_pages_compact([pages], table, refs, table, refs, counts)


def test_pool_array_counts_layers_and_bytes(monkeypatch):
    monkeypatch.setattr(gq, "_check_all", lambda *a: None)
    codes = torch.zeros(3, 2, 7, 4, 16, 64, dtype=torch.uint8)
    scales = torch.zeros(6, 7, 4, 1)
    arr, n = gq._page_pools(0, [codes], 7, 2)
    assert (n, arr[0].layers, arr[0].page_bytes, arr[0].layer_bytes) == (1, 6, 4 * 16 * 64, 7 * 4 * 16 * 64)
    arr, n = gq._page_pools(0, [scales], 7, 1)
    assert (arr[0].layers, arr[0].page_bytes, arr[0].layer_bytes) == (6, 16, 7 * 16)
    assert arr[0].base == scales.data_ptr()
    with pytest.raises(ValueError, match="count 7 pages"):
        gq._page_pools(0, [scales], 7, 0)
    with pytest.raises(ValueError, match="is empty"):
        gq._page_pools(0, [torch.zeros(7, 0)], 7, 0)
    assert ctypes.sizeof(gq.PagePoolT) == 32


def test_host_threads_on_one_stream_do_not_share_a_workspace(monkeypatch):
    """A call of two launches plans in its workspace and reads the plan back:
    another thread's call that is enqueued in between, on the same stream, has a
    workspace of its own. One thread keeps its buffer from call to call; a
    release forgets those of every thread."""
    import threading
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(gq, "_call", lambda *a: gq.GQA_OK)
    monkeypatch.setattr(gq, "_stream_handle", lambda stream, device: ctypes.c_void_p(0))
    like, n = torch.zeros(1), 3
    got, turns, errors = [[] for _ in range(n)], threading.Barrier(n), []

    def work(i):
        try:
            for _ in range(4):                    # every thread is within its call at once
                got[i].append(gq._workspace(64, like, 0, None))
                turns.wait(20)
            if i == 0:
                gq.gqa_decode_release_workspace()
            turns.wait(20)
            got[i].append(gq._workspace(64, like, 0, None))
            got[i].append(gq._workspace(100, like, 0, None))
            got[i].append(gq._workspace(64, like, 0, None))
            turns.wait(20)
        except Exception as e:
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors
    for mine in got:
        assert all(b is mine[0] for b in mine[:4])              # kept
        assert mine[4] is not mine[0]                           # released
        assert mine[5].numel() >= 100 and mine[6] is mine[5]    # grown, then kept
    for turn in range(7):
        at = [mine[turn].data_ptr() for mine in got]
        assert len(set(at)) == n, turn


def test_a_workspace_size_that_could_not_be_found_is_asked_for_again(monkeypatch):
    """0 may mean that the device could not be asked just then."""
    answers = iter([0, 4096])
    monkeypatch.setattr(gq, "_call", lambda *a: next(answers))
    sizes = (1, 1, 8, 2, 64, 16, 77777)
    assert gq.gqa_decode_paged_fp8_workspace_bytes(*sizes, device=0) == 0
    assert gq.gqa_decode_paged_fp8_workspace_bytes(*sizes, device=0) == 4096
    assert gq.gqa_decode_paged_fp8_workspace_bytes(*sizes, device=0) == 4096
