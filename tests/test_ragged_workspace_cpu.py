"""Workspace sizes of packed batches as the binding asks for them, without a GPU."""
import grouped_query_decode_gb300 as gq


def asked(monkeypatch, answers):
    calls = []

    def call(device, fn, *sizes):
        calls.append((device, *sizes))
        return next(answers)

    monkeypatch.setattr(gq, "_call", call)
    gq._known_ragged_bytes.cache_clear()
    return calls


def test_steps_of_changing_sizes_ask_once(monkeypatch):
    """The size depends on D and the device alone: a serving loop's row and sequence counts change every step."""
    calls = asked(monkeypatch, iter([1024, 2048, 4096]))
    got = []
    monkeypatch.setattr(gq, "_ragged_outputs", lambda dev, q, out, lse, ws: (q.shape, 0))
    monkeypatch.setattr(gq, "_row_stride", lambda *a: 0)
    monkeypatch.setattr(gq, "_check_all", lambda *a: None)
    monkeypatch.setattr(gq, "_launch", lambda *a: gq.GQA_OK)
    monkeypatch.setattr(gq, "_raw_stream", lambda *a: None)
    monkeypatch.setattr(gq, "_workspace", lambda n, like, dev, stream: got.append(n) or like)
    import torch
    i32 = torch.int32
    for N in range(1, 40):
        B = 1 + N % 5
        q, k = torch.zeros(N, 8, 64, dtype=torch.bfloat16), torch.zeros(N, 2, 64, dtype=torch.bfloat16)
        cu, pages = torch.zeros(B + 1, dtype=i32), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
        gq.gqa_prefill_packed(q, k, k, cu, 0.1, q)
        gq.gqa_prefill_paged(q, pages, pages, torch.zeros(B, 2, dtype=i32), cu, torch.zeros(B, dtype=i32), 0.1, q)
    assert set(got) == {1024} and len(calls) == 1
    wide = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    gq.gqa_prefill_packed(wide, wide, wide, torch.zeros(2, dtype=i32), 0.1, wide)
    assert got[-1] == 2048 and len(calls) == 2
    gq._known_ragged_bytes.cache_clear()


def test_a_size_that_could_not_be_found_is_asked_for_again(monkeypatch):
    calls = asked(monkeypatch, iter([0, 4096]))
    assert [gq._ragged_workspace_bytes(64, 0) for _ in range(3)] == [0, 4096, 4096] and len(calls) == 2
    gq._known_ragged_bytes.cache_clear()


def test_the_public_size_is_of_the_sizes_given(monkeypatch):
    calls = asked(monkeypatch, iter([512, 0]))
    assert gq.gqa_prefill_ragged_workspace_bytes(70, 3, 8, 2, 64, device=1) == 512
    assert gq.gqa_prefill_ragged_workspace_bytes(70, 3, 7, 2, 64, device=1) == 0
    assert calls == [(1, 70, 3, 8, 2, 64), (1, 70, 3, 7, 2, 64)]
