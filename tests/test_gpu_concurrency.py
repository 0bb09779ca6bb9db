"""Concurrent callers: each stream gets its own library workspace, so steps
enqueued on different streams -- from one host thread or from several --
may overlap on the GPU without their partial slots or arrival counters
mixing. Plans split units over many CTAs so that every step uses them."""
import math
import threading

import numpy as np
import pytest
import torch

import grouped_query_decode_gb300 as gq
import oracle
from gpu_helpers import bf16_to_f64, compare, make_inputs, min_tiles, to_device_bf16

pytestmark = pytest.mark.gpu

D, TMAX = 128, 1200


def _case(seed, H, G, sq, lens):
    B = len(lens)
    q, k, v, lens = make_inputs(B, sq, H, G, D, TMAX, lens, seed=seed)
    dev = dict(q=to_device_bf16(q), k=to_device_bf16(k), v=to_device_bf16(v), l=torch.from_numpy(lens).cuda(),
               out=torch.empty(B, sq, H, D, dtype=torch.bfloat16, device="cuda"),
               lse=torch.empty(B, sq, H, dtype=torch.float32, device="cuda"))
    ref = oracle.gqa_decode_f64(q, k, v, lens, 1 / math.sqrt(D), threads=8)
    return dev, ref


def _check(dev, ref, what):
    compare(bf16_to_f64(dev["out"]), dev["lse"].cpu().numpy().astype(np.float64), ref[0], ref[1], what=what)


def test_two_streams_interleaved():
    cases = [_case(2301, 32, 8, 1, [1200, 700, 77]), _case(2302, 64, 8, 4, [900, 1200, 5]),
             _case(2303, 32, 1, 1, [1100, 300]), _case(2304, 16, 4, 2, [1200, 1199, 640])]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    scale = 1 / math.sqrt(D)
    with min_tiles(1):
        for rep in range(3):
            for i, (dev, _) in enumerate(cases):
                with torch.cuda.stream(streams[i % 2]):
                    gq.gqa_decode(dev["q"], dev["k"], dev["v"], dev["l"], scale, dev["out"], dev["lse"])
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    for i, (dev, ref) in enumerate(cases):
        _check(dev, ref, f"stream {i % 2} case {i}")


def test_host_threads_each_with_a_stream():
    cases = [_case(2401 + i, 32 if i % 2 else 64, 8, 1 if i % 2 else 4, [1200, 650, 33]) for i in range(4)]
    scale = 1 / math.sqrt(D)
    errors = []

    def worker(i):
        try:
            dev, _ = cases[i]
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    gq.gqa_decode(dev["q"], dev["k"], dev["v"], dev["l"], scale, dev["out"], dev["lse"], stream=s)
            s.synchronize()
        except Exception as e:   # reported on the main thread
            errors.append(e)

    with min_tiles(1):
        threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cases))]
        for t in threads:
            t.start()
        for t in threads:
            t.join(timeout=120)
    assert not errors, errors
    torch.cuda.synchronize()
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    for i, (dev, ref) in enumerate(cases):
        _check(dev, ref, f"thread {i}")


def _bits(dev):
    return dev["out"].view(torch.int16).clone(), dev["lse"].clone()


def test_a_larger_call_leaves_the_workspace_of_a_captured_one():
    """A graph captured on a stream is replayed after a larger call there has
    outgrown the stream's buffer, decode and split prefill."""
    scale = 1 / math.sqrt(D)
    small, ref = _case(2501, 32, 8, 1, [1200])
    large, _ = _case(2502, 64, 8, 4, [1200, 700, 900, 1100])
    chunk, chunk_ref = _case(2503, 8, 2, 40, [1200])
    wide, _ = _case(2504, 64, 8, 40, [1200, 1000])
    s = torch.cuda.Stream()
    with min_tiles(1), torch.cuda.stream(s):
        for first, then in ((small, large), (chunk, wide)):
            call = gq.gqa_decode if first is small else gq.gqa_prefill
            args = [first[k] for k in "qkvl"] + [scale, first["out"], first["lse"]]
            call(*args)
            s.synchronize()
            bits = _bits(first)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                call(*args)
            call(*[then[k] for k in "qkvl"], scale, then["out"], then["lse"])
            other = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")   # memory given back would be this
            for _ in range(3):
                first["out"].zero_()
                graph.replay()
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(_bits(first), bits))
            assert bool((other == 0xFF).all())
            del graph
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    gq.gqa_decode_release_workspace(s)
    _check(small, ref, "decode")
    _check(chunk, chunk_ref, "prefill")


def test_host_threads_on_one_stream():
    """Four threads on the current stream, decode steps and split prefill chunks of
    unlike sizes: what one call leaves for its second launch is its own, and no
    buffer goes away under another thread's call."""
    cases = [_case(2601, 8, 2, 40, [1200]), _case(2602, 64, 8, 40, [1200, 600]), _case(2603, 32, 8, 1, [1200, 33]),
             _case(2604, 16, 4, 70, [900])]
    scale = 1 / math.sqrt(D)
    errors, start = [], threading.Barrier(len(cases))
    torch.cuda.synchronize()

    def worker(i):
        try:
            dev, _ = cases[i]
            call = gq.gqa_decode if i == 2 else gq.gqa_prefill
            mine = [(torch.empty_like(dev["out"]), torch.empty_like(dev["lse"])) for _ in range(40)]
            start.wait(60)
            for out, lse in mine:
                call(dev["q"], dev["k"], dev["v"], dev["l"], scale, out, lse)
            torch.cuda.synchronize()
            dev["out"], dev["lse"] = mine[0]
            for out, lse in mine[1:]:
                assert torch.equal(out.view(torch.int16), mine[0][0].view(torch.int16)) and torch.equal(lse, mine[0][1])
        except Exception as e:
            errors.append((i, repr(e)[:300]))

    with min_tiles(1):
        gq.gqa_decode_release_workspace()
        threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cases))]
        for t in threads:
            t.start()
        for t in threads:
            t.join(timeout=120)
    assert not errors and not any(t.is_alive() for t in threads), errors
    assert gq.gqa_decode_check_error() == gq.GQA_OK
    for i, (dev, ref) in enumerate(cases):
        _check(dev, ref, f"thread {i}")
