"""Packed batches without a GPU: refusals of the C calls and of the binding, the
rotary frequencies against their formulas, the test model against torch."""
import ctypes
import math

import pytest
import torch

import grouped_query_decode_gb300 as gq
import ragged_model as model

OK_SIZES = dict(N=16, B=2, H=8, G=2, D=64)


def packed(lib, q=256, k=512, v=768, cu=1024, scale=0.125, out=1280, lse=None, N=16, B=2, H=8, G=2, D=64, qs=None,
           ks=None, vs=None, ws=4096, nbytes=1 << 30):
    return lib.gqa_prefill_packed(q, k, v, cu, scale, out, lse, N, B, H, G, D, H * D if qs is None else qs,
                                  G * D if ks is None else ks, G * D if vs is None else vs, ws, nbytes, None)


def paged(lib, q=256, k=512, v=768, table=1024, cu=1040, lens=1056, scale=0.125, out=1280, lse=None, N=16, B=2, H=8,
          G=2, D=64, qs=None, page=16, num=4, most=4, ws=4096, nbytes=1 << 30):
    return lib.gqa_prefill_paged(q, k, v, table, cu, lens, scale, out, lse, N, B, H, G, D, H * D if qs is None else qs,
                                 page, num, most, ws, nbytes, None)


@pytest.mark.parametrize("call", [packed, paged])
def test_attention_refusals(call):
    lib = gq.load()
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(N=-1), dict(B=0), dict(H=0),
                dict(G=0), dict(D=0), dict(qs=8 * 64 - 8)):
        assert call(lib, **bad) == gq.GQA_ERR_INVALID_ARG, bad
    assert call(lib, H=7) == gq.GQA_ERR_HEAD_RATIO
    for bad in (dict(D=96), dict(H=129, G=1), dict(N=1 << 29)):
        assert call(lib, **bad) == gq.GQA_ERR_UNSUPPORTED, bad
    for bad in (dict(q=264), dict(k=520), dict(v=776), dict(out=1288), dict(cu=1026), dict(lse=1026), dict(qs=8 * 64 + 4)):
        assert call(lib, **bad) == gq.GQA_ERR_MISALIGNED, bad
    assert call(lib, N=0) == gq.GQA_OK
    if call is packed:
        assert call(lib, ks=64) == gq.GQA_ERR_INVALID_ARG and call(lib, vs=129) == gq.GQA_ERR_MISALIGNED
    else:
        for bad in (dict(table=None), dict(lens=None), dict(page=0), dict(num=0), dict(most=0)):
            assert call(lib, **bad) == gq.GQA_ERR_INVALID_ARG, bad
        for bad in (dict(page=8), dict(page=48), dict(page=1 << 17), dict(page=65536, most=1 << 15), dict(num=1 << 30)):
            assert call(lib, **bad) == gq.GQA_ERR_UNSUPPORTED, bad
        assert call(lib, table=1026) == gq.GQA_ERR_MISALIGNED and call(lib, lens=1057) == gq.GQA_ERR_MISALIGNED


def test_rope_refusals():
    lib = gq.load()
    rope = gq.gqa_rope_init(64)

    def call(r=rope, q=256, k=512, pos=768, qo=256, ko=512, N=4, H=8, G=2, D=64, qs=512, ks=128, qos=512, kos=128):
        return lib.gqa_rope(None if r is None else ctypes.addressof(r), q, k, pos, qo, ko, N, H, G, D, qs, ks, qos, kos,
                            0, None)

    for bad in (dict(r=None), dict(q=None, k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(N=-1), dict(H=0),
                dict(G=0), dict(qs=504), dict(kos=120)):
        assert call(**bad) == gq.GQA_ERR_INVALID_ARG, bad
    for bad in (dict(q=264), dict(ko=520), dict(pos=770), dict(qs=516), dict(kos=132)):
        assert call(**bad) == gq.GQA_ERR_MISALIGNED, bad
    for bad in (dict(D=96, qs=96 * 8), dict(N=1 << 29)):
        assert call(**bad) == gq.GQA_ERR_UNSUPPORTED, bad
    assert call(N=0) == gq.GQA_OK
    for field, value in (("dims", 0), ("dims", 3), ("dims", 66), ("gain", math.nan)):
        r = gq.gqa_rope_init(64)
        setattr(r, field, value)
        assert call(r=r) == gq.GQA_ERR_INVALID_ARG
    r = gq.gqa_rope_init(64)
    r.inv_freq[31] = math.inf
    assert call(r=r) == gq.GQA_ERR_INVALID_ARG


def test_in_place_keeps_the_stride():
    """Rotated into itself, a tensor has one stride: with two, tokens would overwrite others."""
    lib = gq.load()
    rope = ctypes.addressof(gq.gqa_rope_init(64))
    args = lambda q, qo, qs, qos: (rope, q, None, 768, qo, None, 4, 8, 0, 64, qs, 0, qos, 0, 0, None)  # noqa: E731
    assert lib.gqa_rope(*args(256, 256, 512, 640)) == gq.GQA_ERR_INVALID_ARG
    key = lambda ks, kos: (rope, None, 256, 768, None, 256, 4, 0, 2, 64, 0, ks, 0, kos, 0, None)       # noqa: E731
    assert lib.gqa_rope(*key(128, 256)) == gq.GQA_ERR_INVALID_ARG
    append = lambda qs, qos: (rope, 256, 512, 768, 256, 1024, 1280, 1536, 1552, 1568, 4, 2, 8, 2, 64,  # noqa: E731
                              qs, 128, 128, qos, 16, 4, 4, None)
    assert lib.gqa_append_paged(*append(512, 640)) == gq.GQA_ERR_INVALID_ARG


def test_append_refusals():
    lib = gq.load()
    rope = gq.gqa_rope_init(64)

    def call(r=ctypes.addressof(rope), q=256, k=512, v=768, qo=256, kp=1024, vp=1280, table=1536, cu=1552, lens=1568,
             N=4, B=2, H=8, G=2, D=64, qs=512, ks=128, vs=128, qos=512, page=16, num=4, most=4):
        return lib.gqa_append_paged(r, q, k, v, qo, kp, vp, table, cu, lens, N, B, H, G, D, qs, ks, vs, qos, page, num,
                                    most, None)

    for bad in (dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(table=None), dict(cu=None),
                dict(lens=None), dict(qo=None), dict(N=-1), dict(B=0), dict(G=0), dict(H=0), dict(page=0), dict(num=0),
                dict(most=0), dict(ks=120), dict(qs=8)):
        assert call(**bad) == gq.GQA_ERR_INVALID_ARG, bad
    assert call(H=7) == gq.GQA_ERR_HEAD_RATIO
    for bad in (dict(page=8), dict(page=24), dict(D=32), dict(page=65536, most=1 << 15), dict(num=1 << 30)):
        assert call(**bad) == gq.GQA_ERR_UNSUPPORTED, bad
    for bad in (dict(k=520), dict(kp=1032), dict(cu=1553), dict(vs=132)):
        assert call(**bad) == gq.GQA_ERR_MISALIGNED, bad
    assert call(N=0) == gq.GQA_OK


@pytest.mark.parametrize("bad", [dict(dims=0), dict(dims=66), dict(dims=7), dict(base=1.0), dict(base=-3.0),
                                 dict(base=math.inf), dict(scaling="linear", factor=0.5),
                                 dict(scaling="bands", factor=2.0), dict(scaling="yarn", factor=2.0, original=10.0, low=2.0, high=1.0)])
def test_rope_init_refusals(bad):
    with pytest.raises(gq.GQADecodeError) as e:
        gq.gqa_rope_init(64, **bad)
    assert e.value.status == gq.GQA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        gq.gqa_rope_init(64, scaling="other")
    with pytest.raises(gq.GQADecodeError):
        gq.gqa_rope_init(96)


@pytest.mark.parametrize("D,dims", [(64, 64), (128, 128), (128, 32), (64, 2), (64, 10)])
@pytest.mark.parametrize("how", [dict(base=10000.0), dict(base=500000.0, scaling="linear", factor=4.0),
                                 dict(base=10000.0, scaling="base", factor=8.0),
                                 dict(base=500000.0, scaling="bands", factor=8.0, original=8192.0, low=1.0, high=4.0),
                                 dict(base=10000.0, scaling="yarn", factor=16.0, original=4096.0, low=1.0, high=32.0)])
def test_frequencies(D, dims, how):
    rope = gq.gqa_rope_init(D, dims=dims, **how)
    f, gain = model.frequencies(dims, **how)
    got = torch.tensor(list(rope.inv_freq), dtype=torch.float64)
    assert rope.dims == dims and abs(rope.gain - gain) < 1e-15
    assert ((got[:dims // 2] - f).abs() <= 2.0 ** -48 * f.abs()).all() and (got[dims // 2:] == 0).all()
    # Lengthened contexts slow pairs down, by the factor at most; the fastest pair of "bands" and "yarn" is kept.
    plain = model.frequencies(dims, how["base"])[0]
    factor = how.get("factor", 1.0)
    assert (got[:dims // 2] <= plain * (1 + 1e-12)).all() and (got[:dims // 2] >= plain / factor * (1 - 1e-9)).all()


def test_binding_refuses():
    bf = torch.bfloat16
    q, k = torch.zeros(4, 8, 64, dtype=bf), torch.zeros(4, 2, 64, dtype=bf)
    cu, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    table, pages = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(4, 2, 16, 64, dtype=bf)
    rope = gq.gqa_rope_init(64)
    for t in (q, q.float()):
        with pytest.raises(TypeError, match="CUDA tensor|must be torch.bfloat16"):
            gq.gqa_prefill_packed(t, k, k, cu, 0.1, q.clone())
        with pytest.raises(TypeError, match="CUDA tensor|must be torch.bfloat16"):
            gq.gqa_prefill_paged(t, pages, pages, table, cu, lens, 0.1, q.clone())
        with pytest.raises(TypeError, match="CUDA tensor|must be torch.bfloat16"):
            gq.gqa_rope(rope, t, k, torch.zeros(4, dtype=torch.int32), t, k)
    with pytest.raises(TypeError, match="CUDA tensor"):
        gq.gqa_append_paged(k, k, pages, pages, table, cu, lens)
    with pytest.raises(TypeError, match="gqa_rope_init"):
        gq.gqa_rope(None, q, k, torch.zeros(4, dtype=torch.int32), q, k)
    with pytest.raises(ValueError, match="q comes with q_out"):
        gq.gqa_append_paged(k, k, pages, pages, table, cu, lens, rope=rope, q=q)
    with pytest.raises(ValueError, match="q comes with q_out"):
        gq.gqa_rope(rope, q, None, torch.zeros(4, dtype=torch.int32), None, None)


def test_the_model_is_torchs_attention():
    """The model of the GPU tests against torch's attention in float64, and its closed forms."""
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(9, h, 64, generator=g).to(torch.bfloat16) for h in (6, 2, 2))
    out, lse, bound, lse_bound = model.attention(q, k, v, 9, 9, 0.2)
    want = torch.nn.functional.scaled_dot_product_attention(
        *(x.double().transpose(0, 1).repeat_interleave(6 // x.shape[1], 0) for x in (q, k, v)), is_causal=True, scale=0.2)
    assert (out - want.transpose(0, 1)).abs().max() < 1e-12
    assert torch.equal(out[0], v[0].double().repeat_interleave(3, 0))
    assert (bound > 0).all() and (bound < 0.1).all() and (lse_bound < 1e-3).all()
    part = model.attention(q[5:], k, v, 4, 9, 0.2)
    assert (part[0] - out[5:]).abs().max() < 1e-12 and (part[1] - lse[5:]).abs().max() < 1e-12
    none = model.attention(q[:4], k[:2], v[:2], 4, 2, 0.2)
    assert (none[0][:2] == 0).all() and torch.isneginf(none[1][:2]).all() and torch.isfinite(none[1][2:]).all()


def test_the_models_rotation_is_a_rotation():
    f, gain = model.frequencies(64, 10000.0)
    x = torch.randn(5, 3, 64, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    t = torch.tensor([0, 1, 7, 100, 5000])
    for pairs in (False, True):
        y, _ = model.rotate(x, t, f, gain, pairs)
        assert (y[0] == x[0]).all() and ((y * y).sum(-1) - (x * x).sum(-1)).abs().max() < 1e-9
        assert (model.rotate(y, t, f, gain, pairs, inverse=True)[0] - x).abs().max() < 1e-10
    y, _ = model.rotate(x, t, f)
    assert torch.allclose(y[2, 0, 0], x[2, 0, 0] * math.cos(7) - x[2, 0, 32] * math.sin(7))
