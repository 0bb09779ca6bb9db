"""Plain float64 models of packed batches: rotary positions, the append to bf16
pages and causal attention with its error bounds."""
from __future__ import annotations

import math

import torch

BF16_HALF = torch.finfo(torch.bfloat16).eps / 2      # a rounding to bf16, relative


def frequencies(dims, base, scaling="none", factor=1.0, original=0.0, low=1.0, high=4.0):
    """Radians per position of every pair, and the factor on sine and cosine."""
    if scaling == "base" and dims > 2:
        base = base * factor ** (dims / (dims - 2))
    f = [base ** (-2 * i / dims) for i in range(dims // 2)]
    gain = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "bands":
        turns = [original * x / (2 * math.pi) for x in f]
        keep = [min(1.0, max(0.0, (t - low) / (high - low))) for t in turns]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
    elif scaling == "yarn":
        gain = 1 + 0.1 * math.log(factor)

        def pair(turns):
            return dims * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

        first, last = max(0, math.floor(pair(high))), min(dims - 1, math.ceil(pair(low)))
        slow = [min(1.0, max(0.0, (i - first) / max(last - first, 0.001))) for i in range(dims // 2)]
        f = [x * (1 - s) + x / factor * s for x, s in zip(f, slow)]
    return torch.tensor(f, dtype=torch.float64), gain


def rotate(x, t, f, gain=1.0, interleaved=False, inverse=False):
    """x [N, heads, D] rotated by positions t [N], in float64; and sum |terms| of every element."""
    h = f.numel()
    y = x.double().clone()
    size = y.abs()
    angle = t.double()[:, None, None] * f * (-1 if inverse else 1)
    c, s = torch.cos(angle) * gain, torch.sin(angle) * gain
    first = slice(0, 2 * h, 2) if interleaved else slice(0, h)
    second = slice(1, 2 * h, 2) if interleaved else slice(h, 2 * h)
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    both = (a.abs() + b.abs()) * abs(gain)
    size[..., first], size[..., second] = both, both
    return y, size


def rotate_bound(want, size):
    """Rounding to bf16, and sine and cosine off by 2^-21 (their angles by less than
    2^-22 radians, their values by less than 2^-22) with three fp32 roundings."""
    return BF16_HALF * want.abs() + 2.0 ** -20 * size


def attention(q, k, v, n, T, scale):
    """Causal attention of the last n of T tokens: q [n, H, D], k, v [T, G, D].
    Returns out and lse in float64 and the bounds of a result whose scores and
    sums are fp32, whose weights are rounded to bf16, and out to bf16."""
    H, D = q.shape[1:]
    G = k.shape[1] if k.dim() == 3 else 1
    r = H // G
    if T == 0 or n == 0:
        z = torch.zeros(n, H, D, dtype=torch.float64)
        l = torch.full((n, H), -math.inf, dtype=torch.float64)
        return z, l, torch.zeros_like(z), torch.zeros_like(l)
    qd, kd, vd = q.double(), k.double(), v.double()
    kd, vd = kd.repeat_interleave(r, 1), vd.repeat_interleave(r, 1)
    see = torch.arange(T)[None, :] <= T - n + torch.arange(n)[:, None]             # [n, T]
    x = torch.einsum("nhd,thd->hnt", qd, kd) * scale
    size = torch.einsum("nhd,thd->hnt", qd.abs(), kd.abs()) * scale
    x = torch.where(see, x, torch.full_like(x, -math.inf))
    none = ~see.any(1)
    lse = torch.logsumexp(x, 2)
    p = torch.exp(x - torch.where(none, 0.0, lse)[..., None])
    p = torch.where(see, p, torch.zeros_like(p))
    # a masked key has no part in the sum, whatever it holds
    vs = torch.where(torch.isfinite(vd), vd, torch.zeros_like(vd))
    out = torch.einsum("hnt,thd->nhd", p, vs)
    weight = torch.einsum("hnt,thd->nhd", p, vs.abs())
    bad = (~torch.isfinite(vd)).double()
    out = torch.where(torch.einsum("hnt,thd->nhd", see.double().expand_as(p), bad) > 0, math.nan, out)
    size = torch.where(see, torch.nan_to_num(size, 0.0, 0.0), torch.zeros_like(size)).amax(2).T          # [n, H]
    lse = lse.T
    # scores: D + 4 fp32 roundings of terms whose sizes sum to `size`; the sum: T of
    # them at most; exponential and logarithm: 2^-21; lse itself.
    off = (D + 4) * 2.0 ** -24 * size + T * 2.0 ** -24 + 2.0 ** -21
    lse_bound = off + 2.0 ** -22 * torch.nan_to_num(lse, 0.0, 0.0, 0.0).abs()
    out_bound = BF16_HALF * out.abs() + (BF16_HALF + 2 * off)[..., None] * weight
    return out, lse, torch.nan_to_num(out_bound, 0.0) + 1e-30, lse_bound


def check_rows(out, lse, want, what=""):
    """Compares device results [n, H, D], [n, H] with attention()'s."""
    ref, ref_lse, bound, lse_bound = want
    out, lse = out.double().cpu(), None if lse is None else lse.double().cpu()
    nan = torch.isnan(ref)
    assert torch.equal(~torch.isfinite(out), nan), f"{what}: NaN in other places ({(~torch.isfinite(out)).sum()}, {nan.sum()})"
    over = torch.where(nan, 0.0, (out - ref).abs() - bound)
    assert (over <= 0).all(), f"{what}: out off by {over.max():.3e} more than its bound at {over.argmax()}"
    if lse is not None:
        same = torch.isneginf(ref_lse) == torch.isneginf(lse)
        assert same.all(), f"{what}: empty rows differ"
        fine = torch.isfinite(ref_lse)
        off = torch.where(fine, (lse - ref_lse).abs() - lse_bound, torch.zeros_like(lse))
        assert torch.isfinite(lse[fine]).all() and (off <= 0).all(), f"{what}: lse off by {off.max():.3e} more than its bound"
        assert torch.isnan(lse[torch.isnan(ref_lse)]).all(), f"{what}: lse of NaN scores"
