"""Plain models of the paged 8-bit cache for the tests: its values, the
quantising append and the page management, in numpy, one step at a time."""
from __future__ import annotations

import numpy as np

import oracle

NAN_CODE = 0x7F


def block_tokens(page_size):
    return min(64, page_size)


def blocks_of(page_size):
    return -(-page_size // 64)


def page_values(codes, scale):
    """[num_pages, G, ps, D] codes times their block's scale, in float64."""
    size = block_tokens(codes.shape[2])
    return oracle.e4m3_to_f64(codes) * np.repeat(np.asarray(scale, dtype=np.float64), size, axis=2)[..., None]


def logical(values, table, lens, tmax):
    """The [B, G, tmax, D] cache behind the pages; entries outside the pool
    read as zeros, positions past a length are NaN."""
    num, G, ps, D = values.shape
    B = table.shape[0]
    out = np.full((B, G, tmax, D), np.nan)
    for b in range(B):
        T = int(min(max(lens[b], 0), tmax))
        for j in range(-(-T // ps)):
            lo, hi = j * ps, min((j + 1) * ps, T)
            p = int(table[b, j])
            out[b, :, lo:hi] = values[p, :, :hi - lo] if 0 <= p < num else 0.0
    return out


_CODE_VALUES = oracle.e4m3_to_f64(np.arange(256, dtype=np.uint8))
_POSITIVE = _CODE_VALUES[:127]          # 0 .. 448 in ascending order, one per code


def nearest_codes(x):
    """e4m3 codes of float64 values of magnitude <= 448: nearest, ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    to_lo, to_hi = a - _POSITIVE[lo], _POSITIVE[hi] - a
    take_lo = (to_lo < to_hi) | ((to_lo == to_hi) & (lo % 2 == 0))
    code = np.where(take_lo, lo, hi).astype(np.uint8) | np.where(np.signbit(x), 128, 0).astype(np.uint8)
    return np.where(np.isnan(x), np.uint8(NAN_CODE), code).astype(np.uint8)


def scale_for(top):
    """Smallest power of two >= top / 448, 0 for 0, at least 2^-126."""
    if top == 0:
        return 0.0
    e = -126
    while 448.0 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def append(codes, scale, new, table, lens):
    """Appends new [B, sq, G, D] (float64 of bf16) to one pool in place, token
    block by token block."""
    num, G, ps, D = codes.shape
    B, sq = new.shape[:2]
    size = block_tokens(ps)
    tmax = table.shape[1] * ps
    for b in range(B):
        T = int(min(max(lens[b], 0), tmax))
        first = max(T - sq, 0)
        for block in range(first // size, -(-T // size)):
            lo, hi = max(block * size, first), min((block + 1) * size, T)
            p = int(table[b, block * size // ps])
            if lo >= hi or not 0 <= p < num:
                continue
            at = block * size % ps
            kept = lo - block * size
            for g in range(G):
                x = new[b, lo - (T - sq):hi - (T - sq), g]
                fin = np.abs(x[np.isfinite(x)])
                top = fin.max() if fin.size else 0.0
                old = float(scale[p, g, at // 64]) if kept else 0.0
                s = old if old > 0 and top <= 448 * old else scale_for(top)
                if kept and s != old:
                    vals = oracle.e4m3_to_f64(codes[p, g, at:at + kept]) * (old / s if s else 0.0)
                    codes[p, g, at:at + kept] = nearest_codes(vals)
                y = np.where(np.isfinite(x), x, np.nan)
                codes[p, g, at + kept:at + kept + hi - lo] = nearest_codes(y / s if s else y * 0.0)
                scale[p, g, at // 64] = s


# ------------------------------------------------------------------- pages

def free_pages(refs):
    return [p for p in range(len(refs)) if refs[p] <= 0]


def tokens(lens, b, table, ps):
    return int(min(max(lens[b], 0), table.shape[1] * ps))


def reserve(table, lens, refs, ps):
    table, refs = table.copy(), refs.copy()
    num = len(refs)
    empty = [(b, j) for b in range(table.shape[0]) for j in range(-(-tokens(lens, b, table, ps) // ps))
             if not 0 <= table[b, j] < num]
    free = free_pages(refs)
    counts = [len(empty), len(free)]
    if len(empty) <= len(free):
        for (b, j), p in zip(empty, free):
            table[b, j], refs[p] = p, 1
    return table, refs, counts


def fork(src, table, lens, refs, ps):
    """Returns table, lens, refs, counts and the (from, to) copies."""
    B, most = table.shape
    num = len(refs)
    free = free_pages(refs)
    out = np.full_like(table, -1)
    lens_out = np.zeros_like(lens)
    pairs, taken = [], set()
    for i in range(B):
        s = int(src[i])
        if not 0 <= s < B:
            continue
        T = tokens(lens, s, table, ps)
        lens_out[i] = T
        if s not in taken:
            taken.add(s)
            out[i] = table[s]
            continue
        out[i, :T // ps] = table[s, :T // ps]
        if T % ps and 0 <= table[s, T // ps] < num:
            if len(pairs) < len(free):
                out[i, T // ps] = free[len(pairs)]
            pairs.append((int(table[s, T // ps]), int(out[i, T // ps])))
    counts = [len(pairs), len(free)]
    if counts[0] > counts[1]:
        return table.copy(), lens.copy(), refs.copy(), counts, []
    refs = refs.copy()
    for e in table.ravel():
        if 0 <= e < num:
            refs[e] -= 1
    for e in out.ravel():
        if 0 <= e < num:
            refs[e] += 1
    return out, lens_out, refs, counts, pairs


def free(done, table, lens, refs):
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    for b in np.nonzero(done)[0]:
        for e in table[b]:
            if 0 <= e < len(refs) and refs[e] > 0:
                refs[e] -= 1
        table[b], lens[b] = -1, 0
    return table, lens, refs


def compact(table, refs):
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] <= 0]
    moved = [p for p in range(live, len(refs)) if refs[p] > 0]
    to = dict(zip(moved, holes))
    out = np.array([to.get(int(e), int(e)) for e in table.ravel()], dtype=table.dtype).reshape(table.shape)
    refs = refs.copy()
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
    return out, refs, [len(moved), live], list(to.items())
