"""Times of the paged 8-bit cache: its attention, its quantising append and the
management of its pages, beside their plain forms in elementary torch.

The cache holds e4m3 codes in pages [num_pages, G, page_size, D] reached through
a block table [B, max_pages], with one fp32 scale per block of min(64, page_size)
tokens of a page and KV head; a value is decode(code) * scale. Pages are shared
between sequences by reference counts.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
LARGEST_KV_BYTES = 2_200_000_000     # codes read by the largest listed attention case


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One short conversation on a small model (32 query heads over 8 KV
        # heads, head size 64): a call whose time is latency.
        attend("decode_tiny_d64_p16", 1, 1, 32, 8, 64, 1024, 1024, 16),
        # The layer of an 8B model in a decode step of a mid-sized batch.
        attend("decode_layer_p64", 16, 1, 32, 8, 128, 4096, 4096, 64),
        # Multi-query attention: every head of a sequence reads one KV head.
        attend("decode_mqa_p32", 64, 1, 32, 1, 128, 8192, 8192, 32),
        # One long context in the shortest pages.
        attend("decode_long_p16", 1, 1, 64, 8, 128, 131072, 131072, 16),
        # Speculative decoding: 4 new tokens of 64 sequences of any length.
        attend("decode_ragged_sq4_p64", 64, 4, 64, 8, 128, 512, 32768, 64),
        # A 64-token chunk of a prompt behind 4032 cached tokens.
        attend("chunk_q64_d64_p64", 1, 64, 32, 8, 64, 4096, 4096, 64),
        # The new token of every sequence of a decode step.
        append("append_step_p16", 64, 1, 8, 128, 512, 8191, 16),
        # A 2048-token chunk of four prompts.
        append("append_prompt_p64", 4, 2048, 8, 128, 8192, 8192, 64),
        # Beam search over one layer: eight groups of four beams.
        pages("fork_beams_p16", "fork", 32, 4, 8, 128, 16, 1, 2048, 512, "bf16"),
        # Beam search over all layers of a model with 8-bit pages.
        pages("fork_layers_p64", "fork", 64, 4, 8, 128, 64, 32, 512, 384, "fp8"),
        # A half-empty pool packed to its lowest pages before it is shrunk.
        pages("compact_p64", "compact", 64, 1, 8, 128, 64, 8, 2048, 1024, "fp8"),
        # The table's part of a serving step of a large pool: pages for the
        # sequences that grow, and the pages of the finished ones given back.
        pages("turnover_p16", "turnover", 256, 1, 8, 128, 16, 0, 65536, 2048, "fp8"),
    ]


def attend(name, B, sq, H, G, D, t_lo, t_hi, page):
    return dict(name=name, op="attend", B=B, sq=sq, H=H, G=G, D=D, t_lo=t_lo, t_hi=t_hi, page=page)


def append(name, B, sq, G, D, t_lo, t_hi, page):
    return dict(name=name, op="append", B=B, sq=sq, G=G, D=D, t_lo=t_lo, t_hi=t_hi, page=page)


def pages(name, op, B, beams, G, D, page, layers, num_pages, t_hi, kind):
    return dict(name=name, op=op, B=B, beams=beams, G=G, D=D, page=page, layers=layers,
                num_pages=num_pages, t_hi=t_hi, kind=kind)


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "fork", "compact", "turnover"])
    page = rng.choice([16, 32, 64, 128, 256])
    D = rng.choice([64, 128])
    if op in ("attend", "append"):
        G = rng.choice([1, 2, 3, 4, 8, 16, 32])
        sq = rng.choice([1, 1, 1, 2, 3, 4, 7, 16]) if op == "attend" else log_int(rng, 1, 2048)
        t_hi = max(log_int(rng, 16, 131072 if op == "attend" else 16384), sq)
        most = LARGEST_KV_BYTES // 2 if op == "attend" else 1 << 29
        B = log_int(rng, 1, max(1, min(128, most // (t_hi * G * D * 2))))
        if op == "append":
            B = max(1, min(B, (4 * 2048 * 8 * 128) // (sq * G * D)))
        t_lo = max(sq, int(t_hi * rng.choice([1.0, 0.5, 0.02])))
        if op == "append":
            c = append("", B, sq, G, D, t_lo, t_hi, page)
        else:
            rows = rng.choice([1, 2, 3, 4, 5, 8])          # query heads of a KV head
            while B * sq * G * rows * t_hi > 64 * 4 * 64 * 16640:
                rows, sq = max(1, rows // 2), max(1, sq // 2)
            c = attend("", B, sq, G * rows, G, D, t_lo, t_hi, page)
    elif op == "fork":
        beams = rng.choice([1, 2, 3, 4, 8])
        B = beams * rng.randint(1, 64 // beams)
        layers = log_int(rng, 1, 32)
        t_hi = log_int(rng, 2, 2048)
        G = rng.choice([1, 2, 8])
        num = B * (t_hi // page + 2) + B + rng.randint(0, 100)
        kind = rng.choice(["bf16", "fp8"])
        size = 2 * layers * G * page * D * (2 if kind == "bf16" else 1)
        while num * size > 2_100_000_000:
            layers, size = max(1, layers // 2), size // 2
            if layers == 1 and num * size > 2_100_000_000:
                t_hi, G = max(2, t_hi // 2), 1
                num = B * (t_hi // page + 2) + B
                size = 2 * page * D * (2 if kind == "bf16" else 1)
        c = pages("", op, B, beams, G, D, page, layers, num, t_hi, kind)
    elif op == "compact":
        num = log_int(rng, 64, 2048)
        B = rng.randint(1, 64)
        layers = rng.randint(1, max(1, min(16, 2_000_000_000 // (num * 2 * 2 * page * D))))
        t_hi = max(1, num * page // (2 * B))
        c = pages("", op, B, 1, 2, D, page, layers, num, t_hi, "fp8")
    else:
        B = log_int(rng, 1, 256)
        num = log_int(rng, 1024, 65536)
        t_hi = max(2, min(2048, num * page // (2 * B) - 2 * page))
        c = pages("", op, B, 1, 1, D, page, 0, num, t_hi, "fp8")
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs

def lengths(c, seed, lo, hi, n):
    r = random.Random(seed * 7919 + 17)
    return [r.randint(lo, hi) for _ in range(n)]


def blocks_of(page):
    return -(-page // 64)


def paged_tables(c, seed, lens):
    """Each sequence's pages drawn from one shuffled pool."""
    page = c["page"]
    g = torch.Generator(device=DEV).manual_seed(seed * 31 + 5)
    need = [-(-t // page) for t in lens]
    most = -(-c["t_hi"] // page)
    num = sum(need) + 3 if c["op"] == "attend" else len(lens) * most + 3   # outputs of one shape
    order = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, num, g


def random_codes(shape, g, spread):
    """e4m3 codes of N(0, spread^2) values, in pieces so that the floats stay small."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=g, device=DEV).mul_(spread).clamp_(-448, 448)
        flat[i:i + n] = x.to(F8).view(torch.uint8)
    return out


def prepare(case, seed):
    c = case
    if c["op"] == "attend":
        B, sq, H, G, D, page = (c[k] for k in ("B", "sq", "H", "G", "D", "page"))
        lens = lengths(c, seed, max(c["t_lo"], sq), c["t_hi"], B)
        table, num, g = paged_tables(c, seed, lens)
        s = {"case": c, "lens_host": lens, "table": table}
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = torch.randn(B, sq, H, D, generator=g, device=DEV).to(torch.bfloat16)
        # Values of about N(0, 1); the scales of neighbouring blocks differ.
        for x in ("k", "v"):
            s[x] = random_codes((num, G, page, D), g, 60.0)
            s[x + "s"] = (0.7 + 0.6 * torch.rand(num, G, blocks_of(page), generator=g, device=DEV)) / 60.0
        s["out"] = torch.empty(B, sq, H, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(B, sq, H, dtype=torch.float32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(D)
        return s
    if c["op"] == "append":
        B, sq, G, D, page = (c[k] for k in ("B", "sq", "G", "D", "page"))
        lens = lengths(c, seed, max(c["t_lo"], sq), c["t_hi"], B)
        table, num, g = paged_tables(c, seed, lens)
        s = {"case": c, "lens_host": lens, "table": table}
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        for x in ("k", "v"):
            # New tokens of unlike magnitudes, so that some outgrow their block's scale.
            size = torch.exp2(torch.randn(B, sq, G, 1, generator=g, device=DEV))
            s[x + "_new"] = (torch.randn(B, sq, G, D, generator=g, device=DEV) * size).to(torch.bfloat16)
            s[x] = random_codes((num, G, page, D), g, 80.0)
            s[x + "s"] = torch.exp2(torch.randint(-8, -5, (num, G, blocks_of(page)), generator=g,
                                                  device=DEV).float())
        return s
    return prepare_pages(c, seed)


def prepare_pages(c, seed):
    B, beams, page, num, layers = (c[k] for k in ("B", "beams", "page", "num_pages", "layers"))
    G, D = c["G"], c["D"]
    r = random.Random(seed * 104729 + 3)
    g = torch.Generator(device=DEV).manual_seed(seed * 31 + 5)
    ids = list(range(num))
    r.shuffle(ids)
    most = c["t_hi"] // page + 2
    rows, lens = [], []
    # Beams of a group share their full pages, as earlier forks left them; each
    # has its own last, partly filled page.
    for b in range(B // beams):
        t = r.randint(max(1, c["t_hi"] // 2), c["t_hi"])
        shared = [ids.pop() for _ in range(t // page)]
        for _ in range(beams):
            last = [ids.pop()] if t % page else []
            rows.append(shared + last)
            lens.append(t)
    table = torch.tensor([x + [-1] * (most - len(x)) for x in rows], dtype=torch.int32)
    refs = torch.zeros(num, dtype=torch.int32)
    for x in rows:
        refs[torch.tensor(x, dtype=torch.long)] += 1
    s = {"case": c, "table": table.to(DEV), "refs": refs.to(DEV),
         "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if layers:
        width = 2 if c["kind"] == "bf16" else 1
        data = torch.randint(0, 256, (2 * layers, num, G * page * D * width), generator=g, device=DEV,
                             dtype=torch.uint8)
        s["data"] = data if width == 1 else data.view(torch.int16)
        s["pools"] = [s["data"].view(2 * layers, num, G, page, D)]     # one tensor for all layers
        if c["kind"] == "fp8":
            s["scales"] = torch.randint(-9, -4, (2 * layers, num, G, blocks_of(page)), generator=g,
                                        device=DEV).float().exp2()
            s["pools"].append(s["scales"])
    s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    s["lens_out"] = torch.empty_like(s["lens"])
    s["counts"] = torch.empty(2, dtype=torch.int32, device=DEV)
    if c["op"] == "fork":
        # Each beam of a group goes on from the one that the search chose.
        src = [b - b % beams + r.randrange(beams) for b in range(B)]
        s["src"] = torch.tensor(src, dtype=torch.int32, device=DEV)
    if c["op"] == "turnover":
        grow = [t + r.choice([1, 1, 1, page]) for t in lens]
        s["grown"] = torch.tensor(grow, dtype=torch.int32, device=DEV)
        s["done"] = torch.tensor([r.random() < 0.1 for _ in lens], device=DEV)
    return s


# -------------------------------------------------------------------- passes

def run(state):
    c = state["case"]
    if c["op"] == "attend":
        return run_attend(state)
    if c["op"] == "append":
        return run_append(state)
    if c["op"] == "fork":
        return run_fork(state)
    if c["op"] == "compact":
        return run_compact(state)
    return run_turnover(state)


def run_attend(s):
    if own:
        import grouped_query_decode_gb300 as gq
        gq.gqa_decode_paged_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"],
                                s["out"], s["lse"])
        return s["out"], s["lse"]
    c = s["case"]
    B, sq, H, G, D, page = (c[k] for k in ("B", "sq", "H", "G", "D", "page"))
    n = H // G
    for b, T in enumerate(s["lens_host"]):
        at = s["table"][b, :-(-T // page)].long()
        k, v = (rows_of(s[x], s[x + "s"], at, page)[:, :T] for x in ("k", "v"))
        q = s["q"][b].float().view(sq, G, n, D).permute(1, 2, 0, 3).reshape(G, n * sq, D)
        x = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
        x = x.view(G, n, sq, T)
        if sq > 1:
            t = torch.arange(T, device=DEV)
            last = T - sq + torch.arange(sq, device=DEV)
            x = x.masked_fill(t[None, :] > last[:, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(G, n * sq, T), v).view(G, n, sq, D) / l
        s["out"][b] = o.permute(2, 0, 1, 3).reshape(sq, H, D).to(torch.bfloat16)
        s["lse"][b] = (m + torch.log(l))[..., 0].permute(2, 0, 1).reshape(sq, H)
    return s["out"], s["lse"]


def rows_of(codes, scales, at, page):
    """The pages `at` of one sequence as [G, tokens, D] values."""
    x = codes[at].view(F8).float()                              # [pages, G, page, D]
    x = x * scales[at].repeat_interleave(min(64, page), dim=2)[..., None]
    return x.transpose(0, 1).flatten(1, 2)


def scale_for(top):
    """The smallest power of two e with top <= 448 * 2^e (0 for 0)."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp_min(-126)
    return torch.where(top > 0, ((e + 127) << 23).view(torch.float32), torch.zeros_like(top))


def run_append(s):
    if own:
        import grouped_query_decode_gb300 as gq
        gq.gqa_append_paged_fp8(s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"])
        return s["k"].view(F8), s["v"].view(F8), s["ks"], s["vs"]
    c = s["case"]
    sq, G, D, page = (c[k] for k in ("sq", "G", "D", "page"))
    size = min(64, page)
    start = (s["lens"] - sq).long()                              # [B], the first new token
    count = (sq + size - 2) // size + 1                          # blocks that may take new tokens
    block = (start // size)[:, None] + torch.arange(count, device=DEV)
    row, _ = touched = (block * size < s["lens"][:, None]).nonzero(as_tuple=True)
    block = block[touched]                                       # [n] blocks that do
    at = s["table"][row, block * size // page].long()
    sub = block * size % page // size
    i = block[:, None] * size + torch.arange(size, device=DEV) - start[row][:, None]     # [n, size] new tokens
    is_new, is_kept = ((i >= 0) & (i < sq))[:, None, :, None], (i < 0)[:, None, :, None]
    for x in ("k", "v"):
        new = s[x + "_new"][row[:, None], i.clamp(0, sq - 1)].float().transpose(1, 2)    # [n, G, size, D]
        new = torch.where(is_new, new, 0.0)
        top = new.abs().amax((2, 3))
        codes = s[x].view(-1, G, page // size, size, D)
        codes_were, was = codes[at, :, sub], s[x + "s"][at, :, sub]
        old = torch.where(is_kept.any(2)[:, :, 0], was, 0.0)
        scale = torch.where((old > 0) & (top <= 448 * old), old, scale_for(top))
        div = torch.where(scale > 0, scale, 1.0)
        moved = (codes_were.view(F8).float() * (old / div)[..., None, None]).to(F8).view(torch.uint8)
        moved = torch.where((old == scale)[..., None, None], codes_were, moved)
        made = (new / div[..., None, None]).to(F8).view(torch.uint8)
        made = torch.where(is_new, made, torch.where(is_kept, moved, codes_were))
        codes[at, :, sub] = made
        s[x + "s"][at, :, sub] = scale
    return s["k"].view(F8), s["v"].view(F8), s["ks"], s["vs"]


def run_fork(s):
    c = s["case"]
    page = c["page"]
    if own:
        import grouped_query_decode_gb300 as gq
        gq.gqa_pages_fork(s["pools"], s["src"], s["table"], s["lens"], s["refs"], page, s["table_out"],
                          s["lens_out"], s["refs_out"], s["counts"], page_dim=1)
    else:
        src, table, refs = s["src"].long(), s["table"], s["refs"]
        B, most = table.shape
        row = torch.arange(B, device=DEV)
        # The lowest row that goes on from a sequence keeps its last page.
        first = (src[:, None] == src[None, :]).int().argmax(1) == row
        lens = s["lens"][src]
        full, part = lens // page, lens % page
        copies = (~first & (part > 0)).nonzero()[:, 0]
        free = (refs == 0).nonzero()[:, 0]
        s["counts"].copy_(torch.tensor([copies.numel(), free.numel()], dtype=torch.int32))
        new = free[:copies.numel()]
        old = table[src[copies], full[copies].long()].long()
        out = table[src].clone()
        j = torch.arange(most, device=DEV)
        out[~first[:, None] & (j[None, :] >= full[:, None])] = -1
        out[copies, full[copies].long()] = new.to(torch.int32)
        for pool in s["pools"]:
            pool[:, new] = pool[:, old]
        count = refs.clone()
        count.index_add_(0, table[table >= 0].long(), torch.full_like(table[table >= 0], -1))
        count.index_add_(0, out[out >= 0].long(), torch.ones_like(out[out >= 0]))
        s["table_out"].copy_(out)
        s["lens_out"].copy_(lens)
        s["refs_out"].copy_(count)
    return (s["data"], s["scales"] if "scales" in s else s["lens"], s["table_out"], s["lens_out"],
            s["refs_out"], s["counts"])


def run_compact(s):
    if own:
        import grouped_query_decode_gb300 as gq
        gq.gqa_pages_compact(s["pools"], s["table"], s["refs"], s["table_out"], s["refs_out"], s["counts"],
                             page_dim=1)
    else:
        table, refs = s["table"], s["refs"]
        live = int((refs > 0).sum())
        holes = (refs[:live] == 0).nonzero()[:, 0]
        moved = (refs[live:] > 0).nonzero()[:, 0] + live
        to = torch.arange(refs.numel(), device=DEV)
        to[moved] = holes
        for pool in s["pools"]:
            pool[:, holes] = pool[:, moved]
        s["table_out"].copy_(torch.where(table >= 0, to[table.clamp_min(0).long()].to(torch.int32), table))
        s["refs_out"].copy_(refs)
        s["refs_out"][holes] = refs[moved]
        s["refs_out"][live:] = 0
        s["counts"].copy_(torch.tensor([moved.numel(), live], dtype=torch.int32))
    return s["data"], s["scales"], s["table_out"], s["refs_out"], s["counts"]


def run_turnover(s):
    c = s["case"]
    page = c["page"]
    table, lens, refs = s["table_out"], s["lens_out"], s["refs_out"]
    table.copy_(s["table"])          # the two calls work in place
    refs.copy_(s["refs"])
    lens.copy_(s["grown"])
    if own:
        import grouped_query_decode_gb300 as gq
        gq.gqa_pages_reserve(table, lens, refs, page, s["counts"])
        gq.gqa_pages_free(s["done"], table, lens, refs)
    else:
        want = (lens + page - 1) // page
        empty = (torch.arange(table.shape[1], device=DEV)[None, :] < want[:, None]) & (table < 0)
        free = (refs == 0).nonzero()[:, 0]
        rank = empty.flatten().cumsum(0) - 1
        s["counts"].copy_(torch.tensor([int(empty.sum()), free.numel()], dtype=torch.int32))
        got = free[rank.clamp(0, free.numel() - 1)].view_as(table)
        table.copy_(torch.where(empty, got.to(torch.int32), table))
        refs[got[empty]] = 1
        gone = table[s["done"]]
        gone = gone[gone >= 0].long()
        refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
        table[s["done"]] = -1
        lens[s["done"]] = 0
    return table, lens, refs, s["counts"]


# --------------------------------------------------------------------- work

def work(case):
    c = case
    G, D, page = c["G"], c["D"], c["page"]
    if c["op"] in ("attend", "append"):
        tokens = c["B"] * (max(c["t_lo"], c["sq"]) + c["t_hi"]) / 2
        if c["op"] == "attend":
            rows = c["B"] * c["sq"] * c["H"]
            kv = 2 * tokens * G * (D + 4 / min(64, page))
            return {"bytes": kv + rows * (4 * D + 4) + 4 * tokens / page,
                    "flops": 4.0 * tokens * c["sq"] * c["H"] * D}
        new = c["B"] * c["sq"] * G
        return {"bytes": 2 * new * (3 * D + 4 / min(64, page)), "flops": 2.0 * new * D * 3}
    table = 4.0 * c["B"] * (c["t_hi"] // page + 2)
    refs = 4.0 * c["num_pages"]
    width = 2 if c["kind"] == "bf16" else 1
    one = 2 * c["layers"] * (G * page * D * width + (4 * G * blocks_of(page) if c["kind"] == "fp8" else 0))
    if c["op"] == "fork":
        # Of k beams that draw from k, k (1 - 1/k)^k are not drawn and as many go on from a copy.
        k = c["beams"]
        return {"bytes": 2 * one * c["B"] * (1 - 1 / k) ** k * (1 - 1 / page) + 2 * table + 2 * refs, "flops": 0}
    if c["op"] == "compact":
        live = min(c["num_pages"], c["B"] * 0.75 * c["t_hi"] / page)
        return {"bytes": 2 * one * live * (1 - live / c["num_pages"]) + 2 * table + 2 * refs, "flops": 0}
    return {"bytes": 2 * table + 2 * refs, "flops": 0}


# -------------------------------------------------------------------- exact

def values64(codes):
    """e4m3 codes to float64 by their definition: 1 sign, 4 exponent (bias 7), 3 mantissa bits."""
    i = codes.long()
    e, m = (i >> 3) & 15, (i & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    x = torch.where((i & 127) == 127, torch.full_like(x, math.nan), x)
    return torch.where(i >= 128, -x, x)


def nearest_code(x):
    """float64 values of magnitude <= 448 rounded to e4m3 (ties to even), as float64."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    e = torch.where(x.abs() >= torch.exp2(e + 1), e + 1, e)      # log2's own rounding
    e = torch.where((x.abs() < torch.exp2(e)) & (e > -6), e - 1, e)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def power_of_two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def exact(case, seed):
    c = case
    if c["op"] == "attend":
        return exact_attend(c, seed)
    if c["op"] == "append":
        return exact_append(c, seed)
    return None


def exact_attend(c, seed):
    s = prepare(c, seed)
    B, sq, H, G, D, page = (c[k] for k in ("B", "sq", "H", "G", "D", "page"))
    n, size = H // G, min(64, page)
    out = torch.empty(B, sq, H, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, sq, H, dtype=torch.float64, device=DEV)
    for b, T in enumerate(s["lens_host"]):
        t = torch.arange(T, device=DEV)
        at, within = s["table"][b].long()[t // page], t % page
        seen = t[None, :] <= (T - sq + torch.arange(sq, device=DEV))[:, None]      # [sq, T]
        for g in range(G):
            k = values64(s["k"][at, g, within]) * s["ks"][at, g, within // size].double()[:, None]
            v = values64(s["v"][at, g, within]) * s["vs"][at, g, within // size].double()[:, None]
            for h in range(g * n, (g + 1) * n):
                x = s["q"][b, :, h].double() @ k.T * s["scale"]
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                z = torch.logsumexp(x, 1)
                lse[b, :, h] = z
                out[b, :, h] = torch.exp(x - z[:, None]) @ v
    return out, lse


def exact_append(c, seed):
    s = prepare(c, seed)
    sq, G, page = c["sq"], c["G"], c["page"]
    size = min(64, page)
    result = []
    for x in ("k", "v"):
        values, scales = values64(s[x]), s[x + "s"].double()
        for b, T in enumerate(s["lens_host"]):
            new = s[x + "_new"][b].double()
            for block in range((T - sq) // size, (T - 1) // size + 1):
                lo, hi = max(block * size, T - sq), min((block + 1) * size, T)
                p = int(s["table"][b, block * size // page])
                j, off = block * size % page // size, block * size % page
                top = new[lo - T + sq:hi - T + sq].abs().amax((0, 2))               # [G]
                want = power_of_two(torch.frexp((top / 448) * (1 - 2.0 ** -40))[1])         # at least top / 448
                old = scales[p, :, j].clone()
                held = lo - block * size
                if held:
                    want = torch.where(top <= 448 * old, old, want)
                    r = (old / want)[:, None, None]
                    values[p, :, off:off + held] = nearest_code(values[p, :, off:off + held] * r)
                made = new[lo - T + sq:hi - T + sq].transpose(0, 1) / want[:, None, None]
                values[p, :, off + held:off + held + hi - lo] = nearest_code(made)
                scales[p, :, j] = want
        result.append((values, scales))
    (kv, ks), (vv, vs) = result
    return kv, vv, ks, vs
