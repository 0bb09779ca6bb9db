"""Times of packed batches over a bf16 cache: rotary positions, the append of new
tokens to pages (rotated on the way), and the attention of whole prompts and of
chunks over pages, beside their plain forms in elementary torch.

New tokens of all sequences lie behind one another, [N, heads, D]; those of
sequence b are rows cu[b] to cu[b + 1]. Rows behind the last sequence are left
as they are. Pages are [num_pages, G, page_size, D], reached through a block
table [B, max_pages]; lens[b] counts a sequence's tokens, the new ones included.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
I32 = torch.int32
LARGEST_FLOPS = 2.2e12        # of the largest listed case
LARGEST_BYTES = 2.2e9         # of a drawn case's cache


# ------------------------------------------------------------------- cases

def listed():
    return [
        # The new tokens of 64 sequences in a decode step: latency.
        rope("rope_step", 64, 32, 8, 128, 128, False, "none", 8192),
        # A 16384-token batch of prompts, half of each head rotated in pairs of
        # neighbours, positions of a context that was lengthened.
        rope("rope_prompts_part", 16384, 32, 8, 128, 64, True, "yarn", 1 << 20),
        # The same step's keys and values rotated and written to their pages.
        append("append_step_p16", 64, 32, 8, 128, 1, 1, 2048, 16, 128, False, "none"),
        # Chunks of six prompts.
        append("append_chunks_p64", 6, 32, 8, 128, 300, 2048, 8192, 64, 128, False, "bands"),
        # One short question to a small model: latency.
        packed("packed_tiny_d64", 1, 32, 8, 64, 17, 17),
        # Equal prompts, every head with a KV head of its own.
        packed("packed_mha_d64", 8, 16, 16, 64, 1024, 1024),
        # A batch of prompts of any length, the layer of an 8B model.
        packed("packed_ragged", 24, 32, 8, 128, 16, 4096),
        # One long document: the matrix products' rate.
        packed("packed_long", 1, 32, 8, 128, 16384, 16384),
        # A decode step over the shortest pages: the cache's bytes.
        paged("paged_step_p16", 64, 32, 8, 128, 1, 1, 1.0, 512, 16384, 16, 0),
        # A long prompt's last chunk.
        paged("paged_chunk_p64", 1, 32, 8, 128, 2048, 2048, 0.0, 32768, 32768, 64, 0),
        # A serving step: single tokens of running sequences and chunks of the
        # prompts that joined, in a batch padded to a captured size.
        paged("paged_mixed_p32", 48, 32, 8, 128, 1, 1024, 0.85, 64, 8192, 32, 37),
        # Seven speculative tokens of a multi-query model.
        paged("paged_spec_mqa_d64", 16, 24, 1, 64, 7, 7, 0.0, 1024, 8192, 128, 0),
    ]


def rope(name, N, H, G, D, dims, pairs, scaling, t_hi):
    return dict(name=name, op="rope", N=N, H=H, G=G, D=D, dims=dims, pairs=pairs, scaling=scaling, t_hi=t_hi)


def append(name, B, H, G, D, n_lo, n_hi, t_hi, page, dims, pairs, scaling):
    return dict(name=name, op="append", B=B, H=H, G=G, D=D, n_lo=n_lo, n_hi=n_hi, singles=0.0, t_lo=n_hi, t_hi=t_hi,
                page=page, dims=dims, pairs=pairs, scaling=scaling, pad=0)


def packed(name, B, H, G, D, n_lo, n_hi):
    return dict(name=name, op="packed", B=B, H=H, G=G, D=D, n_lo=n_lo, n_hi=n_hi, singles=0.0, t_lo=0, t_hi=0, pad=0)


def paged(name, B, H, G, D, n_lo, n_hi, singles, t_lo, t_hi, page, pad):
    return dict(name=name, op="paged", B=B, H=H, G=G, D=D, n_lo=n_lo, n_hi=n_hi, singles=singles, t_lo=t_lo,
                t_hi=t_hi, page=page, pad=pad)


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "packed", "packed", "packed", "paged", "paged", "paged"])
    D = rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 8, 16])
    H = G * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while H > 64:
        H, G = H // 2 // max(1, G // 2) * max(1, G // 2), max(1, G // 2)
    dims = rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)])
    pairs, scaling = rng.random() < 0.5, rng.choice(["none", "linear", "base", "bands", "yarn"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "rope":
        N = min(log_int(rng, 1, 32768), 100_000_000 // (H * D))
        c = rope("", N, H, G, D, dims, pairs, scaling, log_int(rng, 64, 1 << 20))
    elif op == "append":
        n_hi = log_int(rng, 1, 4096)
        n_lo = rng.choice([1, n_hi, (n_hi + 1) // 2])
        t_hi = max(n_hi, log_int(rng, 16, 8192))
        B = log_int(rng, 1, max(1, min(128, 16384 // n_hi, int(5e8) // (4 * G * D * (t_hi + page)))))
        c = append("", B, H, G, D, n_lo, n_hi, t_hi, page, dims, pairs, scaling)
    elif op == "packed":
        n_hi = log_int(rng, 1, 16384)
        n_lo = rng.choice([1, n_hi, (n_hi + 1) // 2])
        B = log_int(rng, 1, max(1, min(64, 32768 // n_hi)))
        c = packed("", B, H, G, D, n_lo, n_hi)
    else:
        n_hi = rng.choice([1, 1, 2, 5, 16, log_int(rng, 1, 4096)])
        n_lo = rng.choice([1, n_hi])
        t_hi = max(n_hi, log_int(rng, 16, 65536))
        t_lo = max(1, int(t_hi * rng.choice([1.0, 0.5, 0.02])))
        B = log_int(rng, 1, max(1, min(96, int(LARGEST_BYTES) // (4 * G * D * (t_hi + page)), 65536 // n_hi)))
        c = paged("", B, H, G, D, n_lo, n_hi, rng.choice([0.0, 0.5, 0.9]), t_lo, t_hi, page, rng.choice([0, 0, 5]))
    while op in ("packed", "paged") and (work(c)["flops"] > LARGEST_FLOPS or work(c)["bytes"] > LARGEST_BYTES):
        if c["B"] > 1:
            c["B"] //= 2
        else:
            c["n_hi"] = max(1, c["n_hi"] // 2)
            c["n_lo"] = min(c["n_lo"], c["n_hi"])
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs

def lengths(c):
    """(new tokens, all tokens) of each sequence, the same for every seed; new
    tokens are spread over their logarithm where they differ."""
    r = random.Random("%s %s %s %s %s %s" % tuple(c[k] for k in ("B", "n_lo", "n_hi", "singles", "t_lo", "t_hi")))
    got = []
    for b in range(c["B"]):
        n = 1 if r.random() < c["singles"] else log_int(r, c["n_lo"], c["n_hi"])
        if b == 0:
            n = c["n_hi"]
        T = n if c["op"] == "packed" else max(n, r.randint(min(c["t_lo"], c["t_hi"]), c["t_hi"]))
        got.append((n, T))
    return got


def rope_of(c):
    """Base, and what a lengthened context changes, as a model's configuration
    names them: the factor, the original context, and the turns that a pair makes
    over it below which it is slowed by the factor, and above which it is left."""
    kind = c["scaling"]
    return dict(base=10000.0 if kind in ("none", "linear", "base") else 500000.0, scaling=kind,
                factor=1.0 if kind == "none" else 8.0, original=8192, low=1.0, high=32.0 if kind == "yarn" else 4.0)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed * 31 + 5)
    H, G, D = c["H"], c["G"], c["D"]
    s = {"case": c}
    if own and c["op"] in ("rope", "append"):
        import grouped_query_decode_gb300 as gq
        s["rope"] = gq.gqa_rope_init(D, dims=c["dims"], interleaved=c["pairs"], **rope_of(c))
    if c["op"] == "rope":
        N = c["N"]
        s["positions"] = torch.randint(0, c["t_hi"], (N,), generator=g, device=DEV, dtype=I32)
        fused(s, N, g)
        s["q_out"], s["k_out"] = (torch.zeros(N, h, D, dtype=BF, device=DEV) for h in (H, G))
        return s
    lens = lengths(c)
    random.Random(seed).shuffle(lens)
    s["lens_host"] = lens
    new = [n for n, _ in lens]
    N = sum(new) + c["pad"]
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    s["cu_host"], s["cu"] = at, torch.tensor(at, dtype=I32, device=DEV)
    s["scale"] = 1.0 / math.sqrt(D)
    if c["op"] != "paged":
        fused(s, N, g)
    else:
        s["q"] = torch.randn(N, H, D, generator=g, device=DEV).to(BF)
    if c["op"] != "packed":
        page = c["page"]
        need = [-(-T // page) for _, T in lens]
        num = sum(need) + 3
        order = torch.randperm(num, generator=g, device=DEV).to(I32)
        s["table"] = torch.full((c["B"], max(need)), -1, dtype=I32, device=DEV)
        first = 0
        for b, n in enumerate(need):
            s["table"][b, :n] = order[first:first + n]
            first += n
        s["lens"] = torch.tensor([T for _, T in lens], dtype=I32, device=DEV)
        for x in ("k_pages", "v_pages"):
            s[x] = torch.empty(num, G, page, D, dtype=BF, device=DEV)
            for i in range(0, num, 4096):
                s[x][i:i + 4096] = torch.randn(s[x][i:i + 4096].shape, generator=g, device=DEV).to(BF)
    if c["op"] == "append":
        s["q_out"] = torch.zeros(N, H, D, dtype=BF, device=DEV)
    else:
        s["out"] = torch.zeros(N, H, D, dtype=BF, device=DEV)
        s["lse"] = torch.zeros(N, H, dtype=torch.float32, device=DEV)
    return s


def fused(s, N, g):
    """Queries, keys and values as one projection leaves them: views of its rows."""
    H, G, D = (s["case"][k] for k in "HGD")
    x = torch.randn(N, H + 2 * G, D, generator=g, device=DEV).to(BF)
    s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + G], x[:, H + G:]


# -------------------------------------------------------------------- passes

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import grouped_query_decode_gb300 as gq
        if op == "rope":
            gq.gqa_rope(s["rope"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"])
        elif op == "append":
            gq.gqa_append_paged(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"],
                                rope=s["rope"], q=s["q"], q_out=s["q_out"])
        elif op == "packed":
            gq.gqa_prefill_packed(s["q"], s["k"], s["v"], s["cu"], s["scale"], s["out"], s["lse"])
        else:
            gq.gqa_prefill_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], s["scale"],
                                 s["out"], s["lse"])
    elif op == "rope":
        plain_rope(s)
    elif op == "append":
        plain_append(s)
    else:
        plain_attention(s)
    if op == "rope":
        return s["q_out"], s["k_out"]
    if op == "append":
        return s["q_out"], s["k_pages"], s["v_pages"]
    return s["out"], s["lse"]


def frequencies(c):
    """Radians per position of every pair (float64), and the factor on sine and cosine."""
    r, n = rope_of(c), c["dims"]
    i = torch.arange(0, n, 2, dtype=torch.float64)
    base, factor, kind = r["base"], r["factor"], r["scaling"]
    if kind == "base" and n > 2:
        base *= factor ** (n / (n - 2))
    f = base ** (-i / n)
    if kind == "linear":
        f = f / factor
    if kind == "bands":
        turns = r["original"] * f / (2 * math.pi)
        keep = ((turns - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    if kind == "yarn":
        def pair(turns):                       # the pair that makes so many turns over the original context
            return n * math.log(r["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(r["high"])), 0), min(math.ceil(pair(r["low"])), n - 1)
        slow = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * slow + f * (1 - slow)
    return f.to(DEV), 1 + 0.1 * math.log(factor) if kind == "yarn" else 1.0


def rotate(x, angle, gain, pairs):
    """The first 2 * angle.shape[1] elements of every head of x [N, heads, D], rotated."""
    h = angle.shape[1]
    cos, sin = (torch.cos(angle) * gain).float()[:, None], (torch.sin(angle) * gain).float()[:, None]
    y = x.float().clone()
    a, b = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if pairs else (y[..., :h], y[..., h:2 * h])
    a_new, b_new = a * cos - b * sin, b * cos + a * sin
    a.copy_(a_new)
    b.copy_(b_new)
    return y.to(BF)


def plain_rope(s):
    c = s["case"]
    f, gain = frequencies(c)
    angle = s["positions"].double()[:, None] * f[None, :]
    s["q_out"].copy_(rotate(s["q"], angle, gain, c["pairs"]))
    s["k_out"].copy_(rotate(s["k"], angle, gain, c["pairs"]))


def plain_append(s):
    c = s["case"]
    f, gain = frequencies(c)
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(c["B"], device=DEV), n)
    at = s["lens"].long()[b] - n[b] + torch.arange(b.numel(), device=DEV) - cu[b]
    angle = at.double()[:, None] * f[None, :]
    total = b.numel()
    s["q_out"][:total] = rotate(s["q"][:total], angle, gain, c["pairs"])
    p = s["table"][b, at // c["page"]].long()
    s["k_pages"][p, :, at % c["page"]] = rotate(s["k"][:total], angle, gain, c["pairs"])
    s["v_pages"][p, :, at % c["page"]] = s["v"][:total]


def plain_attention(s):
    c = s["case"]
    H, G, D = c["H"], c["G"], c["D"]
    r = H // G
    for b, (n, T) in enumerate(s["lens_host"]):
        i = s["cu_host"][b]
        if c["op"] == "packed":
            k, v = (s[x][i:i + n].float().transpose(0, 1) for x in ("k", "v"))              # [G, T, D]
        else:
            at = s["table"][b, :-(-T // c["page"])].long()
            k, v = (s[x][at].float().transpose(0, 1).flatten(1, 2)[:, :T] for x in ("k_pages", "v_pages"))
        t = torch.arange(T, device=DEV)
        most = max(1, (1 << 29) // (H * T))
        for j in range(0, n, most):
            m = min(most, n - j)
            q = s["q"][i + j:i + j + m].float().view(m, G, r, D).permute(1, 2, 0, 3).reshape(G, r * m, D)
            x = (torch.matmul(q, k.transpose(1, 2)) * s["scale"]).view(G, r, m, T)
            if n > 1:
                last = T - n + j + torch.arange(m, device=DEV)
                x = x.masked_fill(t[None, :] > last[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            l = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(G, r * m, T), v).view(G, r, m, D) / l
            s["out"][i + j:i + j + m] = o.permute(2, 0, 1, 3).reshape(m, H, D).to(BF)
            s["lse"][i + j:i + j + m] = (top + torch.log(l))[..., 0].permute(2, 0, 1).reshape(m, H)


# --------------------------------------------------------------------- work

def work(case):
    c = case
    H, G, D = c["H"], c["G"], c["D"]
    if c["op"] == "rope":
        return {"bytes": c["N"] * (4.0 * (H + G) * D + 4), "flops": 3.0 * c["N"] * (H + G) * c["dims"]}
    lens = lengths(c)
    new = sum(n for n, _ in lens)
    if c["op"] == "append":
        return {"bytes": 4.0 * new * (H + 2 * G) * D + 12 * c["B"], "flops": 3.0 * new * (H + G) * c["dims"]}
    seen = sum(n * T - n * (n - 1) / 2 for n, T in lens)          # (query, key) pairs of a head
    held = sum(T for _, T in lens)
    return {"bytes": new * H * (4.0 * D + 4) + 4.0 * held * G * D + 4.0 * (c["B"] + 1), "flops": 4.0 * seen * H * D}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    c = case
    if c["op"] in ("packed", "paged") and work(c)["flops"] > 4e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "rope":
        return tuple(turned(s[x], s["positions"], c) for x in ("q", "k"))
    if c["op"] == "append":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        for b, (n, T) in enumerate(s["lens_host"]):
            i = s["cu_host"][b]
            t = torch.arange(T - n, T, device=DEV)
            out[i:i + n] = turned(s["q"][i:i + n], t, c)
            k, v = turned(s["k"][i:i + n], t, c), s["v"][i:i + n].double()
            for j in range((T - n) // c["page"], (T - 1) // c["page"] + 1):
                p = int(s["table"][b, j])
                here = (t // c["page"] == j).nonzero()[:, 0]
                slot = t[here] % c["page"]
                kp[p].index_copy_(1, slot, k[here].transpose(0, 1))
                vp[p].index_copy_(1, slot, v[here].transpose(0, 1))
        return out, kp, vp
    return exact_attention(s)


def turned(x, t, c):
    """Pairs as complex numbers times gain * e^(i t f)."""
    f, gain = frequencies(c)
    h = f.numel()
    y = x.double().clone()
    first = slice(0, 2 * h, 2) if c["pairs"] else slice(0, h)
    second = slice(1, 2 * h, 2) if c["pairs"] else slice(h, 2 * h)
    turn = torch.polar(torch.full((t.numel(), h), gain, dtype=torch.float64, device=DEV), t.double()[:, None] * f)
    z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact_attention(s):
    c = s["case"]
    H, G, D = c["H"], c["G"], c["D"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b, (n, T) in enumerate(s["lens_host"]):
        i = s["cu_host"][b]
        pos = torch.arange(T, device=DEV)
        for g in range(G):
            if c["op"] == "packed":
                k, v = s["k"][i:i + n, g].double(), s["v"][i:i + n, g].double()
            else:
                p, slot = s["table"][b].long()[pos // c["page"]], pos % c["page"]
                k, v = s["k_pages"][p, g, slot].double(), s["v_pages"][p, g, slot].double()
            for h in range(g * (H // G), (g + 1) * (H // G)):
                for j in range(0, n, 2048):
                    q = s["q"][i + j:min(i + j + 2048, i + n), h].double()
                    see = T - n + j + q.shape[0]                           # keys that the block's last row sees
                    x = q @ k[:see].T * s["scale"]
                    x = torch.where(pos[None, :see] <= T - n + j + torch.arange(q.shape[0], device=DEV)[:, None], x,
                                    torch.full_like(x, -math.inf))
                    z = torch.logsumexp(x, 1)
                    out[i + j:i + j + q.shape[0], h] = torch.exp(x - z[:, None]) @ v[:see]
                    lse[i + j:i + j + q.shape[0], h] = z
    return out, lse
