"""Cases of the paged KV-cache operators: append (bf16 and FP8), read-back, and attention of a chunk of new tokens.

A batch of B sequences brings T packed new tokens, n_b of them for sequence b (``cu``: their prefix sums).  ``lens[b]``
counts the rows of sequence b with its new tokens, so token i of sequence b stands at position lens[b] - n_b + i.  Row r
of a sequence is row r % page of the page ``table[b, r // page]``; pages are [n_pages, Hk, page, d], the FP8 ones with one
fp32 scale per row ([n_pages, Hk, page]).

``run`` computes an operator from elementary torch operations in fp32, or, where ``own`` is set, through the library.
"""
import random

import torch

own = False

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


# ---- cases ---------------------------------------------------------------------------------------------------------


def listed():
    def case(name, op, B, n, ctx, H, Hk, d, page, layout, ones=0, pair=0):
        return dict(name=name, op=op, B=B, n_lo=n[0], n_hi=n[1], ctx_lo=ctx[0], ctx_hi=ctx[1], ones=ones, H=H, Hk=Hk,
                    d=d, page=page, pair=pair, layout=layout)
    return [
        # one decode step's rows of a serving batch go into their pages: a few KB, latency alone
        case("append_step", "append", 16, (1, 1), (1023, 8191), 32, 8, 128, 64, 1),
        # two long prompts, one of odd length, filling fresh pages
        case("append_prompts", "append", 2, (5003, 8192), (0, 0), 32, 8, 128, 64, 2),
        # the smallest FP8 append: one sequence, one token, small heads, half-split rotation
        case("append_fp8_token", "append_fp8", 1, (1, 1), (256, 256), 8, 2, 64, 16, 3, pair=1),
        # chunks of a busy server quantised as they are written, behind rows already cached
        case("append_fp8_chunks", "append_fp8", 12, (700, 2048), (0, 6000), 64, 8, 128, 32, 4),
        # a short prefix read back before it is continued elsewhere
        case("read_fp8_prefix", "read_fp8", 3, (1, 1), (100, 700), 8, 2, 64, 16, 5),
        # a batch of long sequences brought back to a contiguous bf16 cache
        case("read_fp8_long", "read_fp8", 8, (1, 1), (9000, 32767), 64, 8, 128, 64, 6),
        # decode over ragged lengths, pages of 64: the batch of the benchmark's headline
        case("chunk_decode", "attn", 16, (1, 1), (1023, 8191), 32, 8, 128, 64, 7),
        # two prompts continued by up to 4096 tokens behind 4096 cached ones: tensor-core work
        case("chunk_prefill", "attn", 2, (3001, 4096), (4096, 4096), 32, 8, 128, 128, 8),
        # a server's mixed batch: eight decoding sequences beside two chunks of prompts, pages of 16
        case("chunk_mixed", "attn", 10, (500, 1000), (300, 7000), 32, 8, 128, 16, 9, ones=8),
        # the smallest call: a few guessed tokens checked against a short cache, small heads
        case("chunk_fp8_few", "attn_fp8", 2, (4, 5), (200, 251), 8, 2, 64, 16, 10),
        # decode of a batch at 32K tokens from an FP8 cache: half the bytes
        case("chunk_fp8_decode", "attn_fp8", 16, (1, 1), (32767, 32767), 64, 8, 128, 64, 11),
        # a chunk of one long sequence, every head on one KV head, FP8
        case("chunk_fp8_long", "attn_fp8", 1, (1021, 1021), (31000, 31000), 64, 1, 128, 32, 12),
    ]


#: A drawn case stays below the largest listed one in FLOPs and bytes, and in what its plain form holds.
MOST_FLOPS, MOST_BYTES, MOST_SCORES, MOST_ROWS = 7.0e11, 1.1e9, 6.0e8, 6.0e8


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random())) if hi > lo else lo
    while True:
        op = rng.choice(["append", "append_fp8", "read_fp8", "attn", "attn", "attn_fp8", "attn_fp8"])
        H, Hk = rng.choice([(32, 8), (32, 8), (64, 8), (8, 2), (64, 1), (16, 16), (8, 1), (32, 2), (4, 4)])
        B = log(1, 24)
        n_hi = 1 if op == "read_fp8" else rng.choice([1, log(2, 12), log(13, 4096)])
        ctx_hi = rng.choice([0, log(1, 300), log(300, 32767), log(1000, 16384)])
        c = dict(op=op, B=B, n_lo=max(1, n_hi // rng.choice([1, 2, 5])), n_hi=n_hi,
                 ctx_lo=ctx_hi // rng.choice([1, 2, 9]), ctx_hi=ctx_hi,
                 ones=rng.randint(0, B - 1) if rng.random() < 0.3 else 0, H=H, Hk=Hk, d=rng.choice([64, 128, 128]),
                 page=rng.choice([16, 32, 64, 128]), pair=rng.choice([0, 1]), layout=rng.randint(100, 10 ** 6))
        ns, lens = _layout(c)
        w = work(c)
        rows = B * max(lens) * c["d"] * Hk
        scores = B * H * max(ns) * max(lens) if op.startswith("attn") else 0
        if w["flops"] <= MOST_FLOPS and w["bytes"] <= MOST_BYTES and rows <= MOST_ROWS and scores <= MOST_SCORES:
            return c


def _layout(c):
    """(new tokens, rows with them) of every sequence: a function of the case alone."""
    r = random.Random(c["layout"])
    ns = [1 if b < c["ones"] else r.randint(c["n_lo"], c["n_hi"]) for b in range(c["B"])]
    return ns, [n + r.randint(c["ctx_lo"], c["ctx_hi"]) for n in ns]


def work(c):
    ns, lens = _layout(c)
    T, L, H, Hk, d = sum(ns), sum(lens), c["H"], c["Hk"], c["d"]
    row = {"bf16": 2 * Hk * d * 2, "fp8": 2 * Hk * (d + 4)}  # bytes of a token's K and V
    if c["op"] == "append":
        return {"bytes": T * (2 * row["bf16"] + 4 * d), "flops": T * 3 * Hk * d}
    if c["op"] == "append_fp8":
        return {"bytes": T * (row["bf16"] + row["fp8"] + 4 * d), "flops": T * 7 * Hk * d}
    if c["op"] == "read_fp8":
        return {"bytes": L * (row["fp8"] + row["bf16"]), "flops": L * 2 * Hk * d}
    pairs = sum(n * (l - n) + n * (n + 1) // 2 for n, l in zip(ns, lens))
    return {"bytes": T * H * (4 * d + 4) + L * row["fp8" if c["op"] == "attn_fp8" else "bf16"],
            "flops": 4 * H * d * pairs}


# ---- inputs --------------------------------------------------------------------------------------------------------


def _quantised(x):
    """One scale per row of the last axis, absmax / 448, and the E4M3 codes of x / scale (fp32)."""
    s = x.abs().amax(-1) / 448.0
    y = x / torch.where(s > 0, s, 1.0)[..., None]
    return y.to(F8), s


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    ns, lens = _layout(c)
    B, H, Hk, d, page, T = c["B"], c["H"], c["Hk"], c["d"], c["page"], sum(ns)
    per = [-(-l // page) for l in lens]
    n_pages = sum(per) + 3  # a pool with a few pages free, handed out in no order
    order = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.zeros(B, max(per), dtype=torch.int32, device=dev)
    at = 0
    for b, p in enumerate(per):
        table[b, :p] = order[at:at + p]
        at += p
    s = dict(case=c, n_max=max(ns), L_max=max(lens), scale=d ** -0.5, table=table,
             cu=torch.tensor([sum(ns[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev),
             lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if c["op"] != "read_fp8":  # what a fused projection leaves: q, k and v of a token side by side
        qkv = torch.randn(T, (H + 2 * Hk) * d, generator=g, device=dev).to(BF16)
        s["q"] = qkv[:, :H * d].view(T, H, d)
        s["k"] = qkv[:, H * d:(H + Hk) * d].view(T, Hk, d)
        s["v"] = qkv[:, (H + Hk) * d:].view(T, Hk, d)
    fp8 = c["op"].endswith("fp8")
    for x in "kv":
        if c["op"].startswith("append"):  # zeroed pages, written by the call
            s[x + "_pages"] = torch.zeros(n_pages, Hk, page, d, dtype=torch.uint8 if fp8 else BF16, device=dev)
            if fp8:
                s[x + "_scales"] = torch.zeros(n_pages, Hk, page, device=dev)
        else:
            rows = torch.randn(n_pages, Hk, page, d, generator=g, device=dev)
            if fp8:  # tokens differ in size, as keys and values do
                rows *= torch.exp(0.5 * torch.randn(n_pages, Hk, page, 1, generator=g, device=dev))
                codes, s[x + "_scales"] = _quantised(rows)
                s[x + "_pages"] = codes.view(torch.uint8)
            else:
                s[x + "_pages"] = rows.to(BF16)
            del rows
    if c["op"].startswith("append"):
        i = torch.arange(d // 2, device=dev, dtype=torch.float64)
        a = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * 500000.0 ** (-2.0 * i / d)
        s["cos"], s["sin"] = torch.cos(a).float(), torch.sin(a).float()
    if c["op"] == "read_fp8":
        s["k_out"], s["v_out"] = (torch.zeros(B, Hk, max(lens), d, dtype=BF16, device=dev) for _ in range(2))
    return s


# ---- the operators -------------------------------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return _library(s, op)
    if op == "append":
        return _append(s)
    if op == "append_fp8":
        return _append_fp8(s)
    if op == "read_fp8":
        return _read_fp8(s)
    return _attention(s)


def _library(s, op):
    from mqa_kv_cache_b200 import kvattn as K
    c = s["case"]
    if op == "append":
        K.kv_append_paged_rope(s["k"], s["v"], s["cu"], s["lens"], s["table"], s["k_pages"], s["v_pages"], s["cos"],
                               s["sin"], pair_style=c["pair"])
        return s["k_pages"], s["v_pages"]
    if op == "append_fp8":
        K.kv_append_paged_rope_fp8(s["k"], s["v"], s["cu"], s["lens"], s["table"], s["k_pages"], s["k_scales"],
                                   s["v_pages"], s["v_scales"], s["cos"], s["sin"], pair_style=c["pair"])
        return s["k_pages"].view(F8), s["k_scales"], s["v_pages"].view(F8), s["v_scales"]
    if op == "read_fp8":
        K.kv_read_paged_fp8(s["k_pages"], s["k_scales"], s["v_pages"], s["v_scales"], s["table"], s["lens"],
                            s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if "ws" not in s:  # a program keeps one workspace for all its calls of a shape
        s["ws"] = K.workspace(K.attn_chunk_paged_workspace_bytes(c["B"], s["q"].shape[0], s["n_max"], c["H"], c["Hk"],
                                                                 c["d"]))
    if op == "attn":
        return K.attn_chunk_paged(s["q"], s["cu"], s["lens"], s["table"], s["k_pages"], s["v_pages"], s["scale"],
                                  max_q=s["n_max"], ws=s["ws"])
    return K.attn_chunk_paged_fp8(s["q"], s["cu"], s["lens"], s["table"], s["k_pages"], s["k_scales"], s["v_pages"],
                                  s["v_scales"], s["scale"], max_q=s["n_max"], ws=s["ws"])


def _places(s):
    """Of every packed token: its position and its (page, row of the page)."""
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = s["lens"][b].long() - (s["cu"][b + 1].long() - t)
    page = s["case"]["page"]
    return pos, s["table"][b, pos // page].long(), pos % page


def _rotated(s, pos):
    """The new keys rotated at their positions, in fp32."""
    x, half = s["k"].float(), s["case"]["d"] // 2
    c, n = s["cos"][pos][:, None], s["sin"][pos][:, None]
    if s["case"]["pair"] == 0:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * n, a * n + b * c], -1)


def _append(s):
    pos, pg, row = _places(s)
    s["k_pages"][pg, :, row] = _rotated(s, pos).to(BF16)
    s["v_pages"][pg, :, row] = s["v"]
    return s["k_pages"], s["v_pages"]


def _append_fp8(s):
    pos, pg, row = _places(s)
    for x, rows in (("k", _rotated(s, pos)), ("v", s["v"].float())):
        codes, scales = _quantised(rows)
        s[x + "_pages"][pg, :, row] = codes.view(torch.uint8)
        s[x + "_scales"][pg, :, row] = scales
    return s["k_pages"].view(F8), s["k_scales"], s["v_pages"].view(F8), s["v_scales"]


def _rows(s, x):
    """[B, Hk, L_max, d] fp32: the cached rows of every sequence in order (past its length: whatever is there)."""
    r = torch.arange(s["L_max"], device="cuda")
    pg, row = s["table"][:, r // s["case"]["page"]].long(), r % s["case"]["page"]
    if x + "_scales" in s:
        rows = s[x + "_pages"].view(F8)[pg, :, row].float() * s[x + "_scales"][pg, :, row][..., None]
    else:
        rows = s[x + "_pages"][pg, :, row].float()
    return rows.transpose(1, 2)


def _read_fp8(s):
    have = (torch.arange(s["L_max"], device="cuda") < s["lens"][:, None])[:, None, :, None]
    for x in "kv":
        s[x + "_out"] = torch.where(have, _rows(s, x).to(BF16), s[x + "_out"])
    return s["k_out"], s["v_out"]


def _attention(s):
    c, q = s["case"], s["q"]
    T, H, Hk, d, n, L = q.shape[0], c["H"], c["Hk"], c["d"], s["n_max"], s["L_max"]
    i = torch.arange(n, device="cuda")
    first, count = s["cu"][:-1].long()[:, None], (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    tok = torch.where(i < count, first + i, T)  # [B, n]: a packed token, or T where the sequence has no more
    x = torch.cat([q.float(), q.new_zeros(1, H, d, dtype=torch.float32)])[tok]  # [B, n, H, d]
    x = x.view(c["B"], n, Hk, H // Hk, d).permute(0, 2, 1, 3, 4).reshape(c["B"], Hk, -1, d)
    p = (x * s["scale"]) @ _rows(s, "k").transpose(-1, -2)  # [B, Hk, n * g, L]
    pos = s["lens"].long()[:, None] - count + i
    seen = torch.arange(L, device="cuda") <= pos[..., None]  # [B, n, L]
    p = p.view(c["B"], Hk, n, H // Hk, L).masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = p.amax(-1, keepdim=True)
    m = torch.where(m > float("-inf"), m, 0.0)
    p = torch.exp(p - m)
    z = p.sum(-1, keepdim=True)
    have = (torch.arange(L, device="cuda") < s["lens"][:, None])[:, None, :, None]
    o = p.view(c["B"], Hk, -1, L) @ torch.where(have, _rows(s, "v"), 0.0)
    o = o.view(c["B"], Hk, n, H // Hk, d) / z
    out = torch.zeros(T + 1, H, d, device="cuda")
    lse = torch.zeros(T + 1, H, device="cuda")
    out[tok] = o.permute(0, 2, 1, 3, 4).reshape(c["B"], n, H, d)
    lse[tok] = (m + torch.log(z))[..., 0].permute(0, 2, 1, 3).reshape(c["B"], n, H)
    return out[:T].to(BF16), lse[:T]


# ---- the definitions in 64 bits, one sequence and head at a time ---------------------------------------------------


def _e4m3(y):
    """y rounded to the nearest E4M3 value, ties to even, from the format: 3 mantissa bits, exponents from -6."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def exact(c, seed):
    s = prepare(c, seed)
    ns, lens = _layout(c)
    page, d, Hk, g = c["page"], c["d"], c["Hk"], c["H"] // c["Hk"]
    first = [sum(ns[:b]) for b in range(c["B"])]

    def dest(b, lo):
        r = torch.arange(lo, lens[b], device="cuda")
        return s["table"][b][r // page].long(), r % page

    if c["op"].startswith("append"):
        out = {x: s[x].double() for x in ("k_pages", "v_pages")}
        out |= {x: s[x].double() for x in ("k_scales", "v_scales") if x in s}
        for b, n in enumerate(ns):
            pg, row = dest(b, lens[b] - n)
            k, v = (s[x][first[b]:first[b] + n].double() for x in "kv")
            w = torch.complex(s["cos"][lens[b] - n:lens[b]].double(), s["sin"][lens[b] - n:lens[b]].double())[:, None]
            if c["pair"] == 0:
                k = torch.view_as_real(torch.view_as_complex(k.reshape(n, Hk, d // 2, 2)) * w).reshape(n, Hk, d)
            else:
                z = torch.complex(k[..., :d // 2].contiguous(), k[..., d // 2:].contiguous()) * w
                k = torch.cat([z.real, z.imag], -1)
            for x, rows in (("k", k), ("v", v)):
                if c["op"] == "append_fp8":
                    scale = rows.abs().max(-1).values / 448
                    out[x + "_scales"][pg, :, row] = scale
                    rows = _e4m3(rows / scale.clamp(min=1e-300)[..., None])
                out[x + "_pages"][pg, :, row] = rows
        return tuple(out[x] for x in ("k_pages", "k_scales", "v_pages", "v_scales") if x in out)

    def cached(b, x, h):
        pg, row = dest(b, 0)
        rows = s[x + "_pages"][pg, h, row]
        if x + "_scales" in s:
            return rows.view(F8).double() * s[x + "_scales"][pg, h, row].double()[:, None]
        return rows.double()

    if c["op"] == "read_fp8":
        if sum(lens) * Hk * d > 3e8:
            return None
        out = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b in range(c["B"]):
            for h in range(Hk):
                for x, o in zip("kv", out):
                    o[b, h, :lens[b]] = cached(b, x, h)
        return tuple(out)

    T = sum(ns)
    out = torch.zeros(T, c["H"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
    for b, n in enumerate(ns):
        hidden = torch.arange(lens[b], device="cuda") > torch.arange(lens[b] - n, lens[b], device="cuda")[:, None]
        for h in range(Hk):
            k, v = cached(b, "k", h), cached(b, "v", h)
            for j in range(h * g, h * g + g):
                a = (s["q"][first[b]:first[b] + n, j].double() @ k.T) * s["scale"]
                a = a.masked_fill(hidden, float("-inf"))
                z = torch.logsumexp(a, -1)
                lse[first[b]:first[b] + n, j] = z
                out[first[b]:first[b] + n, j] = torch.exp(a - z[:, None]) @ v
    return out, lse
