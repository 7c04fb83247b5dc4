"""More operators of the paged cache over their real range: block tables and slot maps planned on the GPU, a cache held in
8 bits with a scale per page and head (append and attention), and attention with a sliding window and sinks, of one new
token and of runs of rows.

`run` computes them in plain torch operations; with `own` set it makes the calls that a user of the package makes.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}
LLAMA = {"heads": 8, "group": 4, "dim": 128, "dtype": "bf16"}     # Llama-3-8B shape
SMOL = {"heads": 32, "group": 1, "dim": 64, "dtype": "f16"}       # SmolLM2-1.7B shape


# ------------------------------------------------------------------ cases
def listed():
    return [
        # fifteen agents past their window: a decode call that reads the window and the first tokens alone
        {"name": "window_15x7194", "op": "attend", "codes": "", "layers": 1, "seqs": 15, "lo": 3597, "hi": 7194, "empty": 0,
         "page": 32, "window": 1024, "sinks": 4, "out": "in", **LLAMA},
        # a full batch of very different lengths, some inside the window, a few slots empty
        {"name": "window_256_ragged", "op": "attend", "codes": "", "layers": 1, "seqs": 256, "lo": 1, "hi": 32768, "empty": 9,
         "page": 16, "window": 4096, "sinks": 20, "out": "in", **LLAMA},
        # one agent with a short 8-bit cache: a latency-bound decode call
        {"name": "codes_1x600", "op": "attend", "codes": "int8", "layers": 1, "seqs": 1, "lo": 600, "hi": 600, "empty": 0,
         "page": 16, "window": 0, "sinks": 0, "out": "f32", **SMOL},
        # fifteen agents at about 4K private tokens in 8-bit floating point, one decoder layer
        {"name": "codes_15x4096", "op": "attend", "codes": "e4m3", "layers": 1, "seqs": 15, "lo": 3500, "hi": 4096, "empty": 0,
         "page": 32, "window": 0, "sinks": 0, "out": "in", **LLAMA},
        # one long document held in 8 bits; the odd length ends inside a page
        {"name": "codes_1x131071", "op": "attend", "codes": "int8", "layers": 1, "seqs": 1, "lo": 131071, "hi": 131071,
         "empty": 0, "page": 64, "window": 0, "sinks": 0, "out": "f32", **LLAMA},
        # one new token for each of a full batch into 8-bit pages, and the pages it changed read back
        {"name": "append8_256x1", "op": "append8", "codes": "int8", "layers": 1, "seqs": 256, "new_lo": 1, "new_hi": 1,
         "old_hi": 7194, "far": 0, "page": 16, "pairs": "half", **LLAMA},
        # a prompt of 7,194 tokens into an empty 8-bit cache, and its tokens read back as they are held
        {"name": "append8_1x7194", "op": "append8", "codes": "e4m3", "layers": 1, "seqs": 1, "new_lo": 7194, "new_hi": 7194,
         "old_hi": 0, "far": 0, "page": 64, "pairs": "half", **LLAMA},
        # a few drafted tokens for each of fifteen agents, checked against all of their context
        {"name": "rows_15_drafts", "op": "rows", "layers": 1, "seqs": 15, "new_lo": 2, "new_hi": 5, "old_lo": 600, "old_hi": 1851,
         "page": 16, "window": 0, "sinks": 0, **SMOL},
        # five ragged prompts behind earlier tokens, without a window
        {"name": "rows_5_prompts", "op": "rows", "layers": 1, "seqs": 5, "new_lo": 601, "new_hi": 1851, "old_lo": 0, "old_hi": 600,
         "page": 32, "window": 0, "sinks": 0, **LLAMA},
        # a long prompt under a window
        {"name": "rows_1x8191_window", "op": "rows", "layers": 1, "seqs": 1, "new_lo": 8191, "new_hi": 8191, "old_lo": 0, "old_hi": 0,
         "page": 64, "window": 2048, "sinks": 4, **LLAMA},
        # a decode step of fifteen agents: last step's rejected drafts go, four more tokens each are planned
        {"name": "plan_15x4", "op": "plan", "seqs": 15, "lo": 600, "hi": 7194, "draft": 4, "admit": 0, "prompt": 0,
         "page": 32, "window": 0, "sinks": 0},
        # continuous batching: 512 slots, an eighth of them take prompts of up to 4,096 tokens where sequences ended, the rest go on
        # under a window
        {"name": "plan_512_mixed", "op": "plan", "seqs": 512, "lo": 1, "hi": 7194, "draft": 1, "admit": 64, "prompt": 4096,
         "page": 16, "window": 2048, "sinks": 4},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append8", "rows", "plan"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        seqs = _log(rng, 1, 512)
        hi = _log(rng, 1, 7194)
        return {"op": op, "page": page, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "draft": rng.choice([1, 1, _log(rng, 2, 9)]),
                "admit": rng.choice([0, seqs // 8]), "prompt": _log(rng, 1, 4096), "window": rng.choice([0, _log(rng, 1, 4096)]),
                "sinks": rng.choice([0, _log(rng, 1, 130)])}
    heads, group, dim = rng.choice([(8, 4, 128), (32, 1, 64), (4, 8, 64), (8, 2, 128), (2, 16, 128), (1, 7, 128), (8, 1, 128)])
    c = {"op": op, "heads": heads, "group": group, "dim": dim, "dtype": rng.choice(["bf16", "f16"]), "page": page,
         "layers": rng.choice([1, 1, 1, 2, 3])}
    row = heads * dim * c["layers"]
    if op == "append8":
        new_hi = rng.choice([1, _log(rng, 2, 2000)])
        seqs = _log(rng, 1, max(1, min(256, 8_000_000 // (row * new_hi))))
        c.update(codes=rng.choice(["int8", "e4m3"]), seqs=seqs, new_lo=rng.randint(0 if new_hi > 1 else 1, new_hi), new_hi=new_hi,
                 old_hi=rng.choice([0, _log(rng, 1, 600)]), far=rng.choice([0, _log(rng, 1, 4000000)]),
                 pairs=rng.choice(["half", "next"]))
        return c
    if op == "rows":
        c["layers"] = 1
        seqs = _log(rng, 1, 32)
        pairs = 200_000_000_000 // (4 * heads * group * dim)        # of a row and a token, in all
        new_hi = _log(rng, 1, max(1, min(4096, math.isqrt(pairs // seqs))))
        old_hi = rng.choice([0, _log(rng, 1, max(1, min(8192, pairs // (2 * seqs * new_hi))))])
        c.update(seqs=seqs, new_lo=rng.randint(1, new_hi), new_hi=new_hi, old_lo=rng.randint(0, old_hi), old_hi=old_hi,
                 window=rng.choice([0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 4, _log(rng, 1, 200)]))
        return c
    codes = rng.choice(["", "int8", "e4m3"])
    window = _log(rng, 1, 8192) if codes == "" else rng.choice([0, 0, _log(rng, 1, 8192)])
    seqs = _log(rng, 1, 256)
    hi = _log(rng, 1, max(1, min(131072, 130_000_000 // row // seqs)))
    c.update(codes=codes, seqs=seqs, lo=rng.randint(1, hi), hi=hi, empty=rng.choice([0, 0, seqs // 8]), window=window,
             sinks=rng.choice([0, 4, _log(rng, 1, 200)]) if window else 0, out=rng.choice(["f32", "in"]))
    return c


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n lengths in [lo, hi], spread evenly over their logarithm: the same for every seed, which only orders them."""
    a, b = math.log(max(1, lo)), math.log(max(1, hi))
    return [max(lo, min(hi, round(math.exp(b - (b - a) * i / max(1, n - 1))))) for i in range(n)]


def _lens(c):
    return _spread(c["lo"], c["hi"], c["seqs"] - c["empty"]) + [0] * c["empty"]


def _even(lo, hi, n):
    return [round(hi - (hi - lo) * i / max(1, n - 1)) for i in range(n)]


def _shuffled(values, g):
    return torch.tensor(values)[torch.randperm(len(values), generator=g)]


def _table(room, page, n_pages, g, width=0):
    """A block table for sequences with room for that many tokens: their pages in random order, -1 behind. And the pages
    that nobody has, in random order."""
    need = (room + page - 1) // page
    ids = torch.randperm(n_pages, generator=g).int()
    table = torch.full((len(room), max(1, width, int(need.max()))), -1, dtype=torch.int32)
    own_slot = torch.arange(table.shape[1])[None] < need[:, None]
    used = int(need.sum())
    table[own_slot] = ids[:used]
    return table, ids[used:]


def _starts(counts):
    return torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int()


def _prepare_plan(c, host):
    """Live sequences at their lengths, the slots that get prompts idle, free pages for twice what a step takes."""
    A, page = c["seqs"], c["page"]
    order = torch.randperm(A, generator=host)
    lens = torch.full((A,), -1, dtype=torch.long)
    new = torch.zeros(A, dtype=torch.long)
    live, idle = order[c["admit"]:], order[:c["admit"]]
    lens[live] = torch.tensor(_spread(c["lo"], c["hi"], len(live)), dtype=torch.long)
    new[live] = c["draft"]
    new[idle] = torch.tensor(_spread(1, max(1, c["prompt"]), len(idle)), dtype=torch.long)
    ends = lens.clamp(0) + new
    held = (lens.clamp(0) + page - 1) // page
    width = int((ends.max() + page - 1) // page) + 1
    n_pages = int(held.sum()) + 2 * int(((new + page - 1) // page + 1).sum()) + 3
    table, free = _table(lens.clamp(0), page, n_pages, host, width)
    ring = torch.full((n_pages,), -1, dtype=torch.int32)
    ring[:len(free)] = free
    first = torch.full((A,), -(-c["sinks"] // page), dtype=torch.int32)
    return {"new": new.int().cuda(), "keep": lens.int().cuda(), "n_rows": int(new.sum()), "n_pages": n_pages,
            "table": table.cuda(), "lens": lens.int().cuda(), "first": first.cuda(), "ring": ring.cuda(),
            "counts": torch.tensor([0, len(free)], dtype=torch.long).cuda()}


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed + 1)
    s = {"case": c}
    if c["op"] == "plan":
        s.update(_prepare_plan(c, host))
        if own:
            import serving_q8_encode_gb300 as pk
            t = s["tables"] = pk.PageTable(c["seqs"], s["table"].shape[1], s["n_pages"], c["page"], window=c["window"], sinks=c["sinks"])
            t.restore(s["table"], s["lens"], s["first"], s["ring"], s["counts"])
        return s
    dt, L, H, G, d, page = DT[c["dtype"]], c["layers"], c["heads"], c["group"], c["dim"], c["page"]
    randn = lambda *z: torch.randn(z, dtype=dt, device="cuda", generator=gpu)  # noqa: E731
    if c["op"] == "attend":
        old = torch.zeros(c["seqs"], dtype=torch.long)
        ends = _shuffled(_lens(c), host)
    else:
        # long runs behind short contexts; a seed only orders the sequences
        order = torch.randperm(c["seqs"], generator=host)
        new = torch.tensor(_even(c["new_lo"], c["new_hi"], c["seqs"]))[order]
        old = torch.tensor(_even(c.get("old_lo", 0), c["old_hi"], c["seqs"])[::-1])[order]
        ends = old + new
        s["starts"] = _starts(new).cuda()
        s["row_seq"] = torch.repeat_interleave(torch.arange(c["seqs"]), new).cuda()
        s["row_at"] = torch.cat([torch.arange(int(x)) for x in new]).cuda()
    n_pages = int(((ends + page - 1) // page).sum()) + 3
    table = _table(ends, page, n_pages, host)[0]
    s.update(table=table.cuda(), lens=ends.int().cuda(), old=old.int().cuda())
    # keys with outlier channels
    wide = torch.exp(0.5 * torch.randn(L, 1, H, 1, d, device="cuda", generator=gpu)).to(dt)
    k, v = randn(L, n_pages, H, page, d) * wide, randn(L, n_pages, H, page, d)
    s["scales"] = None
    if c.get("codes"):
        # pages as appends leave them: each block's codes under the power of two that its largest value asks for
        kind, top = CODES[c["codes"]]
        scales = torch.stack([_pow2(x.float().abs().amax((3, 4)), top) for x in (k, v)], -1)
        k, v = (_code(x.float(), scales[..., i, None, None], kind) for i, x in enumerate((k, v)))
        s["scales"] = scales.contiguous()
    s["k_pages"], s["v_pages"] = k, v
    if c["op"] == "attend":
        s["q"] = randn(L, c["seqs"], G * H, d)
    elif c["op"] == "rows":
        s["q"] = randn(L, len(s["row_seq"]), G * H, d)
    else:
        # a fused projection's rows: q, k and v are slices of one tensor
        rows = randn(L, len(s["row_seq"]), (G + 2) * H, d)
        s.update(q=rows[:, :, :G * H], k=rows[:, :, G * H:(G + 1) * H], v=rows[:, :, (G + 1) * H:], offset=c["far"],
                 one=c["new_lo"] == c["new_hi"] == 1, inv_freq=500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d))
        s["inv_freq_gpu"] = s["inv_freq"].cuda()
        # what is read back: the tokens from the start of each sequence's first changed page
        back = torch.where(new > 0, old % page + new, 0)
        s["back_starts"], s["n_back"] = _starts(back).cuda(), int(back.sum())
        s["back_seq"] = torch.repeat_interleave(torch.arange(c["seqs"]), back).cuda()
        s["back_at"] = torch.cat([torch.arange(int(e - b), int(e)) for b, e in zip(back, ends)]).cuda()
        # and which pages those are
        first, last = old // page, (ends + page - 1) // page
        s["touched"] = torch.cat([table[a, first[a]:last[a]] for a in range(c["seqs"]) if new[a] > 0] + [table[0, :0]]).long().cuda()
    if own:
        import serving_q8_encode_gb300 as pk
        s["cache"] = pk.PageCache(s["k_pages"], s["v_pages"], scales=s["scales"], row_dtype=dt if c.get("codes") else None)
        if c["op"] == "append8":
            s["rope"] = pk.Rope(s["inv_freq"], interleaved=c["pairs"] == "next", device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms
def _pow2(amax, top):
    """The smallest power of two (2^-100 at least) under which amax is at most `top`: exact, in 32 bits."""
    m, e = torch.frexp(amax)
    m_top, e_top = math.frexp(top)
    e = (e - e_top + (m > m_top).int()).clamp_min(-100)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, -100))


def _code(x, scale, kind):
    x = x / scale
    return x.round().to(kind) if kind is torch.int8 else x.to(kind)


def _plain_rotate(x, cos, sin, pairs):
    x = x.float()
    if pairs == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _bytes(pages):
    return pages.view(torch.uint8) if pages.element_size() == 1 else pages


def _numbers(x, pages):
    """Bytes of codes, or 16-bit values, in 32 bits."""
    return x.view(pages.dtype).float()


def _plain_append8(s):
    c = s["case"]
    dt, page, (kind, top) = DT[c["dtype"]], c["page"], CODES[c["codes"]]
    place = s["old"].long()[s["row_seq"]] + s["row_at"]
    angle = (place + s["offset"]).double()[:, None, None] * s["inv_freq_gpu"]    # 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _plain_rotate(s["q"], cos, sin, c["pairs"]).to(dt)
    rows = (_plain_rotate(s["k"], cos, sin, c["pairs"]), s["v"].float())
    at, slot, t = s["table"][s["row_seq"], place // page].long(), place % page, s["touched"]
    n_pages = s["k_pages"].shape[1]
    fresh = torch.zeros(n_pages + 1, device="cuda").index_fill_(0, torch.where(slot == 0, at, n_pages), 1.0)[t, None] > 0
    from_page = s["table"][s["back_seq"], s["back_at"] // page].long()
    back = []
    for x, pages, scales in zip(rows, (s["k_pages"], s["v_pages"]), s["scales"].unbind(-1)):
        raw = _bytes(pages)
        amax = torch.zeros(pages.shape[:3], device="cuda").index_reduce_(1, at, x.abs().amax(-1), "amax")[:, t]
        before = scales[:, t].masked_fill(fresh, 0.0)
        after = torch.maximum(before, _pow2(amax, top))
        held = _numbers(raw[:, t], pages) * before[..., None, None]
        raw[:, t] = _bytes(_code(held.masked_fill(fresh[..., None, None], 0.0), after[..., None, None], kind))
        scales[:, t] = after
        raw[:, at, :, slot] = _bytes(_code(x, scales[:, at, :, None], kind)).transpose(0, 1)
        held = _numbers(raw[:, from_page, :, s["back_at"] % page], pages).transpose(0, 1)
        back.append((held * scales[:, from_page, :, None]).to(dt))
    return {"q": q, "k": back[0], "v": back[1], "scales": s["scales"]}


def _values(s, lx, at, hx):
    """Keys and values of the named pages in 32 bits."""
    k, v = (_numbers(_bytes(x)[lx, at, hx], x) for x in (s["k_pages"], s["v_pages"]))
    if s["scales"] is None:
        return k, v
    scales = s["scales"][lx, at, hx]                                                                  # [L][A][H][n][2]
    return k * scales[..., 0, None, None], v * scales[..., 1, None, None]


def _softmax_of(x, live):
    x = x.masked_fill_(~live, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    return p, p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_attend(s):
    """softmax(q.k / sqrt(d)) v over each sequence's visible tokens; zeros where there are none."""
    c = s["case"]
    L, A, H, G, d, page, w = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"], c["page"], c["window"]
    lens = s["lens"].long()
    n = s["table"].shape[1]
    pages = torch.arange(n, device="cuda").expand(A, n)
    begin = torch.zeros_like(lens)
    if w and -(-c["sinks"] // page) + w // page + 2 < n:      # the sinks' pages and the window's, in order
        lead = -(-c["sinks"] // page)
        begin = (lens - w).clamp_min(0)
        at = torch.arange(lead + w // page + 2, device="cuda")
        pages = torch.where(at < lead, at, at - lead + (begin // page).clamp_min(lead)[:, None]).clamp_max(n - 1)
        twice = at > lead + n - 1 - (begin // page).clamp_min(lead)[:, None]
    else:
        begin = (lens - w).clamp_min(0) if w else begin
        twice = torch.zeros_like(pages, dtype=torch.bool)
    token = pages[..., None] * page + torch.arange(page, device="cuda")
    live = (token < lens[:, None, None]) & ((token >= begin[:, None, None]) | (token < c["sinks"])) & ~twice[..., None]
    live = live.flatten(1)                                                                            # [A][T]
    at = s["table"].long().gather(1, pages).clamp(0)[None, :, None]                                   # [1][A][1][n]
    lx = torch.arange(L, device="cuda")[:, None, None, None]
    hx = torch.arange(H, device="cuda")[:, None]
    k, v = (z.flatten(3, 4) for z in _values(s, lx, at, hx))                                          # [L][A][H][T][d]
    x = s["q"].float().view(L, A, H, G, d) @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    del k
    p, total = _softmax_of(x, live[None, :, None, None])
    out = (p @ v) / total
    return out.view(L, A, G * H, d).to(torch.float32 if c["out"] == "f32" else DT[c["dtype"]])


def _plain_rows(s):
    """The same for runs of rows: row i of a sequence stands at its place and sees what is before it, inside the window
    or among the sinks. Rows padded to the longest run."""
    c = s["case"]
    L, A, H, G, d, page = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"], c["page"]
    n = c["new_hi"]
    q = torch.zeros(L, A, n, G * H, d, device="cuda")
    q[:, s["row_seq"], s["row_at"]] = s["q"].float()
    q = q.view(L, A, n, H, G, d).permute(0, 1, 3, 4, 2, 5)                                            # [L][A][H][G][n][d]
    at = s["table"].long().clamp(0)[None, :, None]
    lx = torch.arange(L, device="cuda")[:, None, None, None]
    hx = torch.arange(H, device="cuda")[:, None]
    k, v = (z.flatten(3, 4)[:, :, :, None] for z in _values(s, lx, at, hx))                           # [L][A][H][1][T][d]
    place = s["old"].long()[:, None] + torch.arange(n, device="cuda")                                 # [A][n]
    token = torch.arange(k.shape[-2], device="cuda")
    live = token <= place[..., None]
    if c["window"]:
        live &= (token > place[..., None] - c["window"]) | (token < c["sinks"])
    x = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    p, total = _softmax_of(x, live[None, :, None, None])
    out = ((p @ v) / total).permute(0, 1, 4, 2, 3, 5).reshape(L, A, n, G * H, d)
    return out[:, s["row_seq"], s["row_at"]].to(DT[c["dtype"]])


def _push(s, give):
    """Pages of the table that `give` marks go to the ring's tail, slot by slot and page by page."""
    ring, table, counts = s["ring"], s["table"], s["counts"]
    rank = give.flatten().cumsum(0) - 1
    to = torch.where(give.flatten(), (counts[1] + rank) % len(ring), len(ring))
    ring.copy_(torch.cat([ring, ring[:1]]).scatter(0, to, table.flatten())[:-1])
    counts[1] += give.sum()
    table.masked_fill_(give, -1)


def _plain_plan(s):
    c = s["case"]
    page, lead = c["page"], -(-c["sinks"] // c["page"])
    table, lens, first, ring, counts = s["table"], s["lens"], s["first"], s["ring"], s["counts"]
    index = torch.arange(table.shape[1], device="cuda")
    pages = lambda n: (n.clamp_min(0).long() + page - 1) // page  # noqa: E731
    # what is cut: pages behind the tokens that stay
    stay = torch.where(s["keep"] < 0, -1, torch.minimum(lens, s["keep"]))
    left, had = pages(stay), pages(lens)
    held = (index < had[:, None]) & ((index < lead) | (index >= first[:, None]))
    _push(s, held & (index >= left[:, None]))
    lens.copy_(stay)
    first.copy_(torch.where(stay < 0, lead, torch.minimum(first, left.clamp_min(lead).int())))
    # what is planned: pages in slot order while there are any, none past one that got none
    free_before, head = counts[1] - counts[0], counts[0].clone()
    new = s["new"].long().clamp_min(0)
    old = lens.long().clamp_min(0)
    ends = new.cumsum(0)
    fits = (pages(old + new) <= table.shape[1]) & (ends <= s["n_rows"])
    need = torch.where(fits, pages(old + new) - pages(old), 0)
    upto = need.cumsum(0)
    granted = (new > 0) & fits & ((need == 0) | (upto <= free_before))
    # pages behind the window go back
    if c["window"]:
        behind = torch.minimum(((old + 1 - c["window"]).clamp_min(0) // page), pages(old))
        _push(s, (index >= first[:, None]) & (index < behind[:, None]) & (index >= lead) & (lens >= 0)[:, None])
        first.copy_(torch.maximum(first, behind.int()))
    take = granted[:, None] & (index >= pages(old)[:, None]) & (index < pages(old + new)[:, None])
    which = (upto - need)[:, None] + index - pages(old)[:, None]
    table.copy_(torch.where(take, ring[((head + which) % len(ring)).clamp_min(0)], table))
    counts[0] += torch.where(granted, need, 0).sum()
    before = torch.where(granted, old, -1).int()
    after = torch.where(granted, old + new, -1).int()
    lens.copy_(torch.where(granted, after, lens))
    # the rows' places
    row = torch.arange(s["n_rows"], device="cuda")
    seq = torch.searchsorted(ends, row, right=True).clamp_max(len(ends) - 1)
    ok = granted[seq] & (row < ends[-1])
    place = torch.where(ok, old[seq] + row - (ends - new)[seq], -1)
    slot = torch.where(ok, table[seq, (place // page).clamp_min(0)].long() * page + place % page, -1)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends]).clamp_max(s["n_rows"]).int()
    return {"starts": starts, "before": before, "after": after, "slots": slot, "positions": place, "table": table, "lens": lens,
            "first": first, "ring": ring, "counts": counts}


def run(s):
    c = s["case"]
    if not own:
        return {"attend": _plain_attend, "append8": _plain_append8, "rows": _plain_rows, "plan": _plain_plan}[c["op"]](s)
    if c["op"] == "plan":
        t = s["tables"]
        t.cut(s["keep"])
        p = t.plan(s["new"], s["n_rows"])
        return {"starts": p.starts, "before": p.before, "after": p.after, "slots": p.slots, "positions": p.positions,
                "table": t.block_table, "lens": t.lens, "first": t.first, "ring": t.ring, "counts": t.counts}
    cache = s["cache"]
    if c["op"] == "append8":
        q = cache.append(s["k"], s["v"], s["table"], s["old"], starts=None if s["one"] else s["starts"], q=s["q"], rope=s["rope"],
                         pos_offset=s["offset"])
        k, v = cache.gather(s["table"], s["lens"], s["back_starts"], s["n_back"])
        return {"q": q, "k": k, "v": v, "scales": s["scales"]}
    if c["op"] == "rows":
        return cache.attend_rows(s["q"], s["table"], s["lens"], s["starts"], window=c["window"], sinks=c["sinks"])
    return cache.attend(s["q"], s["table"], s["lens"], out_dtype=torch.float32 if c["out"] == "f32" else DT[c["dtype"]],
                        window=c["window"], sinks=c["sinks"])


# ------------------------------------------------------------------ work and the definition in 64 bits
def _seen(length, c):
    """Tokens that a row at the end of `length` tokens sees."""
    return length if not c["window"] else min(length, c["window"]) + min(c["sinks"], max(0, length - c["window"]))


def work(case):
    c = dict(case)
    if c["op"] == "plan":
        live = _spread(c["lo"], c["hi"], c["seqs"] - c["admit"])
        new = [c["draft"]] * len(live) + _spread(1, max(1, c["prompt"]), c["admit"])
        pages = sum(-(-n // c["page"]) for n in new)            # taken, and given back by the cut: id in, id out
        return {"bytes": 4 * 9 * c["seqs"] + 16 * sum(new) + 2 * 16 * pages, "flops": 4 * sum(new)}
    L, A, H, G, d, page = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"], c["page"]
    row = L * H * d                                             # elements of one token's keys, or values
    if c["op"] == "append8":
        new = _even(c["new_lo"], c["new_hi"], A)
        old = sum(n > 0 for n in new) * (min(page, c["old_hi"] + 1) - 1) / 2          # in the first page, read back
        # q in and out, k and v in and their codes out; codes back in, 16-bit rows out
        return {"bytes": int(sum(new) * row * (4 * G + 4 + 2) + (sum(new) + old) * row * (2 + 4)),
                "flops": int(3 * sum(new) * row * (G + 1) + 6 * sum(new) * row)}
    if c["op"] == "rows":
        new = _even(c["new_lo"], c["new_hi"], A)
        old = (c["old_lo"] + c["old_hi"]) / 2
        pairs = sum(_seen(old + i + 1, c) for n in new for i in range(n))
        held = sum(old + n if not c["window"] else min(old + n, n + c["window"] + c["sinks"]) for n in new)
        return {"bytes": int(4 * row * (G * sum(new) + held)), "flops": int(4 * pairs * row * G)}
    lens = [_seen(n, c) for n in _lens(c)]
    ends = A * G * row * (2 + (4 if c["out"] == "f32" else 2))  # q in, the output out
    return {"bytes": int(2 * sum(lens) * row * (1 if c["codes"] else 2) + ends), "flops": int(4 * sum(lens) * row * G)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    page = c["page"]
    if c["op"] == "plan":
        return _exact_plan(s)
    L, A, H, G, d = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    if c["op"] == "append8":
        return _exact_append8(s, table)

    def tokens(a, l):
        """A sequence's keys and values of one layer in 64 bits: [H][len][d]."""
        ids = torch.tensor(table[a][:-(-lens[a] // page)], device="cuda", dtype=torch.long)
        out = []
        for i, x in enumerate((s["k_pages"], s["v_pages"])):
            x = _numbers(_bytes(x)[l, ids], x).double()
            if s["scales"] is not None:
                x = x * s["scales"][l, ids, :, i].double()[..., None, None]
            out.append(x.transpose(0, 1).reshape(H, -1, d)[:, :lens[a]])
        return out

    rows = c["op"] == "rows"
    if rows and L * A * H * G > 2000:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    begin = s["starts"].tolist() if rows else None
    for a in range(A):
        if not lens[a]:
            continue
        n = begin[a + 1] - begin[a] if rows else 1
        if not n:
            continue
        i = torch.arange(lens[a] - n, lens[a], device="cuda")[:, None]
        t = torch.arange(lens[a], device="cuda")[None]
        hidden = t > i
        if c["window"]:
            hidden = hidden | ((t <= i - c["window"]) & (t >= c["sinks"]))
        for l in range(L):
            k, v = tokens(a, l)
            for h in range(G * H):
                q = (s["q"][l, begin[a]:begin[a + 1], h] if rows else s["q"][l, a:a + 1, h]).double()
                z = torch.softmax((q @ k[h // G].T / math.sqrt(d)).masked_fill(hidden, -math.inf), -1) @ v[h // G]
                if rows:
                    out[l, begin[a]:begin[a + 1], h] = z
                else:
                    out[l, a, h] = z[0]
    return out


def _exact_append8(s, table):
    c = s["case"]
    L, H, d, page = c["layers"], c["heads"], c["dim"], c["page"]
    if c["seqs"] * L > 600:
        return None
    kind, top = CODES[c["codes"]]
    place = (s["old"][s["row_seq"]].long() + s["row_at"])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer((place + s["offset"]).double(), s["inv_freq_gpu"]))[:, None]

    def rotated(x):
        x = x.double()
        if c["pairs"] == "half":
            z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn
            return torch.cat([z.real, z.imag], -1)
        return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (d // 2, 2)).contiguous()) * turn).flatten(-2)

    def rounded(x):
        """64-bit numbers, in units of a scale, to the nearest code's value; ties to even."""
        if kind is torch.int8:
            return x.round()
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp_min(-6) - 3)
        return (x / step).round() * step

    starts, old = s["starts"].tolist(), s["old"].tolist()
    back, scales = [], s["scales"].double()
    for i, (x, pages) in enumerate(((rotated(s["k"]), s["k_pages"]), (s["v"].double(), s["v_pages"]))):
        out = torch.empty(L, s["n_back"], H, d, dtype=torch.float64, device="cuda")
        at = 0
        for a in range(c["seqs"]):
            row, t, end = starts[a], old[a], old[a] + starts[a + 1] - starts[a]
            while t < end:
                p, slot = divmod(t, page)
                n, id_ = min(page - slot, end - t), table[a][p]
                part = x[:, row:row + n].transpose(1, 2)                                            # [L][H][n][d]
                asked = (part.abs().amax((2, 3)) / top).log2()
                # the smallest power of two that is not below; log2 of a quotient may be off in the last place
                e = asked.ceil()
                e = torch.where(torch.exp2(e - 1) * top >= part.abs().amax((2, 3)), e - 1, e)
                scale = torch.exp2(e.clamp_min(-100))
                if slot:
                    scale = torch.maximum(scale, scales[:, id_, :, i])
                    was = _numbers(_bytes(pages)[:, id_, :, :slot], pages).double() * scales[:, id_, :, i, None, None]
                    out[:, at:at + slot] = (rounded(was / scale[..., None, None]) * scale[..., None, None]).transpose(1, 2)
                    at += slot
                out[:, at:at + n] = (rounded(part / scale[..., None, None]) * scale[..., None, None]).transpose(1, 2)
                scales[:, id_, :, i] = scale
                at, row, t = at + n, row + n, t + n
        back.append(out)
    return {"q": rotated(s["q"]), "k": back[0], "v": back[1], "scales": scales}


def _exact_plan(s):
    c = s["case"]
    page, lead, n_pages = c["page"], -(-c["sinks"] // c["page"]), s["n_pages"]
    table, lens, first = s["table"].tolist(), s["lens"].tolist(), s["first"].tolist()
    ring, (head, tail) = s["ring"].tolist(), s["counts"].tolist()
    of = lambda n: -(-max(0, n) // page)  # noqa: E731

    def give(a, p):
        nonlocal tail
        ring[tail % n_pages], table[a][p] = table[a][p], -1
        tail += 1

    for a, keep in enumerate(s["keep"].tolist()):
        stay = -1 if keep < 0 else min(lens[a], keep)
        for p in range(of(stay), of(lens[a])):
            if p < lead or p >= first[a]:
                give(a, p)
        lens[a], first[a] = stay, lead if stay < 0 else min(first[a], max(lead, of(stay)))
    free, start, short = tail - head, 0, False
    starts, before, after, slots, positions = [0], [], [], [-1] * s["n_rows"], [-1] * s["n_rows"]
    grants = []
    for a, n in enumerate(max(0, x) for x in s["new"].tolist()):
        old = max(0, lens[a])
        fits = of(old + n) <= len(table[a]) and start + n <= s["n_rows"]
        need = of(old + n) - of(old) if fits else 0
        short = short or need > free
        ok = n > 0 and fits and (need == 0 or not short)
        grants.append((a, old, n, start, ok))
        if ok:
            free -= need
        start += n
        starts.append(min(start, s["n_rows"]))
        before.append(old if ok else -1)
        after.append(old + n if ok else -1)
    for a in range(c["seqs"]):
        if c["window"] and lens[a] >= 0:
            behind = min(max(0, lens[a] + 1 - c["window"]) // page, of(lens[a]))
            for p in range(max(first[a], lead), behind):
                give(a, p)
            first[a] = max(first[a], behind)
    for a, old, n, start, ok in grants:
        if not ok:
            continue
        for p in range(of(old), of(old + n)):
            table[a][p] = ring[head % n_pages]
            head += 1
        for i in range(n):
            positions[start + i] = old + i
            slots[start + i] = table[a][(old + i) // page] * page + (old + i) % page
        lens[a] = old + n
    whole = lambda x: torch.tensor(x, device="cuda")  # noqa: E731
    return {"starts": whole(starts).int(), "before": whole(before).int(), "after": whole(after).int(), "slots": whole(slots),
            "positions": whole(positions), "table": whole(table).int(), "lens": whole(lens).int(), "first": whole(first).int(),
            "ring": whole(ring).int(), "counts": whole([head, tail])}
