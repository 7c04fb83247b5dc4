"""The paged-cache operators over their real range: appending rotated keys and values to a paged cache, attention of
one new token per sequence over the pages, and sparse attention over the pages that a cheap score selects.

`run` computes them in plain torch operations; with `own` set it makes the calls that a user of the package makes.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
LLAMA = {"heads": 8, "group": 4, "dim": 128, "dtype": "bf16"}     # Llama-3-8B shape
SMOL = {"heads": 32, "group": 1, "dim": 64, "dtype": "f16"}       # SmolLM2-1.7B shape


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one agent, one layer, a short context: a latency-bound decode call
        {"name": "attend_1x600", "op": "attend", "layers": 1, "seqs": 1, "lo": 600, "hi": 600, "empty": 0,
         "page": 16, "out": "f32", **SMOL},
        # fifteen agents at about 4K private tokens, one decoder layer: the ordinary decode call
        {"name": "attend_15x4096", "op": "attend", "layers": 1, "seqs": 15, "lo": 3500, "hi": 4096, "empty": 0,
         "page": 32, "out": "in", **LLAMA},
        # a full batch of very different lengths, a few slots empty: continuous batching
        {"name": "attend_256_ragged", "op": "attend", "layers": 1, "seqs": 256, "lo": 1, "hi": 7194, "empty": 9,
         "page": 16, "out": "in", **LLAMA},
        # one long document, split over its length; the odd length ends inside a page
        {"name": "attend_1x131071", "op": "attend", "layers": 1, "seqs": 1, "lo": 131071, "hi": 131071, "empty": 0,
         "page": 64, "out": "f32", **LLAMA},
        # one new token for each of fifteen agents: the append of a decode step
        {"name": "append_15x1", "op": "append", "layers": 1, "seqs": 15, "new_lo": 1, "new_hi": 1, "old_hi": 7194,
         "far": 0, "page": 32, "bounds": True, "pairs": "half", **LLAMA},
        # the same for a full batch at far positions
        {"name": "append_256x1_far", "op": "append", "layers": 1, "seqs": 256, "new_lo": 1, "new_hi": 1,
         "old_hi": 1000, "far": 1000000, "page": 16, "bounds": True, "pairs": "half", **LLAMA},
        # a prompt of 7,194 tokens into an empty cache, one layer
        {"name": "append_1x7194", "op": "append", "layers": 1, "seqs": 1, "new_lo": 7194, "new_hi": 7194, "old_hi": 0,
         "far": 0, "page": 64, "bounds": False, "pairs": "half", **LLAMA},
        # five ragged prompts behind earlier tokens, all 24 layers, neighbouring pairs
        {"name": "append_5_ragged_24", "op": "append", "layers": 24, "seqs": 5, "new_lo": 601, "new_hi": 1851,
         "old_hi": 600, "far": 0, "page": 16, "bounds": True, "pairs": "next", **SMOL},
        # five agents at SmolLM2's context, an eighth of the pages
        {"name": "sparse_5x1851", "op": "sparse", "layers": 1, "seqs": 5, "lo": 1500, "hi": 1851, "empty": 0,
         "page": 16, "take": 15, "first": 1, "last": 1, "out": "f32", **SMOL},
        # fifteen agents at long contexts, 1,024 tokens each
        {"name": "sparse_15x7194", "op": "sparse", "layers": 1, "seqs": 15, "lo": 3597, "hi": 7194, "empty": 0,
         "page": 16, "take": 64, "first": 1, "last": 2, "out": "in", **LLAMA},
        # one long document: the case that selection is for
        {"name": "sparse_1x131072", "op": "sparse", "layers": 1, "seqs": 1, "lo": 131072, "hi": 131072, "empty": 0,
         "page": 32, "take": 128, "first": 0, "last": 1, "out": "in", **LLAMA},
        # a batch of long ragged contexts, some slots empty, four layers in one call
        {"name": "sparse_16_ragged_4", "op": "sparse", "layers": 4, "seqs": 16, "lo": 300, "hi": 32768, "empty": 2,
         "page": 64, "take": 32, "first": 1, "last": 1, "out": "in", **LLAMA},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    heads, group, dim = rng.choice([(8, 4, 128), (32, 1, 64), (4, 8, 64), (8, 2, 128), (2, 16, 128), (1, 7, 128), (8, 1, 128)])
    c = {"heads": heads, "group": group, "dim": dim, "dtype": rng.choice(["bf16", "f16"]), "page": rng.choice([16, 32, 64, 128]),
         "layers": rng.choice([1, 1, 1, 2, 3]), "op": rng.choice(["attend", "append", "sparse"])}
    row = heads * dim * c["layers"]
    if c["op"] == "append":
        new_hi = rng.choice([1, _log(rng, 2, 2000)])
        seqs = _log(rng, 1, max(1, min(256, 150_000_000 // (row * (group + 2) * new_hi))))
        c.update(seqs=seqs, new_lo=rng.randint(0 if new_hi > 1 else 1, new_hi), new_hi=new_hi, old_hi=rng.choice([0, _log(rng, 1, 600)]),
                 far=rng.choice([0, _log(rng, 1, 4000000)]), bounds=rng.choice([True, False]), pairs=rng.choice(["half", "next"]))
        return c
    most = 200_000_000 // row   # tokens in all
    seqs = _log(rng, 1, 256)
    hi = _log(rng, 1, max(1, min(131072, most // seqs)))
    c.update(seqs=seqs, lo=rng.randint(1, hi), hi=hi, empty=rng.choice([0, 0, seqs // 8]), out=rng.choice(["f32", "in"]))
    if c["op"] == "sparse":
        c.update(take=_log(rng, 3, 200), first=rng.choice([0, 1]), last=rng.choice([0, 1, 2]))
    return c


# ------------------------------------------------------------------ inputs
def _lens(case):
    """Lengths in [lo, hi], spread evenly over their logarithm, and the `empty` ones' 0: the same for every seed, which
    only orders them."""
    live = case["seqs"] - case["empty"]
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    return [round(math.exp(hi - (hi - lo) * i / max(1, live - 1))) for i in range(live)] + [0] * case["empty"]


def _new(case):
    """How many tokens each sequence appends: spread evenly over [new_lo, new_hi], in an order that the seed gives."""
    lo, hi, n = case["new_lo"], case["new_hi"], case["seqs"]
    return [round(hi - (hi - lo) * i / max(1, n - 1)) for i in range(n)]


def _shuffled(values, g):
    return torch.tensor(values)[torch.randperm(len(values), generator=g)]


def _table(room, page, n_pages, g):
    """A block table for sequences with room for that many tokens: their pages in random order, -1 behind."""
    need = (room + page - 1) // page
    ids = torch.randperm(n_pages, generator=g).int()
    table = torch.full((len(room), max(1, int(need.max()))), -1, dtype=torch.int32)
    own_slot = torch.arange(table.shape[1])[None] < need[:, None]
    table[own_slot] = ids[:int(need.sum())]
    return table


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed + 1)
    dt, L, H, G, d, page = DT[c["dtype"]], c["layers"], c["heads"], c["group"], c["dim"], c["page"]
    randn = lambda *s: torch.randn(s, dtype=dt, device="cuda", generator=gpu)  # noqa: E731
    s = {"case": c}
    if c["op"] == "append":
        new = _shuffled(_new(c), host)
        old = torch.randint(0, c["old_hi"] + 1, (c["seqs"],), generator=host)
        n_pages = c["seqs"] * -(-(c["old_hi"] + c["new_hi"]) // page) + 3
        table = _table(old + new, page, n_pages, host)
        starts = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)])
        n = int(starts[-1])
        # a fused projection's rows: q, k and v are slices of one tensor
        rows = randn(L, n, (G + 2) * H, d)
        s.update(q=rows[:, :, :G * H], k=rows[:, :, G * H:(G + 1) * H], v=rows[:, :, (G + 1) * H:],
                 starts=starts.int().cuda() if c["new_hi"] > 1 else None, offset=c["far"], lens=old.int().cuda(),
                 inv_freq=500000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d))
        s["inv_freq_gpu"] = s["inv_freq"].cuda()
        # which sequence a row belongs to, and its place there (the scheduler that packed the rows has them)
        s["row_seq"] = torch.repeat_interleave(torch.arange(c["seqs"]), new).cuda()
        s["row_at"] = torch.cat([torch.arange(int(x)) for x in new]).cuda()
    else:
        lens = _shuffled(_lens(c), host)
        n_pages = int(((lens + page - 1) // page).sum()) + 3
        table = _table(lens, page, n_pages, host)
        s.update(q=randn(L, c["seqs"], G * H, d), lens=lens.int().cuda())
    s["table"] = table.cuda()
    s["k_pages"], s["v_pages"] = randn(L, n_pages, H, page, d), randn(L, n_pages, H, page, d)
    s["k_pages"] *= torch.exp(0.5 * torch.randn(L, 1, H, 1, d, device="cuda", generator=gpu)).to(dt)   # outlier channels
    s["bounds"] = None
    if c["op"] == "sparse":
        s["bounds"] = torch.zeros(L, n_pages, H, 2, d, dtype=dt, device="cuda")
        _plain_bounds(s, torch.arange(table.shape[1], device="cuda")[None].expand(table.shape))
    elif c["op"] == "append" and c["bounds"]:
        s["bounds"] = randn(L, n_pages, H, 2, d)
    if own:
        import serving_q8_encode_gb300 as pk
        s["cache"] = pk.PageCache(s["k_pages"], s["v_pages"], key_bounds=s["bounds"])
        if c["op"] == "append":
            s["rope"] = pk.Rope(s["inv_freq"], interleaved=c["pairs"] == "next", device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_bounds(s, pages):
    """Lowest and highest key of the given pages (per sequence, counted along the sequence), over the tokens in use."""
    page = s["case"]["page"]
    seq = torch.arange(pages.shape[0], device="cuda")[:, None].expand(pages.shape)
    fill = (s["lens"][:, None] - pages * page).clamp(0, page)
    live = (fill > 0) & (pages >= 0)
    seq, pages, fill = seq[live], pages[live], fill[live]
    at = s["table"][seq, pages].long()
    keys = s["k_pages"][:, at].float()
    used = (torch.arange(page, device="cuda") < fill[:, None])[None, :, None, :, None]
    s["bounds"][:, at, :, 0] = keys.masked_fill(~used, math.inf).amin(3).to(s["bounds"].dtype)
    s["bounds"][:, at, :, 1] = keys.masked_fill(~used, -math.inf).amax(3).to(s["bounds"].dtype)


def _plain_rotate(x, cos, sin, pairs):
    x = x.float()
    if pairs == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_append(s):
    c = s["case"]
    dt, page = DT[c["dtype"]], c["page"]
    place = s["lens"].long()[s["row_seq"]] + s["row_at"]
    angle = (place + s["offset"]).double()[:, None, None] * s["inv_freq_gpu"]    # [n][1][d/2], 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k = (_plain_rotate(x, cos, sin, c["pairs"]).to(dt) for x in (s["q"], s["k"]))
    at, slot = s["table"][s["row_seq"], place // page].long(), place % page
    s["k_pages"][:, at, :, slot] = k.transpose(0, 1)
    s["v_pages"][:, at, :, slot] = s["v"].transpose(0, 1)
    outs = {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["bounds"] is not None:
        new = torch.zeros_like(s["lens"]).index_add_(0, s["row_seq"], torch.ones_like(s["row_seq"], dtype=torch.int32))
        first = s["lens"].long() // page
        pages = first[:, None] + torch.arange(s["table"].shape[1], device="cuda")
        pages = torch.where((pages * page < (s["lens"] + new)[:, None]) & (new > 0)[:, None], pages, -1)
        _plain_bounds({**s, "lens": s["lens"] + new}, pages)
        outs["bounds"] = s["bounds"]
    return outs


def _plain_attend(s, chosen=None):
    """softmax(q.k / sqrt(d)) v over each sequence's tokens, or over the chosen pages'; zeros where there are none."""
    c = s["case"]
    L, A, H, G, d, page = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"], c["page"]
    lens = s["lens"].long()
    if chosen is None:
        pages = torch.arange(s["table"].shape[1], device="cuda").expand(L, A, H, -1)
    else:
        pages = chosen.long()
    at = s["table"].long()[torch.arange(A, device="cuda")[:, None, None], pages.clamp(0)].clamp(0)   # [L][A][H][n]
    token = pages[..., None] * page + torch.arange(page, device="cuda")
    live = ((token < lens[:, None, None, None]) & (pages[..., None] >= 0)).flatten(3)                # [L][A][H][T]
    lx = torch.arange(L, device="cuda")[:, None, None, None]
    hx = torch.arange(H, device="cuda")[:, None]
    k = s["k_pages"][lx, at, hx].float().flatten(3, 4)                                               # [L][A][H][T][d]
    x = s["q"].float().view(L, A, H, G, d) @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    del k
    x = x.masked_fill(~live[:, :, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    v = s["v_pages"][lx, at, hx].float().flatten(3, 4).masked_fill_(~live[..., None], 0.0)
    out = (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    return out.view(L, A, G * H, d).to(torch.float32 if c["out"] == "f32" else DT[c["dtype"]])


def _plain_select(s):
    """Per sequence and kv head the `take` pages of the highest score, ascending, -1 behind. The score of a page is the
    largest over the group's heads of sum_d max(q_d lo_d, q_d hi_d), in 32 bits and in a fixed order because it decides
    whole numbers: eight neighbouring dimensions from left to right, then halves onto halves."""
    c = s["case"]
    L, A, H, G, d, page = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"], c["page"]
    n = (s["lens"].long() + page - 1) // page
    at = s["table"].long().clamp(0)
    b = s["bounds"][:, at].float()                                      # [L][A][n][H][2][d]
    b = b.permute(0, 1, 3, 2, 4, 5)                                     # [L][A][H][n][2][d]
    q = s["q"].float().view(L, A, H, G, d)

    def of_head(q):                                                     # [L][A][H][d] -> [L][A][H][n]
        x = torch.maximum(b[..., 0, :] * q[..., None, :], b[..., 1, :] * q[..., None, :]).unflatten(-1, (-1, 8))
        x = ((((((x[..., 0] + x[..., 1]) + x[..., 2]) + x[..., 3]) + x[..., 4]) + x[..., 5]) + x[..., 6]) + x[..., 7]
        x = x[..., :8] + x[..., 8:] if d == 128 else x
        x = x[..., :4] + x[..., 4:]
        x = x[..., :2] + x[..., 2:]
        return x[..., 0] + x[..., 1]

    score = torch.stack([of_head(q[:, :, :, g]) for g in range(G)]).amax(0)
    index = torch.arange(at.shape[1], device="cuda")
    here = index < n[:, None]
    kept = ((index < c["first"]) | (index >= (n - c["last"])[:, None])) & here
    score = score.masked_fill(kept[None, :, None], math.inf).masked_fill(~here[None, :, None], -math.inf)
    take = min(c["take"], at.shape[1])
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :take]
    best = torch.where(best < n[:, None, None], best, at.shape[1]).sort(-1).values
    best = torch.where(best == at.shape[1], -1, best)
    return torch.nn.functional.pad(best, (0, c["take"] - take), value=-1).int()


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "append":
            return _plain_append(s)
        if c["op"] == "attend":
            return _plain_attend(s)
        chosen = _plain_select(s)
        return {"pages": chosen, "out": _plain_attend(s, chosen)}
    cache = s["cache"]
    if c["op"] == "append":
        q = cache.append(s["k"], s["v"], s["table"], s["lens"], starts=s["starts"], q=s["q"], rope=s["rope"], pos_offset=s["offset"])
        outs = {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        return outs if s["bounds"] is None else {**outs, "bounds": s["bounds"]}
    dtype = torch.float32 if c["out"] == "f32" else DT[c["dtype"]]
    if c["op"] == "attend":
        return cache.attend(s["q"], s["table"], s["lens"], out_dtype=dtype)
    chosen = cache.select(s["q"], s["table"], s["lens"], c["take"], keep_first=c["first"], keep_last=c["last"])
    return {"pages": chosen, "out": cache.attend(s["q"], s["table"], s["lens"], selected=chosen, out_dtype=dtype)}


# ------------------------------------------------------------------ work and the definition in 64 bits
def work(case):
    c = dict(case)
    L, A, H, G, d, page = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"], c["page"]
    row = 2 * L * H * d                                  # bytes of one token's keys, or values, over the layers
    if c["op"] == "append":
        new = _new(c)
        moved = 2 * sum(new) * row * (G + 2)             # q, k and v, in and out
        if c["bounds"]:
            # the bounds of the pages that get tokens out, and the tokens that stood in each first page in
            touched = sum(1 + (n - 1) / page for n in new if n)
            moved += touched * 2 * row + sum(n > 0 for n in new) * row * min(page - 1, c["old_hi"]) / 2
        return {"bytes": int(moved), "flops": int(3 * sum(new) * L * H * (G + 1) * d)}
    lens = _lens(c)
    ends = A * G * row + A * G * row // 2 * (4 if c["out"] == "f32" else 2)     # q in, the output out
    if c["op"] == "attend":
        return {"bytes": int(2 * sum(lens) * row + ends), "flops": int(4 * sum(lens) * L * H * G * d)}
    pages = sum(-(-n // page) for n in lens)
    read = sum(min(n, c["take"] * page) for n in lens)
    return {"bytes": int(2 * pages * row + 2 * read * row + ends + 4 * L * A * H * c["take"]),
            "flops": int(3 * pages * L * H * G * d + 4 * read * L * H * G * d)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    L, A, H, G, d, page = c["layers"], c["seqs"], c["heads"], c["group"], c["dim"], c["page"]

    def append():
        half = d // 2
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        bounds = None if s["bounds"] is None else s["bounds"].double()
        place = (s["lens"][s["row_seq"]].long() + s["row_at"])
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.outer((place + s["offset"]).double(), s["inv_freq_gpu"]))[:, None]

        def rotated(x):
            x = x.double()
            if c["pairs"] == "half":
                z = torch.complex(x[..., :half], x[..., half:]) * turn
                return torch.cat([z.real, z.imag], -1)
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) * turn).flatten(-2)

        k, table, lens = rotated(s["k"]), s["table"].tolist(), s["lens"].tolist()
        new = torch.bincount(s["row_seq"], minlength=c["seqs"]).tolist()
        row = 0
        for a in range(c["seqs"]):
            done = 0
            while done < new[a]:
                p, slot = divmod(lens[a] + done, page)
                n, at = min(page - slot, new[a] - done), table[a][p]
                k_pages[:, at, :, slot:slot + n] = k[:, row:row + n].transpose(1, 2)
                v_pages[:, at, :, slot:slot + n] = s["v"][:, row:row + n].double().transpose(1, 2)
                if bounds is not None:
                    bounds[:, at, :, 0] = k_pages[:, at, :, :slot + n].min(2).values
                    bounds[:, at, :, 1] = k_pages[:, at, :, :slot + n].max(2).values
                row, done = row + n, done + n
        outs = {"q": rotated(s["q"]), "k_pages": k_pages, "v_pages": v_pages}
        return outs if bounds is None else {**outs, "bounds": bounds}

    def choose(l, a, h, n):
        """The chosen pages of one sequence and kv head. The score is defined in 32 bits, in its order."""
        b = s["bounds"][l, s["table"][a, :n].long(), h].float()                             # [n][2][d]
        q = s["q"][l, a, h * G:(h + 1) * G].float()                                         # [G][d]
        x = torch.where(q[:, None] > 0, q[:, None] * b[None, :, 1], q[:, None] * b[None, :, 0]).view(G, n, d // 8, 8)
        t = x[..., 0]
        for i in range(1, 8):
            t = t + x[..., i]
        while t.shape[-1] > 1:
            t = t[..., :t.shape[-1] // 2] + t[..., t.shape[-1] // 2:]
        score = t[..., 0].max(0).values.tolist()
        must = [p for p in range(n) if p < c["first"] or p >= n - c["last"]]
        rest = sorted((p for p in range(n) if p not in set(must)), key=lambda p: (-score[p], p))
        return sorted((must + rest)[:c["take"]])

    if c["op"] == "append":
        return append()
    if c["op"] == "sparse" and L * A * H > 600:
        return None
    out = torch.zeros(L, A, G * H, d, dtype=torch.float64, device="cuda")
    chosen = torch.full((L, A, H, c.get("take", 1)), -1, dtype=torch.int32)
    lens = s["lens"].tolist()
    for a in range(A):
        if not lens[a]:
            continue
        n = -(-lens[a] // page)
        for l in range(L):
            at = s["table"][a, :n].long()
            if c["op"] == "attend":
                k = s["k_pages"][l, at].double().transpose(0, 1).reshape(H, -1, d)[:, :lens[a]]
                v = s["v_pages"][l, at].double().transpose(0, 1).reshape(H, -1, d)[:, :lens[a]]
                w = torch.softmax(s["q"][l, a].double().view(H, G, d) @ k.mT / math.sqrt(d), -1)
                out[l, a] = (w @ v).view(G * H, d)
                continue
            for h in range(H):
                pick = choose(l, a, h, n)
                chosen[l, a, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
                rows = torch.cat([torch.arange(p * page, min((p + 1) * page, lens[a])) for p in pick]).cuda()
                k, v = (s[x][l, at[rows // page], h, rows % page].double() for x in ("k_pages", "v_pages"))
                w = torch.softmax(s["q"][l, a, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d), -1)
                out[l, a, h * G:(h + 1) * G] = w @ v
    return out if c["op"] == "attend" else {"pages": chosen, "out": out}
