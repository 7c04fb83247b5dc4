"""Attention over a window with sinks, over pages in 16 and in 8 bits, of one new token and of runs of rows; codes appended
and read back; and all of it in one run. Against plain forms in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
KIND = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import serving_q8_encode_gb300 as pk
    return pk


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(pk, lens, page, L, H, d, dtype, codes=None, seed=0, poison=True, extra=3):
    """(cache, block table, lens): pages in random order; with poison, what holds no token is as bad as its type can be."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(0, n) // page) for n in lens]
    ids = torch.randperm(sum(need) + extra, generator=g).tolist()
    P = len(ids)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    used = torch.zeros(P, page, dtype=torch.bool)
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = ids.pop()
            used[table[s, i], :max(0, lens[s] - i * page)] = True
    shape = (L, P, H, page, d)
    k = torch.randn(*shape, generator=g) * torch.exp(0.5 * torch.randn(L, 1, H, 1, d, generator=g))
    v = torch.randn(*shape, generator=g)
    empty = ~used[None, :, None, :, None]
    scales = None
    if codes:
        kind, top = KIND[codes]
        # any positive scales will do for reading
        scales = torch.stack([x.abs().amax((3, 4)) / top * (1 + torch.rand(L, P, H, generator=g)) for x in (k, v)], -1)
        k, v = (x / scales[..., i, None, None] for i, x in enumerate((k, v)))
        k, v = ((x.round() if codes == "int8" else x).to(kind) for x in (k, v))
        if poison:
            bad = 0x80 if codes == "int8" else 0x7F
            k, v = (torch.where(empty, torch.tensor(bad, dtype=torch.uint8), x.view(torch.uint8)).view(kind) for x in (k, v))
            scales[~used.any(1)[None].expand(L, P)] = math.nan
        scales = scales.cuda()
        c = pk.PageCache(k.cuda(), v.cuda(), scales=scales, row_dtype=DT[dtype])
    else:
        k, v = k.to(DT[dtype]), v.to(DT[dtype])
        if poison:
            k, v = k.masked_fill(empty, math.nan), v.masked_fill(empty, math.inf)
        c = pk.PageCache(k.cuda(), v.cuda())
    return c, table.cuda(), ints(lens)


def raw(pages):
    return pages.view(torch.uint8) if pages.element_size() == 1 else pages


def tokens(c, table, s, layer, h, at):
    """Keys and values of a sequence's tokens `at` in 64 bits."""
    page = c.page_tokens
    ids = table[s].long()[at // page]
    out = []
    for i, x in enumerate((c.k_pages, c.v_pages)):
        y = raw(x)[layer, ids, h, at % page].view(x.dtype).double()
        out.append(y if c.scales is None else y * c.scales[layer, ids, h, i].double()[:, None])
    return out


def reference(c, q, table, places, seqs, window, sinks, layer=0, scale=None, rounded_p=False):
    """(out, tolerance) in 64 bits of rows q [L][n][Hq][d] that stand at `places` of sequences `seqs`. Runs of rows
    (rounded_p) take codes as their values in the row's type.

    The tolerance, from the arithmetic. A logit: d products, exact, summed in fp32, off by at most d 2^-23 sum |q k|, and
    four roundings of factors (the scales', the softmax scale), 2^-22 of itself. A probability carries twice that (its own and
    the maximum's), 2^-22 of the exponential, and 2^-22 of its parts; where it enters as one number of the row's type, half a
    step of that instead (rounded_p: 2^-9 or 2^-12), or below f16's normal numbers 2^-25 of a unit that is 2^-7 of the largest.
    Codes' parts end at 2^-40 of the largest. The sums over n tokens keep 2^-23 per addition. All relative to sum p |v|, twice
    because the denominator has the same errors."""
    L, n, Hq, d = q.shape
    G = Hq // c.n_kv_heads
    scale = scale or 1.0 / math.sqrt(d)
    out = torch.zeros(L, n, Hq, d, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    eps = torch.finfo(q.dtype).eps
    for r, (p, s) in enumerate(zip(places, seqs)):
        if p < 0:
            continue
        t = torch.arange(p + 1, device="cuda")
        if window:
            t = t[(t > p - window) | (t < sinks)]
        for l in range(L):
            for h in range(c.n_kv_heads):
                k, v = tokens(c, table, s, layer + l, h, t)
                if rounded_p:
                    k, v = k.to(q.dtype).double(), v.to(q.dtype).double()
                qq = q[l, r, h * G:(h + 1) * G].double()
                x = qq @ k.T * scale
                w = torch.softmax(x, -1)
                out[l, r, h * G:(h + 1) * G] = w @ v
                dx = ((qq.abs() @ k.abs().T * scale).amax(-1) * (d * 2.0**-23) + x.abs().amax(-1) * 2.0**-22)[:, None]
                rel = 2 * dx + 2.0**-22 + (eps / 2 if rounded_p else 2.0**-22) + (len(t) + 64) * 2.0**-23
                least = 2.0**-32 if rounded_p and q.dtype == torch.float16 else 2.0**-40
                tol[l, r, h * G:(h + 1) * G] = 2 * rel * (w @ v.abs()) + 2 * least * v.abs().sum(0) * w.amax(-1, keepdim=True)
    return out, tol


def check(out, ref, tol):
    t = tol + (torch.finfo(out.dtype).eps / 2 * (ref.abs() + tol) + torch.finfo(out.dtype).smallest_normal
               if out.dtype != torch.float32 else 2.0**-24 * ref.abs())
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= t).all(), f"worst {((err - t).max()).item():.3e} over, max error {err.max().item():.3e}"


def places_of(lens):
    return [n - 1 for n in lens], range(len(lens))


# ------------------------------------------------------------------ one new token
ONE = [
    # page, d, H, G, dtype, codes, lens, window, sinks, L
    (16, 128, 2, 4, "bf16", None, [1, 15, 16, 17, 300, 0], 16, 0, 1),
    (16, 128, 2, 4, "bf16", None, [1, 100, 500, 333, 20], 1, 5, 2),
    (32, 64, 4, 1, "f16", None, [200, 201, 199, 64, 65], 64, 40, 1),
    (64, 128, 1, 7, "bf16", None, [2000, 70, 1], 100, 65, 1),
    (128, 64, 1, 11, "f16", None, [700, 129, 128, 127], 200, 3, 2),
    (128, 128, 1, 16, "bf16", None, [513, 1000], 127, 130, 1),
    (16, 128, 2, 4, "bf16", "int8", [1, 15, 16, 17, 300, 0], 0, 0, 2),
    (16, 64, 4, 1, "f16", "int8", [600, 1, 33], 0, 0, 1),
    (32, 128, 2, 4, "bf16", "e4m3", [1000, 31, 32, 33], 0, 0, 1),
    (64, 64, 3, 2, "bf16", "e4m3", [65, 500, 63, 1], 0, 0, 2),
    (128, 128, 1, 16, "f16", "int8", [513, 1000, 7], 0, 0, 1),
    (16, 64, 1, 11, "f16", "e4m3", [300, 200], 0, 0, 1),
    (16, 128, 2, 2, "f16", "e4m3", [700, 300, 20], 50, 17, 1),
    (64, 128, 8, 1, "bf16", "int8", [2000, 100, 64], 65, 4, 1),
]


@pytest.mark.parametrize("page,d,H,G,dtype,codes,lens,window,sinks,L", ONE)
@pytest.mark.parametrize("out", ["f32", "in"])
def test_one_token(pk, page, d, H, G, dtype, codes, lens, window, sinks, L, out):
    c, table, n = make(pk, lens, page, L + 1, H, d, dtype, codes, seed=len(lens))
    q = torch.randn(L, len(lens), G * H, d, generator=torch.Generator().manual_seed(5)).to(DT[dtype]).cuda()
    got = c.attend(q, table, n, out_dtype=torch.float32 if out == "f32" else DT[dtype], window=window, sinks=sinks, layer=1)
    check(got, *reference(c, q, table, *places_of(lens), window, sinks, layer=1))
    assert c.status() == 0


@pytest.mark.parametrize("codes", [None, "int8", "e4m3"])
def test_one_token_of_a_long_sequence(pk, codes):
    lens = [40001, 9000]
    c, table, n = make(pk, lens, 16, 1, 2, 128, "bf16", codes)
    q = torch.randn(1, 2, 8, 128).to(torch.bfloat16).cuda()
    for window, sinks in ((0, 0), (4096, 4), (39990, 16), (40001, 0), (1 << 31 - 1, 1 << 31 - 1)):
        got = c.attend(q, table, n, window=window, sinks=sinks)
        check(got, *reference(c, q, table, *places_of(lens), window, sinks))


@pytest.mark.parametrize("codes", [None, "int8"])
def test_pages_behind_the_window_may_be_gone(pk, codes):
    lens, page, window, sinks = [500, 41, 260], 16, 70, 20
    c, table, n = make(pk, lens, page, 1, 2, 64, "f16", codes)
    q = torch.randn(1, 3, 4, 64).half().cuda()
    want = c.attend(q, table, n, window=window, sinks=sinks)
    gone = table.clone()
    for s, ln in enumerate(lens):
        gone[s, 2:max(2, (ln - window) // page)] = -1
    assert torch.equal(c.attend(q, gone, n, window=window, sinks=sinks), want)
    starts = ints([0, 1, 2, 3])
    rows = c.attend_rows(q, table, n, starts, window=window, sinks=sinks)
    assert torch.equal(c.attend_rows(q, gone, n, starts, window=window, sinks=sinks), rows)
    assert c.status() == 0
    c.attend(q, gone, n)
    with pytest.raises(pk.PolyKVError):
        c.status()


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_codes_with_extreme_scales_and_queries(pk, codes, dtype):
    """Scales that differ by 2^60 from page to page, queries near the ends of their type."""
    lens = [100, 64]
    c, table, n = make(pk, lens, 16, 1, 1, 128, dtype, codes, poison=False)
    g = torch.Generator().manual_seed(1)
    c.scales.copy_(torch.exp2(torch.randint(-40, 20, c.scales.shape, generator=g).float()))
    for size in (1.0, 1e-4, 6e4 if dtype == "f16" else 1e30):
        q = (torch.randn(1, 2, 4, 128, generator=g).clamp(-1, 1) * size).to(DT[dtype]).cuda()
        scale = 1.0 / (size * 2.0**28)
        check(c.attend(q, table, n, softmax_scale=scale), *reference(c, q, table, *places_of(lens), 0, 0, scale=scale))


def test_codes_of_chosen_pages(pk):
    lens, page = [300, 40, 0, 129], 16
    c, table, n = make(pk, lens, page, 1, 2, 64, "bf16", "e4m3")
    q = torch.randn(1, 4, 4, 64, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    chosen = torch.tensor([[0, 5, 18], [0, 1, 2], [-1, -1, -1], [2, 8, -1]], dtype=torch.int32)[None, :, None].expand(1, 4, 2, 3).contiguous().cuda()
    out = c.attend(q, table, n, selected=chosen)
    for s in range(4):
        at = [t for p in chosen[0, s, 0].tolist() if p >= 0 for t in range(p * page, min((p + 1) * page, lens[s]))]
        for h in range(2):
            if not at:
                assert (out[0, s] == 0).all()
                continue
            k, v = tokens(c, table, s, 0, h, torch.tensor(at, device="cuda"))
            want = torch.softmax(q[0, s, 2 * h:2 * h + 2].double() @ k.T / 8, -1) @ v
            # logits of up to about 10 off by 64 2^-23 of their terms, sums of 48: 2^-15 of the values is ample
            assert ((out[0, s, 2 * h:2 * h + 2] - want).abs() <= 2.0**-15 * v.abs().amax()).all()
    assert c.status() == 0


def test_codes_of_a_block_that_is_not_finite(pk):
    """Only the rows that see such a block are NaN."""
    lens = [100, 100]
    c, table, n = make(pk, lens, 16, 1, 2, 64, "bf16", "int8")
    q = torch.randn(1, 2, 4, 64).to(torch.bfloat16).cuda()
    want = c.attend(q, table, n)
    c.scales[0, table[0, 2].item(), 1, 0] = math.nan
    got = c.attend(q, table, n)
    assert got[0, 0, 2:].isnan().all() and torch.equal(got[0, 0, :2], want[0, 0, :2]) and torch.equal(got[0, 1], want[0, 1])
    seen = c.attend(q, table, n, window=50)      # the block is behind the window
    assert torch.isfinite(seen).all()


def test_codes_keep_small_probabilities(pk):
    """One token with a small value far above the many others: what they add does not go missing."""
    n = 131072
    k = torch.zeros(1, n // 64, 1, 64, 64, dtype=torch.int8, device="cuda")
    v = torch.full_like(k, 100)
    k[0, 0, 0, 0], v[0, 0, 0, 0] = 100, 0
    scales = torch.full((1, n // 64, 1, 2), 2.0**-6, device="cuda")
    c = pk.PageCache(k, v, scales=scales, row_dtype=torch.float16)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None]
    q = torch.full((1, 1, 1, 64), 1.0, dtype=torch.float16, device="cuda")
    nats = 18.0
    got = c.attend(q, table, ints([n]), softmax_scale=nats / 100.0)
    p = math.exp(-nats)
    # the logit is off by at most 2^-20 of itself (18 nats)
    want = (n - 1) * p / (1 + (n - 1) * p) * 100 / 64
    assert abs(got.double() - want).max().item() <= want * (18 * 2.0**-20 + 2.0**-18)


# ------------------------------------------------------------------ codes appended and read back
def rope_plain(x, pos, inv, inter):
    x = x.double()
    ang = pos.double()[:, None, None] * inv
    cos, sin = ang.cos(), ang.sin()
    half = inv.shape[0]
    y = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if inter else (x[..., :half], x[..., half:2 * half])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if inter:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ra, rb
    else:
        y[..., :half], y[..., half:2 * half] = ra, rb
    return y


def pow2_for(amax, top):
    """The smallest power of two under which amax is at most top."""
    if amax == 0:
        return 2.0**-100
    e = math.ceil(math.log2(amax / top))
    while 2.0**(e - 1) * top >= amax:
        e -= 1
    while 2.0**e * top < amax:
        e += 1
    return 2.0**max(-100, e)


def nearest(x, kind):
    if kind is torch.int8:
        return x.round()
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0**-30))).clamp_min(-6) - 3)
    return (x / step).round() * step


class Blocks:
    """What the pages of one sequence hold, appended run by run, in 64 bits: per layer, head and page (scale, values)."""

    def __init__(self, L, H, d, page, codes):
        self.page, (self.kind, self.top) = page, KIND[codes]
        self.at = [[[] for _ in range(H)] for _ in range(L)]

    def append(self, x):   # [L][n][H][d], 64 bits
        for l in range(x.shape[0]):
            for h in range(x.shape[2]):
                blocks = self.at[l][h]
                rows, i = x[l, :, h], 0
                while i < rows.shape[0]:
                    if not blocks or blocks[-1][1].shape[0] == self.page:
                        blocks.append((0.0, rows[:0]))
                    old, held = blocks[-1]
                    part = rows[i:i + self.page - held.shape[0]]
                    i += part.shape[0]
                    s = max(old, pow2_for(part.abs().max().item(), self.top))
                    blocks[-1] = (s, torch.cat([nearest(held / s, self.kind) * s, nearest(part / s, self.kind) * s]))

    def values(self):
        return torch.stack([torch.stack([torch.cat([v for _, v in b]) for b in layer], 1) for layer in self.at])

    def scales(self):
        return [[[s for s, _ in b] for b in layer] for layer in self.at]


APPENDS = [
    # page, d, H, G, dtype, codes, runs of each sequence
    (16, 128, 2, 4, "bf16", "int8", [[1] * 20, [5, 1, 1, 30, 1], [0, 0, 17, 16, 16]]),
    (16, 64, 4, 1, "f16", "e4m3", [[33, 1, 1], [1] * 3, [16, 16, 1]]),
    (32, 128, 1, 7, "bf16", "e4m3", [[70, 3], [1, 31], [100, 28]]),
    (64, 128, 2, 2, "f16", "int8", [[200, 1, 1, 1], [63, 1, 1, 1], [1, 64, 64, 64]]),
    (64, 64, 3, 1, "bf16", "int8", [[130, 1], [5, 200]]),
    (128, 128, 2, 1, "bf16", "int8", [[300, 1, 90], [127, 1, 1]]),
    (128, 64, 5, 3, "f16", "e4m3", [[129, 200], [1, 1]]),
]


@pytest.mark.parametrize("page,d,H,G,dtype,codes,runs", APPENDS)
def test_append_codes_without_rotation(pk, page, d, H, G, dtype, codes, runs):
    """Dividing by a power of two is exact, so scales and codes are the 64-bit form's, rewritten blocks among them."""
    L, A = 2, len(runs)
    c = pk.PageCache.empty(L, H, d, 40, page, dtype, codes=codes)
    raw(c.k_pages).fill_(0x7F), raw(c.v_pages).fill_(0x7F), c.scales.fill_(math.nan)   # leftovers
    ends = [sum(r) for r in runs]
    table = ints([[a * 12 + i for i in range(12)] for a in range(A)])
    g = torch.Generator().manual_seed(page + d)
    want = [[Blocks(L, H, d, page, codes) for _ in range(2)] for _ in range(A)]
    lens = [0] * A
    for step in range(max(map(len, runs))):
        new = [r[step] if step < len(r) else 0 for r in runs]
        n = sum(new)
        # sizes rise and fall by powers of ten, rows of zeros among them
        size = torch.exp(2.5 * torch.randn(L, n, H, 1, generator=g)) * (torch.rand(L, n, H, 1, generator=g) > 0.1)
        k, v = ((torch.randn(L, n, H, d, generator=g) * size).to(DT[dtype]).cuda() for _ in range(2))
        starts = [0]
        for x in new:
            starts.append(starts[-1] + x)
        if all(x == 1 for x in new):
            c.append(k, v, table, ints(lens))
        else:
            c.append(k, v, table, ints(lens), starts=ints(starts))
        for a in range(A):
            for x, w in zip((k, v), want[a]):
                w.append(x[:, starts[a]:starts[a + 1]].double())
        lens = [a + b for a, b in zip(lens, new)]
    starts = [0]
    for x in ends:
        starts.append(starts[-1] + x)
    k, v = c.gather(table, ints(lens), ints(starts), starts[-1])
    for a in range(A):
        for i, (x, w) in enumerate(zip((k, v), want[a])):
            ref = w.values().to(DT[dtype])     # exact in bf16; rounded once in f16
            assert torch.equal(x[:, starts[a]:starts[a + 1]], ref)
            for l in range(L):
                for h in range(H):
                    for p, s in enumerate(w.scales()[l][h]):
                        assert c.scales[l, table[a, p].item(), h, i].item() == s
    assert c.status() == 0


@pytest.mark.parametrize("page,d,H,G,dtype,codes,runs", APPENDS)
@pytest.mark.parametrize("inter,rot", [(False, None), (True, None), (True, 32), (False, 48)])
def test_append_codes_with_rotation(pk, page, d, H, G, dtype, codes, runs, inter, rot):
    """Each value back within half a step of its rotated original (a step under the block's scale: 1, or e4m3's), half a
    step more for each time that the scale rose, and the rotation's own error (angles to 2^-24 turns of 2 pi, the products)."""
    L, A = 1, len(runs)
    rot = rot or d
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    rope = pk.Rope(inv, interleaved=inter)
    c = pk.PageCache.empty(L, H, d, 40, page, dtype, codes=codes)
    table = ints([[a * 12 + i for i in range(12)] for a in range(A)])
    g = torch.Generator().manual_seed(page + d)
    lens, offset, kept = [0] * A, 1000, [[[], []] for _ in range(A)]
    for step in range(max(map(len, runs))):
        new = [r[step] if step < len(r) else 0 for r in runs]
        n = sum(new)
        k, v = (torch.randn(L, n, H, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
        q = torch.randn(L, n, G * H, d, generator=g).to(DT[dtype]).cuda()
        starts = [0]
        for x in new:
            starts.append(starts[-1] + x)
        pos = torch.tensor([lens[a] + i + offset for a in range(A) for i in range(new[a])], device="cuda")
        qo = c.append(k, v, table, ints(lens), starts=None if all(x == 1 for x in new) else ints(starts), q=q, rope=rope,
                      pos_offset=offset)
        rq, rk = (rope_plain(x, pos, inv.cuda(), inter) for x in (q, k))
        near = 2.0**-21 * q.double().abs().amax()
        assert ((qo.double() - rq).abs() <= torch.finfo(q.dtype).eps / 2 * rq.abs() + near).all()
        for a in range(A):
            kept[a][0].append(rk[:, starts[a]:starts[a + 1]])
            kept[a][1].append(v[:, starts[a]:starts[a + 1]].double())
        lens = [x + y for x, y in zip(lens, new)]
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    back = c.gather(table, ints(lens), ints(starts), starts[-1])
    for a in range(A):
        t = torch.arange(lens[a], device="cuda")
        for i in range(2):
            x = torch.cat(kept[a][i], 1)
            s = c.scales[:, table[a].long()[t // page], :, i].double()[..., None]
            # the last rounding, and less than a step in all for those before (1/2 + 1/4 + ... of the last scale's)
            if codes == "int8":
                tol = s
            else:
                tol = 2.0**-3 * x.abs() + 2.0**-9 * s
            got = back[i][:, starts[a]:starts[a + 1]].double()
            # reading back rounds to f16 once more
            assert ((got - x).abs() <= tol * 1.001 + 2.0**-20 * x.abs().amax() + 2.0**-11 * x.abs()).all()
    assert c.status() == 0


def test_append_codes_not_finite(pk):
    c = pk.PageCache.empty(1, 2, 64, 4, 16, "bf16", codes="e4m3")
    table = ints([[0, 1], [2, 3]])
    k = torch.randn(1, 2, 2, 64).to(torch.bfloat16).cuda()
    k[0, 0, 1, 5] = math.inf
    c.append(k, k, table, ints([0, 0]))
    assert c.scales[0, 0, 1].isnan().all() and not c.scales[0, [0, 2]][:, 0].isnan().any() and not c.scales[0, 2].isnan().any()
    one = torch.randn(1, 2, 2, 64).to(torch.bfloat16).cuda()
    c.append(one, one, table, ints([1, 1]))           # still not: its page goes on
    assert c.scales[0, 0, 1].isnan().all()
    got = c.gather(table, ints([2, 2]), ints([0, 2, 4]), 4)[0]
    assert got[0, :2, 1].isnan().all() and torch.isfinite(got[0, :2, 0]).all() and torch.isfinite(got[0, 2:]).all()
    c.append(one, one, table, ints([0, 0]))           # begun again
    assert torch.isfinite(c.scales[0, [0, 2]]).all()


def test_append_codes_skips_idle_slots_and_bad_pages(pk):
    c = pk.PageCache.empty(1, 2, 64, 4, 16, "f16", codes="int8")
    c.k_pages.fill_(3), c.v_pages.fill_(4), c.scales.fill_(5.0)
    table = ints([[0], [9], [2], [-1]])
    k = torch.randn(1, 4, 2, 64).half().cuda()
    c.append(k, k, table, ints([0, 0, -1, 0]))
    with pytest.raises(pk.PolyKVError):
        c.status()
    assert (c.k_pages[0, 1:] == 3).all() and (c.v_pages[0, 1:] == 4).all() and (c.scales[0, 1:] == 5).all()
    assert (c.k_pages[0, 0, :, 1:] == 3).all() and not (c.k_pages[0, 0, :, 0] == 3).all()
    c.append(k, k, table, ints([16, 0, 0, 0]), starts=ints([0, 2, 3, 3, 4]))     # beyond the table; a bad page; none; a bad page
    with pytest.raises(pk.PolyKVError):
        c.status()
    assert (c.k_pages[0, 1:] == 3).all() and (c.scales[0, 1:] == 5).all()


@pytest.mark.parametrize("codes", [None, "int8", "e4m3"])
def test_gather(pk, codes):
    lens = [100, 0, 33, 16, -1]
    c, table, n = make(pk, lens, 16, 3, 2, 64, "bf16", codes)
    counts = [37, 0, 33, 1, 0]
    starts = [0, 37, 37, 70, 71, 71]
    k = torch.full((2, 75, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    got = c.gather(table, n, ints(starts), 75, k=k, v=v, layer=1)
    assert got[0] is k or got[0].data_ptr() == k.data_ptr()
    assert (k[:, 71:] == 9).all() and (v[:, 71:] == 9).all()
    for s, cnt in enumerate(counts):
        t = torch.arange(max(0, lens[s]) - cnt, max(0, lens[s]), device="cuda")
        for l in range(2):
            for h in range(2):
                rk, rv = tokens(c, table, s, 1 + l, h, t)
                assert torch.equal(k[l, starts[s]:starts[s] + cnt, h].double(), rk.to(torch.bfloat16).double())
                assert torch.equal(v[l, starts[s]:starts[s] + cnt, h].double(), rv.to(torch.bfloat16).double())
    assert c.status() == 0
    c.gather(table, ints([100, 0, 32, 16, -1]), ints(starts), 75)    # more rows than tokens
    with pytest.raises(pk.PolyKVError):
        c.status()


# ------------------------------------------------------------------ runs of rows
ROWS = [
    # page, d, H, G, dtype, codes, old, new, window, sinks
    (16, 128, 2, 4, "bf16", None, [0, 100, 7, 0], [1, 1, 5, 40], 0, 0),
    (32, 128, 1, 4, "bf16", None, [0], [700], 0, 0),
    (64, 64, 2, 1, "f16", None, [0, 300], [300, 129], 0, 0),
    (16, 64, 1, 8, "bf16", None, [50, 0, 3], [17, 33, 0], 0, 0),
    (128, 128, 1, 7, "f16", None, [10, 200], [37, 19], 0, 0),
    (16, 128, 1, 16, "bf16", None, [130], [70], 0, 0),
    (32, 128, 1, 4, "f16", None, [0, 500], [400, 70], 64, 4),
    (16, 64, 2, 2, "bf16", None, [600, 0], [150, 300], 100, 40),
    (64, 128, 1, 1, "bf16", None, [0], [1000], 1, 0),
    (64, 64, 1, 4, "f16", None, [333], [600], 257, 130),
    (128, 64, 1, 3, "bf16", None, [1000, 90], [3, 260], 130, 1),
    (16, 64, 1, 130, "bf16", None, [20], [3], 0, 0),
    (16, 128, 2, 4, "bf16", "int8", [0, 100, 7], [60, 1, 5], 0, 0),
    (32, 64, 1, 2, "f16", "e4m3", [0, 300], [200, 30], 50, 4),
    (64, 128, 1, 8, "bf16", "e4m3", [0], [300], 0, 0),
    (128, 64, 2, 1, "f16", "int8", [200], [140], 0, 0),
]


def rows_case(pk, page, d, H, G, dtype, codes, old, new, L=1, seed=3, behind=2):
    lens = [a + b for a, b in zip(old, new)]
    c, table, n = make(pk, lens, page, L + 1, H, d, dtype, codes, seed=seed)
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    q = torch.randn(L, starts[-1] + behind, G * H, d, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()
    seqs = [s for s in range(len(new)) for _ in range(new[s])] + [0] * behind
    places = [old[s] + i for s in range(len(new)) for i in range(new[s])] + [-1] * behind
    return c, table, n, ints(starts), q, places, seqs


@pytest.mark.parametrize("page,d,H,G,dtype,codes,old,new,window,sinks", ROWS)
def test_rows(pk, page, d, H, G, dtype, codes, old, new, window, sinks):
    c, table, n, starts, q, places, seqs = rows_case(pk, page, d, H, G, dtype, codes, old, new)
    out = torch.zeros_like(q)      # rows behind the last stay as they are
    got = c.attend_rows(q, table, n, starts, window=window, sinks=sinks, layer=1, out=out)
    assert got.data_ptr() == out.data_ptr()
    check(out, *reference(c, q, table, places, seqs, window, sinks, layer=1, rounded_p=True))
    assert c.status() == 0


def test_rows_of_several_layers_and_strides(pk):
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 64, 2, 2, "f16", None, [30, 0, 5], [20, 50, 1], L=3)
    wide = torch.zeros(3, q.shape[1], 9, 64, dtype=torch.float16, device="cuda")
    wide[:, :, 2:6] = q
    want = c.attend_rows(q, table, n, starts, layer=1)[:, :71]
    assert torch.equal(c.attend_rows(wide[:, :, 2:6], table, n, starts, layer=1)[:, :71], want)
    one = q[:1].expand(3, -1, -1, -1)       # one tensor for all layers
    want = c.attend_rows(one.contiguous(), table, n, starts, layer=1, softmax_scale=0.3)[:, :71]
    assert torch.equal(c.attend_rows(one, table, n, starts, layer=1, softmax_scale=0.3)[:, :71], want)


@pytest.mark.parametrize("G,d,dtype", [(1, 64, "f16"), (4, 128, "bf16")])
def test_rows_agree_with_one_token(pk, G, d, dtype):
    """A run of single rows is the decode call."""
    lens = [1, 77, 300, 20, 513]
    c, table, n = make(pk, lens, 32, 1, 2, d, dtype)
    q = torch.randn(1, 5, 2 * G, d).to(DT[dtype]).cuda()
    got = c.attend_rows(q, table, n, ints([0, 1, 2, 3, 4, 5]), window=100, sinks=3)
    check(got, *reference(c, q, table, *places_of(lens), 100, 3, rounded_p=True))


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_keep_to_what_they_see(pk, bad, window, sinks):
    """Keys and values that are not finite reach the rows that see them, and no others."""
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 64, 1, 2, "bf16", None, [40], [200], behind=0)
    want = c.attend_rows(q, table, n, starts, window=window, sinks=sinks, layer=1)
    for what in ("v", "k"):
        t = 110
        pages = c.v_pages if what == "v" else c.k_pages
        old = pages[1, table[0, t // 16].item(), 0, t % 16].clone()
        pages[1, table[0, t // 16].item(), 0, t % 16] = bad
        got = c.attend_rows(q, table, n, starts, window=window, sinks=sinks, layer=1)
        pages[1, table[0, t // 16].item(), 0, t % 16] = old
        sees = torch.tensor([p >= t and (not window or t > p - window or t < sinks) for p in places]).cuda()
        # the same to the last bits: a row may be computed another way beside one that is not finite
        assert torch.allclose(got[0, ~sees].float(), want[0, ~sees].float(), rtol=2.0**-6, atol=2.0**-7)
        if what == "v":
            assert not torch.isfinite(got[0, sees]).any()
        else:
            assert got[0, sees].isnan().any()
        assert (~sees).sum() > 20 and sees.sum() > 20


def test_rows_leave_idle_slots_and_flag_broken_starts(pk):
    c, table, n, _, q, places, seqs = rows_case(pk, 16, 64, 1, 2, "f16", None, [10, 20, 30], [5, 6, 7], behind=0)
    out = torch.full_like(q, 7.0)
    lens = n.clone()
    lens[1] = -1
    c.attend_rows(q, table, lens, ints([0, 5, 11, 18]), layer=1, out=out)
    assert (out[:, 5:11] == 7).all() and not (out[:, :5] == 7).any() and not (out[:, 11:] == 7).any()
    assert c.status() == 0
    out.fill_(7.0)
    lens[1], lens[2] = 3, 1000      # fewer tokens than rows; beyond the table
    c.attend_rows(q, table, lens, ints([0, 5, 11, 18]), layer=1, out=out)
    assert (out[:, 5:] == 7).all() and not (out[:, :5] == 7).any()
    with pytest.raises(pk.PolyKVError):
        c.status()
    c.attend_rows(q, table, n, ints([0, 30, 11, 18]), layer=1, out=out)
    with pytest.raises(pk.PolyKVError):
        c.status()


def test_rows_without_a_page_leave_its_tokens_out(pk):
    c, table, n, starts, q, places, seqs = rows_case(pk, 32, 128, 1, 4, "bf16", None, [100], [60], behind=0)
    cut = table.clone()
    cut[0, 1] = 1 << 20
    got = c.attend_rows(q, cut, n, starts, layer=1)
    with pytest.raises(pk.PolyKVError):
        c.status()
    # the same as with values that count for nothing: keys whose logits are -inf
    page = table[0, 1].item()
    ref = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    for r, p in enumerate(places):
        t = torch.arange(p + 1, device="cuda")
        k, v = tokens(c, table, 0, 1, 0, t[t // 32 != 1])
        ref[0, r] = torch.softmax(q[0, r].double() @ k.T / math.sqrt(128), -1) @ v
    assert ((got.double() - ref).abs() <= 0.02).all() and page >= 0


def test_rows_peaked_and_huge_logits(pk):
    for dtype in ("bf16", "f16"):
        c, table, n, starts, q, places, seqs = rows_case(pk, 16, 128, 1, 4, dtype, None, [0, 200], [300, 90], behind=0)
        for size in (30.0, 300.0):
            check(c.attend_rows(q * size, table, n, starts, layer=1),
                  *reference(c, q * size, table, places, seqs, 0, 0, layer=1, rounded_p=True))


def test_rows_rising_logits(pk):
    """The running maximum rises in every tile: what was summed before is scaled down each time."""
    c, table, n, starts, q, places, seqs = rows_case(pk, 32, 64, 1, 2, "bf16", None, [600], [100], behind=0)
    t = torch.arange(table.shape[1] * 32, device="cuda")
    c.k_pages[1, table[0].long(), 0] = (0.05 * t.view(-1, 32, 1) / 8).to(torch.bfloat16).expand(-1, -1, 64)
    q = q.abs()
    check(c.attend_rows(q, table, n, starts, layer=1), *reference(c, q, table, places, seqs, 0, 0, layer=1, rounded_p=True))


def test_rows_of_queries_that_share_their_places(pk):
    """Strides of zero: one query for all heads, one for all rows."""
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 64, 2, 2, "bf16", None, [30, 0], [20, 150], behind=0)
    for one in (q[:, :, :1].expand(-1, -1, 4, -1), q[:, :1].expand(-1, 170, -1, -1), q[:, :1, :1].expand(-1, 170, 4, -1)):
        assert torch.equal(c.attend_rows(one, table, n, starts, layer=1), c.attend_rows(one.contiguous(), table, n, starts, layer=1))


def test_rows_of_none(pk):
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 64, 1, 2, "f16", None, [30], [20], behind=0)
    assert c.attend_rows(q[:, :0], table, n, ints([0, 0])).shape == (1, 0, 2, 64)
    k, v = c.gather(table, n, ints([0, 0]), 0)
    assert k.shape == v.shape == (2, 0, 1, 64)


@pytest.mark.parametrize("codes", [None, "e4m3"])
def test_shared_out_rows_repeat_to_the_bit(pk, codes):
    """Few rows behind a long context: parts are joined in their order, whichever block comes last."""
    c, table, n, starts, q, places, seqs = rows_case(pk, 64, 128, 2, 4, "bf16", codes, [30000, 100, 0], [2, 3, 40], behind=0)
    want = c.attend_rows(q, table, n, starts, layer=1)
    for _ in range(20):
        assert torch.equal(c.attend_rows(q, table, n, starts, layer=1), want)


def test_rows_stalled_wait_times_out_and_context_survives(pk):
    """The producer is told to copy nothing: the bounded waits give up, the status says so, and the next call is right."""
    import os
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 128, 1, 4, "bf16", None, [2000, 30], [3, 90], behind=0)
    os.environ["POLYKV_TEST_STALL"] = "1"
    try:
        c.attend_rows(q, table, n, starts, layer=1)
        torch.cuda.synchronize()
    finally:
        del os.environ["POLYKV_TEST_STALL"]
    with pytest.raises(pk.PolyKVError) as e:
        c.status()
    assert e.value.status == 5
    assert c.status() == 0
    for _ in range(2):
        check(c.attend_rows(q, table, n, starts, layer=1), *reference(c, q, table, places, seqs, 0, 0, layer=1, rounded_p=True))
    assert c.status() == 0


def test_many_short_runs(pk):
    g = torch.Generator().manual_seed(2)
    new = torch.randint(0, 6, (300,), generator=g).tolist()
    old = torch.randint(0, 90, (300,), generator=g).tolist()
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 64, 2, 1, "f16", None, old, new)
    out = torch.zeros_like(q)
    c.attend_rows(q, table, n, starts, window=40, sinks=2, layer=1, out=out)
    check(out, *reference(c, q, table, places, seqs, 40, 2, layer=1, rounded_p=True))


@pytest.mark.parametrize("A", [14, 32, 33])
def test_rows_in_several_turns(pk, A):
    """More blocks of rows than the card runs at once, from few sequences and from more, idle ones and some without rows among
    them: each is taken once, whoever takes it, call after call and under a graph; a stalled call leaves the next one right."""
    import os
    g = torch.Generator().manual_seed(A)
    new = torch.randint(1, 9, (A,), generator=g).tolist()
    old = torch.randint(0, 700, (A,), generator=g).tolist()
    new[3], new[A - 1], new[5] = 0, 0, 40
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 64, 16, 1, "f16", None, old, new, behind=3)
    n[2] = -1
    places = [-1 if s == 2 else p for p, s in zip(places, seqs)]
    want = None
    ref = reference(c, q, table, places, seqs, 300, 5, layer=1, rounded_p=True)
    for _ in range(5):
        out = torch.zeros_like(q)
        c.attend_rows(q, table, n, starts, window=300, sinks=5, layer=1, out=out)
        check(out, *ref)
        assert want is None or torch.equal(out, want)
        want = out
    graph, again = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        c.attend_rows(q, table, n, starts, window=300, sinks=5, layer=1, out=again)
    for _ in range(3):
        again.zero_()
        graph.replay()
        assert torch.equal(again, want)
    os.environ["POLYKV_TEST_STALL"] = "1"
    try:
        c.attend_rows(q, table, n, starts, layer=1)
        torch.cuda.synchronize()
    finally:
        del os.environ["POLYKV_TEST_STALL"]
    with pytest.raises(pk.PolyKVError):
        c.status()
    out = torch.zeros_like(q)
    c.attend_rows(q, table, n, starts, window=300, sinks=5, layer=1, out=out)
    assert torch.equal(out, want) and c.status() == 0


def test_few_rows_of_a_long_context(pk):
    for codes in (None, "int8"):
        c, table, n, starts, q, places, seqs = rows_case(pk, 64, 128, 1, 4, "bf16", codes, [20000, 5000], [3, 1], behind=0)
        for window, sinks in ((0, 0), (9000, 70)):
            check(c.attend_rows(q, table, n, starts, window=window, sinks=sinks, layer=1),
                  *reference(c, q, table, places, seqs, window, sinks, layer=1, rounded_p=True))


@pytest.mark.parametrize("codes,dtype", [("int8", "f16"), ("e4m3", "bf16")])
def test_rows_over_codes_of_a_wide_table(pk, codes, dtype):
    """Far more places in the table than pages in the cache: the copies lie by page id."""
    c, table, n, starts, q, places, seqs = rows_case(pk, 128, 64, 64, 1, dtype, codes, [150], [3], behind=1)
    wide = torch.full((1, 1 << 18), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out = torch.zeros_like(q)
    c.attend_rows(q, wide, n, starts, window=90, sinks=4, layer=1, out=out)
    check(out, *reference(c, q, table, places, seqs, 90, 4, layer=1, rounded_p=True))


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_rows_over_codes_take_no_more_than_the_cache_twice(pk, codes):
    """The workspace of tables with many empty places, and pages that two sequences share, in a workspace that starts as NaN."""
    c, table, n, starts, q, places, seqs = rows_case(pk, 32, 64, 2, 2, "bf16", codes, [100, 200], [50, 30], L=2)
    table[0, :3] = table[1, :3]
    many = torch.full((2, 4096), -1, dtype=torch.int32, device="cuda")
    many[:, :table.shape[1]] = table
    seq = pk.PagesSeqs(many.data_ptr(), n.data_ptr(), many.shape[1], 2, 1, 2)
    need = pk.polykv_pages_attend_rows_workspace_size(c.handle, seq, 4, q.shape[1], 0, 0)
    plain = pk.PageCache.empty(3, 2, 64, c.n_pages, 32, "bf16")
    own = pk.polykv_pages_attend_rows_workspace_size(plain.handle, seq, 4, q.shape[1], 0, 0)
    assert need <= own + 4096 + 1024 + 2 * c.k_pages[1:].numel() * 2        # keys and values, two bytes each
    for tables in (many, table):
        size = pk.polykv_pages_attend_rows_workspace_size(c.handle, pk.PagesSeqs(tables.data_ptr(), n.data_ptr(), tables.shape[1], 2, 1, 2),
                                                          4, q.shape[1], 0, 0)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        ws[:4096] = 0
        out = torch.zeros_like(q)
        c.attend_rows(q, tables, n, starts, layer=1, out=out, workspace=ws)
        check(out, *reference(c, q, table, places, seqs, 0, 0, layer=1, rounded_p=True))
        assert not ws[:4096].any()
    assert c.status() == 0


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_rows_over_codes_at_the_end_of_f16(pk, codes):
    """The largest f16 values, as codes: what they stand for is finite, and so are the rows that see them."""
    c = pk.PageCache.empty(1, 1, 64, 8, 16, "f16", codes=codes)
    k = torch.randn(1, 40, 1, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    v = torch.full_like(k, 65504.0)
    v[:, ::2] = -65504.0
    table, n, starts = ints([[3, 1, 7, 0]]), ints([40]), ints([0, 40])
    c.append(k, v, table, ints([0]), starts=starts)
    assert torch.isfinite(c.gather(table, n, starts, 40)[1]).all()
    q = torch.randn(1, 40, 2, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    out = c.attend_rows(q, table, n, starts)
    assert torch.isfinite(out).all()


# ------------------------------------------------------------------ in a run
@pytest.mark.parametrize("dtype,codes,window,sinks", [("bf16", None, 40, 5), ("f16", "int8", 0, 0), ("bf16", "e4m3", 33, 16),
                                                      ("f16", None, 0, 0)])
def test_plan_append_attend(pk, dtype, codes, window, sinks):
    """Prompts, decode steps, rejected drafts, sequences that end and slots that are taken again: plan, append, attention."""
    A, H, G, d, page, P = 4, 2, 2, 64, 16, 60
    t = pk.PageTable(A, 20, P, page, window=window, sinks=sinks)
    c = pk.PageCache.empty(1, H, d, P, page, dtype, codes=codes)
    raw(c.k_pages).fill_(0x7F) if codes else c.k_pages.fill_(math.nan)
    raw(c.v_pages).fill_(0x7F) if codes else c.v_pages.fill_(math.nan)
    g = torch.Generator().manual_seed(9)
    k_all = [torch.zeros(0, H, d, dtype=DT[dtype], device="cuda") for _ in range(A)]
    v_all = [x.clone() for x in k_all]
    lens = [-1] * A
    big = 1 << 30
    steps = [([50, 0, 7, 0], None), ([1, 100, 1, 16], None), ([4, 4, 4, 4], "reject"), ([1, 1, 1, 1], None), ([0, 30, 1, 1], 2),
             ([1, 1, 33, 1], None), ([1, 1, 1, 0], 3), ([1, 1, 1, 90], None), ([1, 1, 1, 1], None)]
    for new, after in steps:
        n = sum(new)
        plan = t.plan(ints(new), n)
        rows = torch.randn(1, n, (G + 2) * H, d, generator=g).to(DT[dtype]).cuda()
        q, k, v = rows[:, :, :G * H], rows[:, :, G * H:(G + 1) * H], rows[:, :, (G + 1) * H:]
        c.append(k, v, t.block_table, plan.before, starts=plan.starts)
        out = c.attend_rows(q, t.block_table, plan.after, plan.starts, window=window, sinks=sinks)
        places, seqs, at = [], [], 0
        for s in range(A):
            if new[s]:
                old = max(0, lens[s])
                places += range(old, old + new[s])
                seqs += [s] * new[s]
                k_all[s] = torch.cat([k_all[s][:old], k[0, at:at + new[s]]])
                v_all[s] = torch.cat([v_all[s][:old], v[0, at:at + new[s]]])
                lens[s] = old + new[s]
            at += new[s]
        assert t.lens.tolist() == lens and plan.positions.tolist() == places
        check(out, *reference(c, q, t.block_table, places, seqs, window, sinks, rounded_p=True))
        if codes is None:     # what the slots map says is where the rows are
            flat = c.k_pages[0].transpose(1, 2).reshape(P * page, H, d)
            assert torch.equal(flat[plan.slots], k[0])
        last = torch.stack([q[0, plan.starts[s + 1] - 1] if new[s] else q[0, 0] * 0 for s in range(A)])[None]
        one = c.attend(last, t.block_table, plan.after, window=window, sinks=sinks)
        ref, tol = reference(c, last, t.block_table, [lens[s] - 1 if new[s] else -1 for s in range(A)], range(A), window, sinks)
        check(one, ref, tol)
        if after == "reject":
            keep = [lens[s] - 3 for s in range(A)]
            t.cut(ints(keep))
            lens = keep
        elif after is not None:
            t.cut(ints([-1 if s == after else big for s in range(A)]))
            lens[after] = -1
    assert c.status() == 0 and t.status() == 0


def test_codes_to_pool(pk):
    """An agent's 8-bit pages read back and encoded as a shared pool."""
    c, table, n = make(pk, [64], 16, 2, 2, 64, "bf16", "int8", poison=False)
    k, v = c.gather(table, n, ints([0, 64]), 64)
    pool = pk.Pool(2, 2, 64, 64, "bf16")
    pool.encode(k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous())
    q = torch.randn(2, 1, 4, 64).to(torch.bfloat16).cuda()
    out = pool.attend(q, 64)
    ref, _ = reference(c, q, table, [63], [0], 0, 0)
    assert (out.double() - ref).abs().max().item() < 0.6     # 3-bit values


def test_pool_with_private_codes(pk):
    """The pool and each agent's private tokens in 8 bits under one softmax."""
    L, H, G, d, T = 2, 2, 4, 128, 300
    g = torch.Generator().manual_seed(4)
    pool = pk.Pool(L, H, d, T, "bf16")
    pool.encode(*(torch.randn(L, H, T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)))
    lens = [70, 0, 333]
    c, table, n = make(pk, lens, 16, L, H, d, "bf16", "int8")
    w = pk.PageCache(*(torch.zeros(c.k_pages.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    w.scales_ = None
    for i, (x, y) in enumerate(((c.k_pages, w.k_pages), (c.v_pages, w.v_pages))):
        y.copy_((x.float() * c.scales[..., i, None, None].nan_to_num(0.0)))
    q = torch.randn(L, 3, G * H, d, generator=g).to(torch.bfloat16).cuda()
    got = pool.attend_with_pages(q, T, c, table, n)
    # the 16-bit cache of the same values, rounded to bf16: 2^-9 of each
    want = pool.attend_with_pages(q, T, w, table, n)
    assert torch.isfinite(got).all() and (got - want).abs().max().item() < 0.02


def test_streams_and_graphs(pk):
    lens = [200, 77]
    new = [90, 5]
    old = [110, 72]
    c, table, n, starts, q, places, seqs = rows_case(pk, 16, 128, 1, 4, "bf16", None, old, new, behind=0)
    c8, table8, n8 = make(pk, lens, 16, 1, 2, 64, "f16", "e4m3")
    q8 = torch.randn(1, 2, 4, 64).half().cuda()
    want = c.attend_rows(q, table, n, starts, window=64, sinks=4, layer=1)
    want8 = c8.attend(q8, table8, n8, window=50, sinks=2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            got.append((c.attend_rows(q, table, n, starts, window=64, sinks=4, layer=1, stream=s),
                        c8.attend(q8, table8, n8, window=50, sinks=2, stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want8) for a, b in got)
    graphs = []
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a, b = c.attend_rows(q, table, n, starts, window=64, sinks=4, layer=1), c8.attend(q8, table8, n8, window=50, sinks=2)
        graphs.append((g, s, a, b))
    for _ in range(5):
        for g, s, a, b in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want8) for _, _, a, b in graphs)
    # another length, the same graph
    n8.copy_(ints([33, 60]))
    ref = c8.attend(q8, table8, n8, window=50, sinks=2)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][3], ref)
