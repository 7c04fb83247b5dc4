"""Runs of rows where a block takes many units, long contexts with values that are not finite, and the ends of windows. Against
plain forms in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import serving_q8_encode_gb300 as pk
    return pk


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(pk, old, new, page, H, G, d, dtype, codes=None, seed=1, idle=()):
    """A cache whose sequences have old + new tokens in pages in random order, the new ones as rows: (cache, table, lens,
    starts, q)."""
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(old, new)]
    pages = [-(-n // page) for n in lens]
    P = sum(pages) + 2
    ids = torch.randperm(P, generator=g).tolist()
    table = torch.full((len(lens), max(pages) + 1), -1, dtype=torch.int32)
    for s, n in enumerate(pages):
        table[s, :n] = torch.tensor([ids.pop() for _ in range(n)])
    c = pk.PageCache.empty(1, H, d, P, page, dtype, codes=codes)
    k, v = (torch.randn(1, P, H, page, d, generator=g) for _ in range(2))
    if codes == "int8":
        c.k_pages.copy_((k * 30).round().clamp(-127, 127)), c.v_pages.copy_((v * 30).round().clamp(-127, 127))
        c.scales.copy_(torch.exp2(torch.randint(-6, -3, c.scales.shape, generator=g).float()))
    elif codes == "e4m3":
        c.k_pages.copy_(k * 30), c.v_pages.copy_(v * 30)
        c.scales.copy_(torch.exp2(torch.randint(-6, -3, c.scales.shape, generator=g).float()))
    else:
        c.k_pages.copy_(k), c.v_pages.copy_(v)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = torch.randn(1, starts[-1], G * H, d, generator=g).to(DT[dtype]).cuda()
    lens = [-1 if s in idle else n for s, n in enumerate(lens)]
    return c, table.cuda(), ints(lens), starts, q


def check(c, q, table, lens, starts, window, sinks, out, fill=None):
    """Against 64 bits, sequence by sequence. The tolerance, relative to sum p |v|: a logit is d exact products summed in fp32 (d 2^-23
    of sum |q k| at most) and rounded four times (2^-22 of itself); a probability has twice that, half a step of the row's type (once in
    the sum, once in the product, so twice in all) and the sums' 2^-23 an addition; f16's probabilities end at 2^-32 of the largest.
    Then the output's own rounding."""
    lens, page, d, Hq = lens.tolist(), c.page_tokens, q.shape[3], q.shape[2]
    G, eps = Hq // c.n_kv_heads, torch.finfo(q.dtype).eps
    for s, n in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        if a == b:
            continue
        if n < 0:
            assert fill is None or (out[0, a:b] == fill).all()
            continue
        t = torch.arange(n, device="cuda")
        ids = table[s].long()[t // page]
        k, v = (x[0, ids, :, t % page].double() for x in (c.k_pages, c.v_pages))      # [n][H][d]
        if c.scales is not None:
            k, v = (x * c.scales[0, ids, :, i].double()[..., None] for i, x in enumerate((k, v)))
            k, v = k.to(q.dtype).double(), v.to(q.dtype).double()
        k, v = (x.repeat_interleave(G, 1) for x in (k, v))
        p = torch.arange(n - (b - a), n, device="cuda")[:, None]
        see = t <= p
        if window:
            see &= (t > p - window) | (t < sinks)
        x = torch.einsum("rhd,thd->hrt", q[0, a:b].double(), k) / math.sqrt(d)
        big = torch.einsum("rhd,thd->hrt", q[0, a:b].double().abs(), k.abs()) / math.sqrt(d)
        x, big = x.masked_fill(~see, -math.inf), big.masked_fill(~see, 0.0)
        w = torch.softmax(x, -1)
        ref = torch.einsum("hrt,thd->rhd", w, v)
        dx = big.amax(-1) * (d * 2.0**-23) + x.masked_fill(~see, 0.0).abs().amax(-1) * 2.0**-22     # [h][r]
        rel = 2 * dx + 2.0**-22 + eps / 2 + (see.sum(-1) + 64) * 2.0**-23
        least = 2.0**-32 if q.dtype == torch.float16 else 2.0**-40
        tol = 2 * rel.T[..., None] * torch.einsum("hrt,thd->rhd", w, v.abs()) + 2 * least * w.amax(-1).T[..., None] * v.abs().sum(0)
        tol = tol + eps / 2 * (ref.abs() + tol) + torch.finfo(q.dtype).smallest_normal
        err = (out[0, a:b].double() - ref).abs()
        assert (err <= tol).all(), f"sequence {s}: {(err - tol).max().item():.3e} over"


SHORT = [
    # sequences, tokens before, rows, page, H, G, d, dtype, codes, window, sinks
    (64, 0, 100, 16, 32, 1, 64, "bf16", None, 0, 0),
    (300, 0, 128, 32, 32, 1, 64, "f16", None, 0, 0),
    (64, 128, 128, 16, 32, 1, 64, "bf16", None, 90, 3),
    (150, 100, 128, 64, 16, 2, 64, "f16", None, 0, 0),
    (64, 0, 100, 16, 32, 1, 64, "bf16", "int8", 0, 0),
    (100, 128, 128, 16, 32, 1, 64, "f16", "e4m3", 33, 20),
    (31, 900, 40, 32, 32, 1, 64, "bf16", None, 0, 0),
    (64, 0, 100, 16, 32, 1, 128, "bf16", None, 0, 0),
]


@pytest.mark.parametrize("A,old,new,page,H,G,d,dtype,codes,window,sinks", SHORT)
def test_many_short_sequences(pk, A, old, new, page, H, G, d, dtype, codes, window, sinks):
    """Many more units than blocks, each of few key tiles."""
    g = torch.Generator().manual_seed(A)
    olds = torch.randint(0, old + 1, (A,), generator=g).tolist()
    news = torch.randint(1, new + 1, (A,), generator=g).tolist()
    news[A // 2], news[0] = 0, new
    c, table, lens, starts, q = case(pk, olds, news, page, H, G, d, dtype, codes, idle=(3,))
    first = None
    for _ in range(4):
        out = torch.full_like(q, 9.0)
        c.attend_rows(q, table, lens, ints(starts), window=window, sinks=sinks, out=out)
        assert c.status() == 0
        assert first is None or torch.equal(out, first)
        first = out
    check(c, q, table, lens, starts, window, sinks, out, 9.0)


def test_rows_done_again_behind_a_long_context(pk):
    """An infinite value that only the last row sees: the 252 rows beside it are done again one by one, 32 a warp, each over 524,288
    tokens. At 0.19 us a token that is 3 s for a warp, beyond the waits' 2 s, while its block has another unit to do (320 units,
    152 blocks). And a NaN key that all rows see: they are NaN, without being done again."""
    T, n, H, G, d, page = 524288, 2560, 8, 4, 128, 128
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(3)
    shape = (1, T // page, H, page, d)
    k, v = (torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16) for _ in range(2))
    c = pk.PageCache(k, v)
    table = torch.randperm(T // page, generator=torch.Generator().manual_seed(3)).to(torch.int32)[None].cuda()
    q = torch.randn(1, n, H * G, d, generator=g, device=dev, dtype=torch.bfloat16)
    lens, starts, h, col = ints([T]), ints([0, n]), 5, 7
    want = c.attend_rows(q, table, lens, starts)
    assert c.status() == 0 and torch.isfinite(want).all()
    at = (0, table[0, -1].item(), h, page - 1, col)
    old, v[at] = v[at].item(), math.inf
    got = c.attend_rows(q, table, lens, starts)
    assert c.status() == 0
    v[at] = old
    mine = slice(h * G, (h + 1) * G)
    assert not torch.isfinite(got[0, -1, mine, col]).any()
    got[0, -1, mine, col] = want[0, -1, mine, col]
    # probabilities rounded to bf16 or not: half a step of each (2^-8) over values below 6, beside which the outputs' half steps are small
    assert (got.float() - want.float()).abs().max().item() <= 2.0**-8 * 6
    same = torch.ones(n, H * G, dtype=torch.bool, device=dev)
    same[-64:, mine] = False
    assert torch.equal(got[0][same], want[0][same])
    k[0, table[0, 0].item(), 2, 100, 3] = math.nan
    got = c.attend_rows(q, table, lens, starts)
    assert c.status() == 0
    assert got[0, :, 2 * G:3 * G].isnan().all()
    got[0, :, 2 * G:3 * G] = want[0, :, 2 * G:3 * G]
    assert torch.equal(got, want)


@pytest.mark.parametrize("codes", [None, "int8"])
@pytest.mark.parametrize("d,G,window,sinks", [(64, 1, 0, 0), (128, 4, 200, 5), (64, 2, 100, 30)])
def test_rows_beside_what_is_not_finite(pk, d, G, window, sinks, codes):
    """One NaN key, or one infinite value, in front of a few thousand tokens, and one among the rows: it reaches the rows that see
    it, in its head (and column), and no others."""
    old, n, H = 3000, 300, 2
    c, table, lens, starts, q = case(pk, [old], [n], 16, H, G, d, "bf16", codes, seed=d + G)
    want = c.attend_rows(q, table, lens, ints(starts), window=window, sinks=sinks)
    check(c, q, table, lens, starts, window, sinks, want)
    p = torch.arange(old, old + n)
    for t in (1, old + 120):
        sees = (p >= t) & ((p - t < window) | (t < sinks) if window else torch.tensor(True))
        page, slot = table[0, t // 16].item(), t % 16
        if codes is None:
            lo, hi = t, t                                  # what is not finite
            pages = c.v_pages
            kept, pages[0, page, 1, slot, 9] = pages[0, page, 1, slot, 9].item(), math.inf
        else:                                              # a whole block
            lo, hi = t // 16 * 16, t // 16 * 16 + 15
            kept = c.scales[0, page, 1, 1].item()
            c.scales[0, page, 1, 1] = math.nan
            sees = torch.stack([(p >= u) & ((p - u < window) | (u < sinks) if window else torch.tensor(True)) for u in range(lo, hi + 1)]).any(0)
        got = c.attend_rows(q, table, lens, ints(starts), window=window, sinks=sinks)
        assert torch.equal(got[0, :, :G], want[0, :, :G])
        bad = ~torch.isfinite(got[0, :, G:])
        assert torch.equal(bad[..., 9 if codes is None else slice(None)].flatten(1).all(1).cpu(), sees)
        if codes is None:
            assert not bad[..., :9].any() and not bad[..., 10:].any() and not bad[~sees.cuda()].any()
            pages[0, page, 1, slot, 9] = kept
        else:
            c.scales[0, page, 1, 1] = kept
        # probabilities rounded to bf16 or not, half a step of each (2^-8) over values below 8, and two half steps of the output
        ok = torch.isfinite(got)
        assert (got[ok].float() - want[ok].float()).abs().max().item() <= 3 * 2.0**-8 * 8
        if codes is None:
            pages = c.k_pages
            kept, pages[0, page, 1, slot, 9] = pages[0, page, 1, slot, 9].item(), math.nan
            got = c.attend_rows(q, table, lens, ints(starts), window=window, sinks=sinks)
            pages[0, page, 1, slot, 9] = kept
            assert got[0, sees.cuda(), G:].isnan().all()
            got[0, sees.cuda(), G:] = want[0, sees.cuda(), G:]
            assert torch.equal(got, want)
        assert c.status() == 0


def test_rows_leave_out_a_logit_of_minus_infinity(pk):
    """Whatever the token's value is."""
    c, table, lens, starts, q = case(pk, [500], [100], 32, 1, 2, 64, "f16")
    q = q.abs()
    at = [(0, table[0, t // 32].item(), 0, t % 32) for t in (3, 450, 540)]
    for x in at:
        c.k_pages[x] = -math.inf
    want = c.attend_rows(q, table, lens, ints(starts))
    for x in at:
        c.v_pages[x] = math.inf
    got = c.attend_rows(q, table, lens, ints(starts))
    assert torch.isfinite(want).all() and torch.isfinite(got).all() and c.status() == 0
    # probabilities rounded to f16 or not, half a step of each (2^-11) over values below 8, and two half steps of the output
    assert (got.float() - want.float()).abs().max().item() <= 3 * 2.0**-11 * 8


BIG = (1 << 31) - 1


@pytest.mark.parametrize("codes", [None, "e4m3"])
@pytest.mark.parametrize("window,sinks", [(BIG, 0), (BIG, BIG), (1, BIG), (200, BIG - 127), (BIG - 1, 5), (0, BIG)])
def test_largest_windows_and_sinks(pk, window, sinks, codes):
    """The largest that the calls take: each sees everything."""
    c, table, lens, starts, q = case(pk, [1000, 0, 129], [300, 200, 64], 32, 1, 4, 128, "bf16", codes)
    out = c.attend_rows(q, table, lens, ints(starts), window=window, sinks=sinks)
    check(c, q, table, lens, starts, 0, 0, out)
    one = q[:, [299, 499, 563]]
    check(c, one, table, lens, [0, 1, 2, 3], 0, 0, c.attend(one, table, lens, window=window, sinks=sinks))
    t = pk.PageTable(2, 40, 50, 32, window=window, sinks=sinks)
    for new in ([1000, 200], [1, 1], [40, 0]):
        t.plan(ints(new), sum(new))
    assert t.lens.tolist() == [1041, 201] and t.counts.tolist() == [40, 50]
    t.cut(ints([33, -1]))
    assert t.lens.tolist() == [33, -1] and t.counts.tolist() == [40, 88] and (t.block_table[0, :2] >= 0).all()
    assert c.status() == 0 and t.status() == 0
