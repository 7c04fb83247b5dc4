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
