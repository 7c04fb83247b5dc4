"""The paged cache's kernels against plain 64-bit forms: append with rotation, attention of one new token,
page selection, all of them in a run, and together with the shared pool."""
import math
from fractions import Fraction

import numpy as np
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


def randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, dtype=torch.float32).to(dtype).cuda()


def make_table(lens, page, extra=3, width=None, seed=0):
    """(block_table on the host, number of pages): pages in random order, -1 behind each sequence's last."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(0, int(x)) // page) for x in lens]
    ids = torch.randperm(sum(need) + extra, generator=g).tolist()
    table = torch.full((len(lens), width or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    return table, sum(need) + extra


def make_cache(pk, lens, page, L, H, d, dtype, seed=0, bounds=False, poison=True, width=None):
    """A filled cache. With poison, every slot that holds no token is NaN (a recycled page's leftovers)."""
    g = torch.Generator().manual_seed(seed)
    table, P = make_table(lens, page, seed=seed, width=width)
    shape = (L, P, H, page, d)
    k, v = randn(g, *shape, dtype=dtype), randn(g, *shape, dtype=dtype)
    k *= torch.exp(0.5 * torch.randn(L, 1, H, 1, d, generator=g)).to(dtype).cuda()
    if poison:
        used = torch.zeros(P, page, dtype=torch.bool)
        for s, n in enumerate(lens):
            for t in range(max(0, int(n))):
                used[table[s, t // page], t % page] = True
        empty = ~used[None, :, None, :, None].cuda()
        k.masked_fill_(empty, math.nan)
        v.masked_fill_(empty, math.inf)
    b = torch.full((L, P, H, 2, d), math.nan, dtype=dtype, device="cuda") if bounds else None
    c = pk.PageCache(k, v, b)
    lens = torch.tensor(lens, dtype=torch.int32).cuda()
    return c, table.cuda(), lens


def tokens_of(c, table, lens, layer, s, h, chosen=None):
    """(keys, values) of one sequence and kv head in 64 bits, over all its tokens or over the chosen pages'."""
    n, page = max(0, int(lens[s])), c.page_tokens
    rows = range(n) if chosen is None else [t for p in chosen if p >= 0 for t in range(p * page, min((p + 1) * page, n))]
    rows = torch.tensor(list(rows), dtype=torch.long, device="cuda")
    ids = table[s].long()[rows // page]
    return c.k_pages[layer, ids, h, rows % page].double(), c.v_pages[layer, ids, h, rows % page].double()


def attend_ref(c, q, table, lens, layer=0, chosen=None, scale=None):
    """(out, tolerance before any output rounding), both [L][A][Hq][d] in 64 bits.

    The tolerance, per element, from the arithmetic: a logit is a sum of d exact products in fp32, off by at
    most d 2^-23 sum|q k| (each of at most d additions keeps 2^-23 of the running sum's size) and 2^-23 of
    itself for the scale; a probability carries twice that (its own and the maximum's) and 2^-22 of the
    exponential; it enters the value product off by at most 2^-22 of itself (f16: plus 2^-25, half the
    smallest step there), and the sums over n tokens keep 2^-23 per addition. All relative to sum p |v| / sum p
    (f16's floor to sum |v| / sum p), twice because the denominator has the same errors."""
    L, A, Hq, d = q.shape
    G = Hq // c.n_kv_heads
    scale = scale or 1.0 / math.sqrt(d)
    out = torch.zeros(L, A, Hq, d, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for l in range(L):
        for s in range(A):
            for h in range(c.n_kv_heads):
                k, v = tokens_of(c, table, lens, layer + l, s, h, None if chosen is None else chosen[l, s, h].tolist())
                n = k.shape[0]
                if n == 0:
                    continue
                qq = q[l, s, h * G:(h + 1) * G].double()
                x = qq @ k.T * scale
                p = torch.softmax(x, -1)
                out[l, s, h * G:(h + 1) * G] = p @ v
                dx = ((qq.abs() @ k.abs().T * scale).amax(-1) * (d * 2.0**-23) + x.abs().amax(-1) * 2.0**-23)[:, None]
                rel = 2 * dx + 2.0**-22 + 2.0**-22 + (n + 64) * 2.0**-23
                t = 2 * rel * (p @ v.abs())
                if q.dtype == torch.float16:
                    t = t + 2 * 2.0**-25 * v.abs().sum(0) * p.amax(-1, keepdim=True)
                tol[l, s, h * G:(h + 1) * G] = t
    return out, tol


def check_attend(out, ref, tol):
    t = tol + (torch.finfo(out.dtype).eps / 2 * (ref.abs() + tol) + torch.finfo(out.dtype).smallest_normal
               if out.dtype != torch.float32 else 2.0**-24 * ref.abs())
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= t).all(), f"worst {((err - t).max()).item():.3e} over, max error {err.max().item():.3e}"


# ------------------------------------------------------------------ append
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def angles(pos, inv_freq):
    """pos * inv_freq modulo 2 pi, in 64 bits of an exact product: [n][1][len(inv_freq)]."""
    turns = [round(Fraction(f) / TWO_PI * 2**160) for f in inv_freq]
    turn = [[((p * t + 2**159) % 2**160 - 2**159) / 2**160 for t in turns] for p in pos.tolist()]
    return torch.tensor(turn, dtype=torch.float64, device=pos.device)[:, None] * (2 * math.pi)


def rope_ref(x, pos, inv_freq, interleaved, mscale=1.0):
    """(rotated, tolerance) of x [L][n][heads][d] in 64 bits. Tolerance: the angle is off by at most
    2 pi 2^-25 (the turn as an fp32 number, 2^-26 and 2^-32; its 64-bit fraction, 2^-65 a position) + pi 2^-24
    (its product with 2 pi), cosine and sine by 2^-21.1 at any angle in [-pi, pi] (the function's documented bound),
    mscale, the two products and the sum by 2^-24 of themselves each, then half a step of the output type."""
    rot = 2 * len(inv_freq)
    y = x.double().clone()
    ang = angles(pos, inv_freq).to(x.device)
    cos, sin = torch.cos(ang) * mscale, torch.sin(ang) * mscale
    a, b = (x[..., 0:rot:2].double(), x[..., 1:rot:2].double()) if interleaved else \
        (x[..., :rot // 2].double(), x[..., rot // 2:rot].double())
    ra, rb = a * cos - b * sin, b * cos + a * sin
    size = (a.abs() + b.abs()) * abs(mscale)
    t = torch.zeros_like(y)
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
        t[..., 0:rot:2] = t[..., 1:rot:2] = size
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
        t[..., :rot // 2] = t[..., rot // 2:rot] = size
    pre = t * (2 * math.pi * 2.0**-25 + math.pi * 2.0**-24 + 2.0**-21.1 + 4 * 2.0**-24)
    eps = torch.finfo(x.dtype).eps
    tiny = 2.0**-25 if x.dtype == torch.float16 else 2.0**-134   # half a subnormal step
    return y, torch.where(t > 0, pre + eps / 2 * (y.abs() + pre) + tiny, 0.0)


APPENDS = [
    # page, d, H, G, dtype, old lengths, new tokens (None: one each, no starts), interleaved, rot, bounds, layers
    (16, 128, 8, 4, "bf16", [0, 5, 15, 16, 31, 700], None, False, 128, True, 1),
    (32, 64, 4, 1, "f16", [0, 1, 31, 32, 33, 64, 95], None, True, 64, True, 2),
    (64, 128, 2, 8, "bf16", [0], [1], False, 128, True, 1),
    (128, 64, 1, 7, "bf16", [0, 127, 129], [300, 0, 1], True, 32, True, 2),
    (16, 64, 3, 2, "f16", [3, 0, 16, 40], [13, 14, 16, 33], False, 32, True, 1),
    (64, 128, 2, 3, "f16", [0, 100, 63], [257, 0, 66], False, 96, False, 3),
    (128, 128, 1, 16, "bf16", [250], [130], True, 128, True, 1),
    (16, 128, 2, 2, "bf16", [7] * 40, [(5 * i) % 37 for i in range(40)], False, 16, True, 1),
]


@pytest.mark.parametrize("page,d,H,G,dtype,old,new,inter,rot,bounds,L", APPENDS)
@pytest.mark.parametrize("how", ["plain", "offset", "positions", "in_place"])
def test_append(pk, page, d, H, G, dtype, old, new, inter, rot, bounds, L, how):
    A, dt = len(old), DT[dtype]
    counts = [1] * A if new is None else new
    g = torch.Generator().manual_seed(page + d + A)
    table, P = make_table([o + n for o, n in zip(old, counts)], page, seed=A)
    layer0 = 1
    k0, v0 = randn(g, L + 2, P, H, page, d, dtype=dt), randn(g, L + 2, P, H, page, d, dtype=dt)
    b0 = randn(g, L + 2, P, H, 2, d, dtype=dt) if bounds else None
    c = pk.PageCache(k0.clone(), v0.clone(), b0.clone() if bounds else None)
    n = sum(counts)
    pad = 0 if new is None else 5                 # rows that belong to nobody
    fused = randn(g, L, n + pad, (G + 2) * H, d, dtype=dt)
    q, k, v = fused[:, :, :G * H], fused[:, :, G * H:(G + 1) * H], fused[:, :, (G + 1) * H:]
    inv = [500000.0 ** (-2 * j / rot) for j in range(rot // 2)]
    mscale = 1.25 if how == "offset" else 1.0
    rope = pk.Rope(inv, interleaved=inter, mscale=mscale)
    starts = None if new is None else torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()
    seq = torch.repeat_interleave(torch.arange(A), torch.tensor(counts))
    place = torch.cat([torch.arange(o, o + m) for o, m in zip(old, counts)])
    kw, pos = {}, place
    if how == "offset":
        kw["pos_offset"], pos = 987654321, place + 987654321
    if how == "positions":
        pos = torch.randint(-1000, 1 << 33, (n,), generator=g)
        kw["positions"] = torch.cat([pos, torch.full((pad,), 1 << 62)]).cuda()
    q_before = q.clone()
    q_out = q if how == "in_place" else torch.full((L, n + pad, G * H, d), 7.0, dtype=dt, device="cuda")
    got = c.append(k, v, table.cuda(), torch.tensor(old, dtype=torch.int32).cuda(), starts=starts, q=q, q_out=q_out,
                   rope=rope, layer=layer0, **kw)
    torch.cuda.synchronize()
    assert got is q_out and c.status() == 0

    # q
    ref, tol = rope_ref(q_before[:, :n], pos.cuda(), inv, inter, mscale)
    assert ((got[:, :n].double() - ref).abs() <= tol).all()
    assert torch.equal(got[:, n:], (q_before if how == "in_place" else torch.full_like(got, 7.0))[:, n:])
    # pages: the new slots hold the rotated keys and the values, everything else is as it was
    ref, tol = rope_ref(k[:, :n], pos.cuda(), inv, inter, mscale)
    at, slot = table[seq, place // page].long().cuda(), (place % page).cuda()
    lay = slice(layer0, layer0 + L)
    mine = c.k_pages[lay][:, at, :, slot].transpose(0, 1)
    assert ((mine.double() - ref).abs() <= tol).all()
    assert torch.equal(c.v_pages[lay][:, at, :, slot].transpose(0, 1), v[:, :n])
    for have, before in ((c.k_pages, k0), (c.v_pages, v0)):
        want = before.clone()
        want[lay][:, at, :, slot] = have[lay][:, at, :, slot]
        assert torch.equal(have, want)
    # bounds: exact over the page's tokens, others as they were
    if bounds:
        want = b0.clone()
        for s in range(A):
            for p in range(old[s] // page, -(-(old[s] + counts[s]) // page) if counts[s] else 0):
                pid, fill = int(table[s, p]), min(page, old[s] + counts[s] - p * page)
                keys = c.k_pages[lay, pid, :, :fill]
                want[lay, pid, :, 0], want[lay, pid, :, 1] = keys.amin(2), keys.amax(2)
        assert torch.equal(c.key_bounds, want)


@pytest.mark.parametrize("dtype,inter", [("f16", False), ("bf16", True)])
def test_append_at_far_positions(pk, dtype, inter):
    """Angles hold their accuracy at positions of up to 2^38, either way, whatever the frequencies."""
    n, d = 400, 128
    g = torch.Generator().manual_seed(61)
    k = randn(g, 1, n, 4, d, dtype=DT[dtype])
    pos = (2.0 ** (38 * torch.rand(n, generator=g, dtype=torch.float64))).long() * (2 * torch.randint(0, 2, (n,), generator=g) - 1)
    pos[:2] = torch.tensor([2**38, -2**38])
    inv = [500000.0 ** (-2 * j / d) for j in range(d // 2 - 2)] + [-1.0 / 3.0, 1e5 / 7.0]
    c = pk.PageCache.empty(1, 4, d, 25, 16, dtype)
    table = torch.arange(25, dtype=torch.int32).cuda()[None]
    zero, starts = torch.zeros(1, dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    q = c.append(k, k, table, zero, starts=starts, q=k, rope=pk.Rope(inv, interleaved=inter), positions=pos.cuda())
    ref, tol = rope_ref(k, pos.cuda(), inv, inter)
    assert ((q.double() - ref).abs() <= tol).all()
    assert torch.equal(c.k_pages[0].transpose(1, 2).reshape(n, 4, d), q[0])


def test_append_without_rotation_copies(pk):
    c = pk.PageCache.empty(1, 2, 64, 4, 16, "f16")
    g = torch.Generator().manual_seed(1)
    k, v = randn(g, 1, 2, 2, 64, dtype=torch.float16), randn(g, 1, 2, 2, 64, dtype=torch.float16)
    table = torch.tensor([[2, -1], [0, 3]], dtype=torch.int32).cuda()
    assert c.append(k, v, table, torch.tensor([4, 20], dtype=torch.int32).cuda()) is None
    for s, pid, slot in ((0, 2, 4), (1, 3, 4)):
        assert torch.equal(c.k_pages[0, pid, :, slot], k[0, s]) and torch.equal(c.v_pages[0, pid, :, slot], v[0, s])


def test_append_of_no_rows_returns_an_empty_q(pk):
    c = pk.PageCache.empty(2, 2, 64, 4, 16, "f16")
    table = torch.tensor([[2, -1], [0, 3]], dtype=torch.int32).cuda()
    n, starts = torch.tensor([4, 20], dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    k, q = torch.empty(2, 0, 2, 64, dtype=torch.float16).cuda(), torch.empty(2, 0, 6, 64, dtype=torch.float16).cuda()
    out = c.append(k, k, table, n, starts=starts, q=q, rope=pk.Rope.from_theta(64))
    assert out.shape == q.shape and out.dtype == q.dtype and out.device == q.device
    assert c.append(k, k, table, n, starts=starts, q=q, q_out=q, rope=pk.Rope.from_theta(64)) is q
    assert c.status() == 0


def test_append_after_a_cut_has_exact_bounds(pk):
    g = torch.Generator().manual_seed(2)
    c = pk.PageCache.empty(1, 1, 64, 2, 32, "bf16", bounds=True)
    table = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    big, small = 100 * randn(g, 1, 20, 1, 64, dtype=torch.bfloat16), randn(g, 1, 3, 1, 64, dtype=torch.bfloat16)
    lens = lambda n: torch.tensor([n], dtype=torch.int32).cuda()  # noqa: E731
    starts = lambda n: torch.tensor([0, n], dtype=torch.int32).cuda()  # noqa: E731
    c.append(small, small, table, lens(0), starts=starts(3))
    c.append(big, big, table, lens(3), starts=starts(20))
    c.append(small, small, table, lens(3), starts=starts(3))   # cut back to 3 and appended to again
    want = torch.cat([small, small], 1)[0, :, 0]
    assert torch.equal(c.key_bounds[0, 1, 0, 0], want.amin(0)) and torch.equal(c.key_bounds[0, 1, 0, 1], want.amax(0))


def test_append_skips_idle_slots_and_bad_pages(pk):
    g = torch.Generator().manual_seed(3)
    P, page = 5, 16
    for bad_id, n_bad in ((-1, 1), (P, 1), (0x7FFFFFFF, 1), (-0x80000000, 1), (4, 0)):
        c = pk.PageCache.empty(1, 2, 64, P, page, "bf16", bounds=True)
        c.k_pages.fill_(3.0), c.v_pages.fill_(4.0), c.key_bounds.fill_(5.0)
        k = randn(g, 1, 3, 2, 64, dtype=torch.bfloat16)
        rope = pk.Rope.from_theta(64)
        table = torch.tensor([[0, -1], [1, bad_id], [2, 3]], dtype=torch.int32).cuda()
        q_out = torch.full((1, 3, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        # sequence 0 is idle, sequence 1's second page is bad, sequence 2 is in order
        c.append(k, k, table, torch.tensor([-1, 20, 17], dtype=torch.int32).cuda(), q=k, q_out=q_out, rope=rope)
        torch.cuda.synchronize()
        if n_bad:
            with pytest.raises(pk.PolyKVError) as e:
                c.status()
            assert e.value.status == 6 and "page id" in str(e.value)
        assert c.status() == 0    # read and cleared
        assert torch.equal(q_out[0, 0], torch.full_like(q_out[0, 0], 9.0))
        assert torch.equal(c.v_pages[0, 3, :, 1], k[0, 2])
        touched = torch.zeros(P, page, dtype=torch.bool)
        touched[3, 1] = True
        if not n_bad:
            touched[4, 4] = True
        same = (c.v_pages == 4.0).all(-1).all(2)[0].cpu()
        assert torch.equal(~same, touched)


def test_append_leaves_the_rows_of_idle_slots(pk):
    """Runs of tokens: an idle slot's rows in the middle write nothing, and q_out keeps what it had there."""
    g = torch.Generator().manual_seed(4)
    c = pk.PageCache.empty(1, 2, 64, 4, 16, "bf16", bounds=True)
    c.k_pages.fill_(3.0), c.v_pages.fill_(4.0), c.key_bounds.fill_(5.0)
    k, q = randn(g, 1, 9, 2, 64, dtype=torch.bfloat16), randn(g, 1, 9, 4, 64, dtype=torch.bfloat16)
    table = torch.tensor([[0], [1], [2]], dtype=torch.int32).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q_out = torch.full_like(q, 9.0)
    inv = [10000.0 ** (-j / 32) for j in range(32)]
    c.append(k, k, table, i32(2, -1, 0), starts=i32(0, 3, 7, 9), q=q, q_out=q_out, rope=pk.Rope(inv))
    assert c.status() == 0
    ref, tol = rope_ref(q, torch.tensor([2, 3, 4, 0, 0, 0, 0, 0, 1]).cuda(), inv, False)
    live = [0, 1, 2, 7, 8]
    assert ((q_out.double() - ref).abs() <= tol)[:, live].all()
    assert (q_out[:, 3:7] == 9.0).all()
    assert (c.v_pages[0, 1] == 4.0).all() and (c.key_bounds[0, 1] == 5.0).all() and (c.v_pages[0, 3] == 4.0).all()
    assert torch.equal(c.v_pages[0, 0, :, 2:5], k[0, :3].transpose(0, 1)) and torch.equal(c.v_pages[0, 2, :, :2], k[0, 7:].transpose(0, 1))


def test_append_beyond_the_table_and_broken_starts_are_flagged(pk):
    c = pk.PageCache.empty(1, 1, 64, 4, 16, "bf16")
    c.v_pages.fill_(4.0)
    k = torch.ones(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    for lens, starts in ((i32(32, 1), i32(0, 2, 2)), (i32(0x7FFFFFF0, 1), i32(0, 4, 4)), (i32(0, 0), i32(0, 9, 9)),
                         (i32(0, 0), i32(-3, 2, 2)), (i32(0, 0), i32(3, 1, 7))):
        c.append(k, k, table, lens, starts=starts)
        torch.cuda.synchronize()
        with pytest.raises(pk.PolyKVError, match="length"):
            c.status()


# ------------------------------------------------------------------ attention of one new token
EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 100, 127, 128, 129, 600]
ATTENDS = [
    # page, d, H, G, dtype, lens, layers, scale
    (16, 128, 8, 4, "bf16", EDGES, 1, None),
    (32, 64, 32, 1, "f16", EDGES, 2, None),
    (64, 128, 2, 8, "f16", EDGES, 1, 0.3),
    (128, 64, 4, 8, "bf16", EDGES, 1, None),
    (16, 64, 1, 7, "bf16", [1], 1, None),
    (64, 128, 1, 16, "bf16", EDGES, 1, None),
    (32, 64, 2, 12, "f16", EDGES, 1, None),
    (16, 128, 1, 20, "f16", [0, 5, 1851], 2, None),
    (128, 64, 1, 40, "bf16", [0, 200, 33], 1, 0.5),
    (16, 128, 8, 4, "bf16", [0, 0, 0], 1, None),
    (64, 128, 2, 4, "bf16", [7194, 1, 0, 4096], 1, None),
    (16, 64, 2, 2, "f16", [13001], 1, None),
    (32, 128, 1, 1, "bf16", [(37 * i) % 90 for i in range(300)], 1, None),
]


@pytest.mark.parametrize("page,d,H,G,dtype,lens,L,scale", ATTENDS)
@pytest.mark.parametrize("out", ["f32", "in"])
def test_attend(pk, page, d, H, G, dtype, lens, L, scale, out):
    c, table, n = make_cache(pk, lens, page, L + 1, H, d, DT[dtype], seed=d + G)
    g = torch.Generator().manual_seed(5)
    wide = randn(g, L, len(lens), (G + 1) * H, d, dtype=DT[dtype])
    q = wide[:, :, H:]     # strided, as a slice of a fused projection
    got = c.attend(q, table, n, out_dtype=torch.float32 if out == "f32" else None if out is None else DT[dtype],
                   softmax_scale=scale or 0.0, layer=1)
    torch.cuda.synchronize()
    assert c.status() == 0
    ref, tol = attend_ref(c, q, table, n, layer=1, scale=scale)
    check_attend(got, ref, tol)
    empty = torch.tensor([x == 0 for x in lens])
    assert (got[:, empty] == 0).all()


def test_attend_peaked_and_huge_logits(pk):
    """One key far above the rest, and logits near a thousand: the running maximum carries them."""
    c, table, n = make_cache(pk, [500, 40], 16, 1, 2, 128, torch.bfloat16, seed=9)
    g = torch.Generator().manual_seed(6)
    q = 40 * randn(g, 1, 2, 8, 128, dtype=torch.bfloat16)
    got = c.attend(q, table, n)
    ref, tol = attend_ref(c, q, table, n)
    check_attend(got, ref, tol)


@pytest.mark.parametrize("page,d,G,dtype", [(16, 128, 4, "bf16"), (64, 64, 11, "f16")])
def test_attend_nan_reaches_its_rows(pk, page, d, G, dtype):
    """A NaN key or query makes the rows that read it NaN and no others: alone in its 16 tokens, in the last chunk, in
    one of many pieces, in the first token of all."""
    lens, at = [1, 17, 33, 80, 700, 20000, 20000], [0, 16, 32, 64, 699, 19999, 5]
    H = 2
    c, table, n = make_cache(pk, lens, page, 1, H, d, DT[dtype], seed=13)
    q = randn(torch.Generator().manual_seed(14), 1, len(lens), H * G, d, dtype=DT[dtype])
    ref, tol = attend_ref(c, q, table, n)
    nan = torch.zeros(1, len(lens), H * G, 1, dtype=torch.bool, device="cuda")
    for s, t in enumerate(at):       # kv head 0 of every sequence reads a NaN key
        c.k_pages[0, table[s, t // page].item(), 0, t % page, 3] = math.nan
    nan[:, :, :G] = True
    q[0, :, H * G - 1, d - 1] = math.nan   # and the last query head is NaN itself
    nan[:, :, H * G - 1] = True
    out = c.attend(q, table, n)
    assert (out.isnan() == nan).all()
    check_attend(out.masked_fill(nan, 0), ref.masked_fill(nan, 0), tol)


def test_attend_minus_infinite_logits_leave_tokens_out(pk):
    c, table, n = make_cache(pk, [40, 16, 17], 16, 1, 1, 64, torch.bfloat16, seed=15)
    q = randn(torch.Generator().manual_seed(16), 1, 3, 4, 64, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    kept = torch.full((1, 3, 1, 3), -1)
    kept[0, 0, 0, :2] = torch.tensor([0, 2])
    kept[0, 2, 0, 0] = 0
    ref, tol = attend_ref(c, q, table, n, chosen=kept)
    for s, p in ((0, 1), (1, 0), (2, 1)):   # one page of each sequence; it is all that sequence 1 has
        c.k_pages[0, table[s, p].item(), 0, :, 0] = -math.inf
    c.k_pages[0, table[2, 1].item(), 0, 1:, 0] = math.nan   # behind the last token
    out = c.attend(q, table, n)
    assert (out[0, 1] == 0).all()
    check_attend(out, ref, tol)


def test_attend_idle_slots_and_repeated_calls(pk):
    c, table, n = make_cache(pk, [300, 77, 5000], 32, 1, 8, 128, torch.bfloat16, seed=11)
    g = torch.Generator().manual_seed(7)
    q = randn(g, 1, 3, 32, 128, dtype=torch.bfloat16)
    n2 = n.clone()
    n2[1] = -4
    a = c.attend(q, table, n2)
    assert (a[:, 1] == 0).all()
    ref, tol = attend_ref(c, q, table, n2)
    check_attend(a, ref, tol)
    for _ in range(20):
        assert torch.equal(c.attend(q, table, n2), a)


def test_attend_bad_pages_and_lengths_are_left_out_and_flagged(pk):
    c, table, n = make_cache(pk, [100, 64, 40], 16, 1, 2, 64, torch.float16, seed=12)
    g = torch.Generator().manual_seed(8)
    q = randn(g, 1, 3, 4, 64, dtype=torch.float16)
    for wrong in (-1, c.n_pages, 0x7FFFFFFF, -0x80000000):
        t = table.clone()
        t[0, 2] = wrong
        t[2, :] = wrong          # nothing is left of sequence 2
        got = c.attend(q, t, n)
        with pytest.raises(pk.PolyKVError, match="page id"):
            c.status()
        chosen = torch.full((1, 3, 2, 8), -1)
        chosen[0, 0, :, :6] = torch.tensor([0, 1, 3, 4, 5, 6])
        chosen[0, 1, :, :4] = torch.arange(4)
        ref, tol = attend_ref(c, q, table, n, chosen=chosen)
        check_attend(got, ref, tol)
        assert (got[0, 2] == 0).all()
    n2 = n.clone()
    n2[0] = 0x7FFFFFFF           # far beyond the table: cut to it (7 pages of 16; the last 12 slots are NaN)
    c.k_pages.nan_to_num_(0.5), c.v_pages.nan_to_num_(0.5, 0.5, 0.5)
    got = c.attend(q, table, n2)
    with pytest.raises(pk.PolyKVError, match="length"):
        c.status()
    n2[0] = 112
    ref, tol = attend_ref(c, q, table, n2)
    check_attend(got, ref, tol)


def test_attend_chosen_pages(pk):
    c, table, n = make_cache(pk, [100, 16, 0, 500, 33], 16, 2, 3, 64, torch.bfloat16, seed=13)
    g = torch.Generator().manual_seed(9)
    q = randn(g, 2, 5, 6, 64, dtype=torch.bfloat16)
    K = 5
    sel = torch.full((2, 5, 3, K), -1, dtype=torch.int32)
    rng = np.random.default_rng(1)
    for l in range(2):
        for s, length in enumerate([100, 16, 0, 500, 33]):
            pages = -(-length // 16)
            for h in range(3):
                m = int(rng.integers(0, min(K, pages) + 1))
                pick = np.sort(rng.choice(pages, m, replace=False)) if pages else []
                spot = rng.choice(min(K, pages), m, replace=False) if pages else []   # -1 entries anywhere
                for i, p in zip(sorted(spot), pick):
                    sel[l, s, h, i] = int(p)
    got = c.attend(q, table, n, selected=sel.cuda())
    ref, tol = attend_ref(c, q, table, n, chosen=sel)
    check_attend(got, ref, tol)
    assert c.status() == 0
    # more entries than pages: all of them are listed
    every = torch.arange(40, dtype=torch.int32).expand(2, 5, 3, 40).clone()
    for s, length in enumerate([100, 16, 0, 500, 33]):
        every[:, s, :, -(-length // 16):] = -1
    check_attend(c.attend(q, table, n, selected=every.cuda()), *attend_ref(c, q, table, n))
    # a page twice counts twice; one beyond the sequence is flagged and left out
    twice = torch.full((2, 5, 3, 4), -1, dtype=torch.int32)
    twice[:, 3, :, :3] = torch.tensor([4, 4, 31])
    check_attend(c.attend(q, table, n, selected=twice.cuda()), *attend_ref(c, q, table, n, chosen=twice))
    assert c.status() == 0
    for wrong in (32, 0x7FFFFFFF):
        w = twice.clone()
        w[:, 3, :, 2] = wrong
        got = c.attend(q, table, n, selected=w.cuda())
        with pytest.raises(pk.PolyKVError, match="chosen page"):
            c.status()
        w[:, 3, :, 2] = -1
        check_attend(got, *attend_ref(c, q, table, n, chosen=w))


def test_offsets_beyond_32_bits(pk):
    """A cache of more than 2^32 bytes and 2^31 elements, the sequence's pages at its far end."""
    H, d, page = 8, 128, 64
    P = (1 << 31) // (H * d * page) + 40
    c = pk.PageCache.empty(1, H, d, P, page, "bf16", bounds=True)
    g = torch.Generator().manual_seed(14)
    n = 150
    table = torch.tensor([[P - 1, P - 30, P - 2]], dtype=torch.int32).cuda()
    k, v = randn(g, 1, n, H, d, dtype=torch.bfloat16), randn(g, 1, n, H, d, dtype=torch.bfloat16)
    zero, full = torch.zeros(1, dtype=torch.int32).cuda(), torch.full((1,), n, dtype=torch.int32).cuda()
    c.append(k, v, table, zero, starts=torch.tensor([0, n], dtype=torch.int32).cuda())
    rows = torch.arange(n).cuda()
    assert torch.equal(c.k_pages[0, table[0].long()[rows // page], :, rows % page], k[0])
    q = randn(g, 1, 1, 32, d, dtype=torch.bfloat16)
    ref, tol = attend_ref(c, q, table, full)
    check_attend(c.attend(q, table, full), ref, tol)
    sel = c.select(q, table, full, 2)
    check_attend(c.attend(q, table, full, selected=sel), *attend_ref(c, q, table, full, chosen=sel.cpu()))
    assert c.status() == 0


# ------------------------------------------------------------------ selection
def select_ref(c, q, table, lens, n_sel, first, last, layer=0):
    L, A, Hq, d = q.shape
    H, page = c.n_kv_heads, c.page_tokens
    G = Hq // H
    out = np.full((L, A, H, n_sel), -1, np.int32)
    qf = q.float().cpu().numpy()
    b = c.key_bounds.float().cpu().numpy()
    t = table.cpu().numpy()
    for l in range(L):
        for s in range(A):
            n = -(-max(0, int(lens[s])) // page)
            for h in range(H):
                score = np.full(n, -np.inf, np.float32)
                for g in range(G):
                    x = np.maximum(qf[l, s, h * G + g] * b[layer + l, t[s, :n], h, 0],
                                   qf[l, s, h * G + g] * b[layer + l, t[s, :n], h, 1]).reshape(n, d // 8, 8)
                    y = x[..., 0]
                    for i in range(1, 8):
                        y = y + x[..., i]
                    while y.shape[-1] > 1:
                        y = y[..., :y.shape[-1] // 2] + y[..., y.shape[-1] // 2:]
                    assert y.dtype == np.float32
                    score = np.maximum(score, y[..., 0])
                must = [p for p in range(n) if p < first or p >= n - last]
                rest = sorted(set(range(n)) - set(must), key=lambda p: (-score[p], p))
                pick = sorted((must + rest)[:n_sel])
                out[l, s, h, :len(pick)] = pick
    return torch.from_numpy(out)


def fill_bounds(c, table, lens):
    for s in range(table.shape[0]):
        n = max(0, int(lens[s]))
        for p in range(-(-n // c.page_tokens)):
            keys = c.k_pages[:, int(table[s, p]), :, :min(c.page_tokens, n - p * c.page_tokens)]
            c.key_bounds[:, int(table[s, p]), :, 0] = keys.amin(2)
            c.key_bounds[:, int(table[s, p]), :, 1] = keys.amax(2)


SELECTS = [
    # page, d, H, G, dtype, lens, n_sel, first, last, layers
    (16, 128, 8, 4, "bf16", [0, 1, 16, 17, 1000, 1851], 8, 1, 2, 1),
    (16, 64, 4, 1, "f16", [300, 1500, 64], 15, 0, 1, 2),
    (32, 64, 2, 7, "bf16", [4096, 33], 1, 0, 0, 1),
    (64, 128, 1, 16, "f16", [7194], 20, 3, 3, 1),
    (128, 128, 2, 5, "bf16", [0, 5000], 64, 1, 1, 1),
    (16, 128, 2, 2, "bf16", [1040], 64, 0, 64, 1),
]


@pytest.mark.parametrize("page,d,H,G,dtype,lens,n_sel,first,last,L", SELECTS)
def test_select(pk, page, d, H, G, dtype, lens, n_sel, first, last, L):
    c, table, n = make_cache(pk, lens, page, L + 1, H, d, DT[dtype], seed=G, bounds=True, width=-(-max(lens) // page) + 3)
    fill_bounds(c, table, n)
    g = torch.Generator().manual_seed(10)
    q = randn(g, L, len(lens), (G + 1) * H, d, dtype=DT[dtype])[:, :, H:]
    got = c.select(q, table, n, n_sel, keep_first=first, keep_last=last, layer=1)
    torch.cuda.synchronize()
    assert c.status() == 0
    assert torch.equal(got.cpu(), select_ref(c, q, table, n, n_sel, first, last, layer=1))


def test_select_ties_go_to_the_lowest_page(pk):
    c = pk.PageCache.empty(1, 1, 64, 50, 16, "bf16", bounds=True)
    c.key_bounds.fill_(1.0)
    table = torch.randperm(50, generator=torch.Generator().manual_seed(1)).int()[None].cuda()
    n = torch.tensor([50 * 16], dtype=torch.int32).cuda()
    q = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    assert c.select(q, table, n, 6, keep_last=0)[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5]
    assert c.select(q, table, n, 6, keep_last=2)[0, 0, 0].tolist() == [0, 1, 2, 3, 48, 49]
    # a zero score of either sign is one score
    q.zero_()
    c.key_bounds[0, table[0, ::2].long()] = -1.0
    assert c.select(q, table, n, 6, keep_last=0)[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5]
    # negative scores: the least negative page first
    q.fill_(-1.0)
    c.key_bounds.fill_(60.0)
    c.key_bounds[0, table[0].long(), 0] = torch.arange(1, 51, device="cuda")[:, None, None].bfloat16()
    assert c.select(q, table, n, 3, keep_last=0)[0, 0, 0].tolist() == [0, 1, 2]


@pytest.mark.parametrize("P", [20011, 50003])
def test_select_many_pages(pk, P):
    """Thousands of pages (the larger number of them goes through the workspace), and few distinct scores."""
    c = pk.PageCache.empty(1, 1, 64, P, 16, "f16", bounds=True)
    g = torch.Generator().manual_seed(15)
    for values in (None, 5):
        b = torch.randn(P, 2, 64, generator=g) if values is None else torch.randint(0, values, (P, 1, 1), generator=g).expand(P, 2, 64).float()
        c.key_bounds[0, :, 0] = b.sort(1).values.half().cuda()
        table = torch.randperm(P, generator=g).int()[None].cuda()
        n = torch.tensor([P * 16 - 3], dtype=torch.int32).cuda()
        q = randn(g, 1, 1, 2, 64, dtype=torch.float16).abs()
        for n_sel in (1, 100, 19000)[:3 if P < 30000 else 2]:
            got = c.select(q, table, n, n_sel)
            assert torch.equal(got.cpu(), select_ref(c, q, table, n, n_sel, 0, 1))


def test_select_bad_pages_score_lowest(pk):
    c, table, n = make_cache(pk, [320], 16, 1, 1, 64, torch.bfloat16, seed=3, bounds=True)
    fill_bounds(c, table, n)
    q = randn(torch.Generator().manual_seed(11), 1, 1, 2, 64, dtype=torch.bfloat16)
    t = table.clone()
    t[0, 3], t[0, 11] = c.n_pages, -1
    got = c.select(q, t, n, 18, keep_last=0)[0, 0, 0].tolist()
    assert got == [p for p in range(20) if p not in (3, 11)]
    with pytest.raises(pk.PolyKVError, match="page id"):
        c.status()


# ------------------------------------------------------------------ streams and graphs
def test_other_stream_and_caller_buffers(pk):
    c, table, n = make_cache(pk, [900, 33], 16, 1, 2, 128, torch.bfloat16, seed=21, bounds=True)
    fill_bounds(c, table, n)
    q = randn(torch.Generator().manual_seed(12), 1, 2, 8, 128, dtype=torch.bfloat16)
    want, want_sel = c.attend(q, table, n), c.select(q, table, n, 5)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ws = torch.full((pk.polykv_pages_attend_workspace_size(c.handle, 8),), 255, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0    # the arrival counts, cleared once
    out, sel = torch.full_like(want, 7.0), torch.full_like(want_sel, 7)
    torch.cuda.synchronize()
    for _ in range(3):
        c.attend(q, table, n, out=out, workspace=ws, stream=st)
    c.select(q, table, n, 5, out=sel, stream=st)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(sel, want_sel)
    assert not ws[:4096].any()    # every call leaves the counts at zero
    got, got_sel = c.attend(q, table, n, stream=st), c.select(q, table, n, 5, stream=st)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(got_sel, want_sel)
    with pytest.raises(pk.PolyKVError) as e:
        c.attend(q, table, n, workspace=ws[:-16])
    assert e.value.status == 3


def test_captured_graph_follows_lengths(pk):
    """A decode step captured once: replays append, select and attend at the lengths of their time."""
    L, H, G, d, page, A = 2, 2, 4, 64, 16, 3
    dt = torch.bfloat16
    P = 64
    g = torch.Generator().manual_seed(22)
    rope = pk.Rope.from_theta(d)

    def fresh():
        c = pk.PageCache(torch.zeros(L, P, H, page, d, dtype=dt, device="cuda"), torch.zeros(L, P, H, page, d, dtype=dt, device="cuda"),
                         torch.zeros(L, P, H, 2, d, dtype=dt, device="cuda"))
        return c, torch.tensor([0, 3, 30], dtype=torch.int32).cuda()

    table = torch.randperm(P, generator=g)[:A * 8].view(A, 8).int().cuda()
    steps = [[randn(g, L, A, n, d, dtype=dt) for n in (H, H, H * G)] for _ in range(40)]

    def step(c, lens, k, v, q):
        qr = c.append(k, v, table, lens, q=q, rope=rope)
        lens += 1
        sel = c.select(qr, table, lens, 2)
        return c.attend(qr, table, lens), c.attend(qr, table, lens, selected=sel)

    c, lens = fresh()
    want = []
    for kvq in steps:
        want.append([x.clone() for x in step(c, lens, *kvq)])
    c2, lens2 = fresh()
    buf = [x.clone() for x in steps[0]]
    step(c2, lens2, *buf)                       # warm-up
    c2.k_pages.zero_(), c2.v_pages.zero_(), c2.key_bounds.zero_()
    lens2.copy_(torch.tensor([0, 3, 30], dtype=torch.int32))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(c2, lens2, *buf)
    for kvq, w in zip(steps, want):
        for b, x in zip(buf, kvq):
            b.copy_(x)
        graph.replay()
        assert torch.equal(outs[0], w[0]) and torch.equal(outs[1], w[1])
    assert torch.equal(c2.k_pages, c.k_pages) and torch.equal(c2.key_bounds, c.key_bounds)
    assert c.status() == 0 and c2.status() == 0


# ------------------------------------------------------------------ a run of them, as a server makes it
@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("f16", True)])
def test_prompt_then_decode(pk, dtype, inter):
    """Ragged prompts, then one token at a time: attention over everything appended so far, dense and sparse,
    against the formula on the history kept in 64 bits."""
    L, H, G, d, page = 2, 2, 4, 128, 16
    dt = DT[dtype]
    prompts = [70, 5, 130]
    A, steps = len(prompts), 20
    g = torch.Generator().manual_seed(30)
    table, P = make_table([p + steps for p in prompts], page, seed=4)
    table = table.cuda()
    c = pk.PageCache(torch.full((L, P, H, page, d), math.nan, dtype=dt, device="cuda"),
                     torch.full((L, P, H, page, d), math.nan, dtype=dt, device="cuda"),
                     torch.full((L, P, H, 2, d), math.nan, dtype=dt, device="cuda"))
    inv = [10000.0 ** (-2 * j / d) for j in range(d // 2)]
    rope = pk.Rope(inv, interleaved=inter)
    lens = torch.zeros(A, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0] + list(np.cumsum(prompts)), dtype=torch.int32).cuda()
    hist = [[], []]
    k, v = (randn(g, L, sum(prompts), H, d, dtype=dt) for _ in range(2))
    c.append(k, v, table, lens, starts=starts, rope=rope)
    pos = torch.cat([torch.arange(p) for p in prompts]).cuda()
    kr = rope_ref(k, pos, inv, inter)[0]
    for s in range(A):
        a, b = int(starts[s]), int(starts[s + 1])
        hist[0].append(kr[:, a:b]), hist[1].append(v[:, a:b].double())
    lens += torch.tensor(prompts, dtype=torch.int32).cuda()
    for _ in range(steps):
        k, v = (randn(g, L, A, H, d, dtype=dt) for _ in range(2))
        q = randn(g, L, A, H * G, d, dtype=dt)
        qr = c.append(k, v, table, lens, q=q, rope=rope)
        kr = rope_ref(k, lens, inv, inter)[0]
        qr64 = rope_ref(q, lens, inv, inter)[0]
        lens += 1
        out = c.attend(qr, table, lens)
        # 4 pages hold whole sequences 0 and 1 at first, later only a part
        sel = c.select(qr, table, lens, 4, keep_first=1)
        sparse = c.attend(qr, table, lens, selected=sel)
        ref_sparse, tol_sparse = attend_ref(c, qr, table, lens, chosen=sel.cpu())
        check_attend(sparse, ref_sparse, tol_sparse)
        assert torch.equal(sel.cpu(), select_ref(c, qr, table, lens, 4, 1, 1))
        for s in range(A):
            hist[0][s] = torch.cat([hist[0][s], kr[:, s:s + 1]], 1)
            hist[1][s] = torch.cat([hist[1][s], v[:, s:s + 1].double()], 1)
            kk, vv = hist[0][s].transpose(1, 2), hist[1][s].transpose(1, 2)          # [L][H][T][d]
            qq = qr64[:, s].view(L, H, G, d)
            x = qq @ kk.mT / math.sqrt(d)
            ref = (torch.softmax(x, -1) @ vv).view(L, H * G, d)
            # q and k were rounded to the type: each logit is off by eps/2 (1 + eps) of sum|q k| for either, a
            # probability by twice that, the output by twice that of max |v|
            eps = torch.finfo(dt).eps
            dx = (qq.abs() @ kk.abs().mT / math.sqrt(d)).amax() * eps * 1.01
            assert ((out[:, s].double() - ref).abs() <= 4 * dx * vv.abs().amax() + 1e-5).all()
    assert c.status() == 0


@pytest.mark.parametrize("d,H,G,dtype,lens,n_ctx", [
    (128, 2, 4, "bf16", [0, 1, 40, 256, 17], 300),      # ten or more rows per kv head: the tensor-core pool kernel
    (128, 2, 2, "f16", [33, 0], 129),                   # few rows: the warp-level pool kernel
    (64, 4, 1, "f16", [5, 0, 100], 64),
    (64, 2, 16, "bf16", [90, 3], 100),                  # the CUDA-core pool kernel
])
def test_pool_with_private_pages(pk, d, H, G, dtype, lens, n_ctx):
    """The shared pool and ragged private pages under one softmax, against the oracle with each agent's
    tokens as its private suffix."""
    import oracle
    import synth
    L, A = 2, len(lens)
    kb, vb = synth.gen_kv(L, H, n_ctx, d, dtype, seed=2)
    qb = synth.gen_q(L, A, H * G, d, dtype, seed=2)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()  # noqa: E731
    pool = pk.Pool(L, H, d, n_ctx, dtype)
    pool.encode(dev(kb), dev(vb))
    c32, b32 = oracle.codebook.codebook_f32()
    ref_pool = oracle.attention.encode_pool(kb, vb, dtype, b32)
    c, table, n = make_cache(pk, lens, 16, L, H, d, DT[dtype], seed=5)
    q = dev(qb)
    out = pool.attend_with_pages(q, n_ctx, c, table, n)
    torch.cuda.synchronize()
    assert pool.status() == 0 and c.status() == 0
    for s in range(A):
        kw = {}
        if lens[s]:
            rows = torch.arange(lens[s]).cuda()
            ids = table[s].long()[rows // 16]
            bits = lambda x: x[:, ids, :, rows % 16].permute(1, 2, 0, 3).contiguous().view(torch.int16).cpu().numpy().view(np.uint16)[:, None]  # noqa: E731
            kw = dict(suffix_k_bits=bits(c.k_pages), suffix_v_bits=bits(c.v_pages))
        ref = oracle.attention.attend_pool(np.ascontiguousarray(qb[:, s:s + 1]), dtype, ref_pool, n_ctx, c32, **kw)
        err = np.abs(out[:, s:s + 1].cpu().numpy().astype(np.float64) - ref).max()
        assert err <= 2e-3, (s, err)     # the pool kernels' contract
    # over chosen pages
    sel = torch.zeros(L, A, H, 1, dtype=torch.int32, device="cuda")   # the first page only
    first = pool.attend_with_pages(q, n_ctx, c, table, n, selected=sel)
    cut = pool.attend_with_pages(q, n_ctx, c, table, n.clamp(max=16))
    assert (first - cut).abs().max() <= 1e-5
    # without private tokens it is the pool's own attention
    none = pool.attend_with_pages(q, n_ctx, c, table, torch.zeros_like(n))
    assert (none - pool.attend(q, n_ctx)).abs().max() <= 1e-6


def test_pool_with_private_pages_keeps_a_nan(pk):
    """A NaN among an agent's private keys, the only one it has or the last of many, is not lost beside the pool's part."""
    L, H, d, G, n_ctx, lens = 1, 2, 128, 2, 200, [1, 65, 3000]
    pool = pk.Pool(L, H, d, n_ctx, "bf16")
    g = torch.Generator().manual_seed(54)
    rows = lambda: randn(g, L, H, n_ctx, d, dtype=torch.bfloat16).view(torch.int16)  # noqa: E731
    pool.encode(rows(), rows())
    c, table, n = make_cache(pk, lens, 16, L, H, d, torch.bfloat16, seed=55)
    q = randn(g, L, len(lens), H * G, d, dtype=torch.bfloat16)
    clean = pool.attend_with_pages(q, n_ctx, c, table, n)
    for s, t in enumerate(lens):
        c.k_pages[0, table[s, (t - 1) // 16].item(), 0, (t - 1) % 16] = math.nan
    out = pool.attend_with_pages(q, n_ctx, c, table, n)
    assert out[:, :, :G].isnan().all()
    assert torch.equal(out[:, :, G:], clean[:, :, G:]) and torch.isfinite(clean).all()


def test_pool_with_private_pages_in_a_graph(pk):
    """Captured once, on two branches of one graph that may overlap; replays follow lengths and queries."""
    L, H, d, G, n_ctx, lens = 2, 2, 64, 4, 300, [100, 0, 2500]
    pool = pk.Pool(L, H, d, n_ctx, "f16")
    g = torch.Generator().manual_seed(56)
    rows = lambda: randn(g, L, H, n_ctx, d, dtype=torch.float16).view(torch.int16)  # noqa: E731
    pool.encode(rows(), rows())
    c, table, n = make_cache(pk, lens, 32, L, H, d, torch.float16, seed=57)
    qs = [[randn(g, L, len(lens), H * G, d, dtype=torch.float16) for _ in range(2)] for _ in range(5)]
    shorter = [n - 7 * i for i in range(5)]    # an idle slot from the second on, the others shrink
    want = [[pool.attend_with_pages(q, n_ctx, c, table, m) for q in two] for two, m in zip(qs, shorter)]
    buf, m, side = [q.clone() for q in qs[0]], n.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        a = pool.attend_with_pages(buf[0], n_ctx, c, table, m)
        b = pool.attend_with_pages(buf[1], n_ctx, c, table, m, stream=side)
        main.wait_stream(side)
    for two, at, w in zip(qs, shorter, want):
        buf[0].copy_(two[0]), buf[1].copy_(two[1]), m.copy_(at)
        graph.replay()
        assert torch.equal(a, w[0]) and torch.equal(b, w[1])
    assert c.status() == 0 and pool.status() == 0


def test_sequences_that_share_their_first_pages(pk):
    """Two sequences with a common prefix in the same pages, then pages of their own."""
    c, table, n = make_cache(pk, [100, 100], 16, 1, 2, 128, torch.bfloat16, seed=51, bounds=True)
    table[1, :4] = table[0, :4]
    fill_bounds(c, table, n)
    q = randn(torch.Generator().manual_seed(52), 1, 2, 8, 128, dtype=torch.bfloat16)
    check_attend(c.attend(q, table, n), *attend_ref(c, q, table, n))
    assert torch.equal(c.select(q, table, n, 3).cpu(), select_ref(c, q, table, n, 3, 0, 1))


def test_rows_of_one_tensor_for_all(pk):
    """Broadcast inputs (row stride 0) and a q that is not contiguous in its heads."""
    c = pk.PageCache.empty(2, 2, 64, 8, 16, "f16")
    g = torch.Generator().manual_seed(53)
    k1, v1 = randn(g, 1, 1, 2, 64, dtype=torch.float16), randn(g, 1, 1, 2, 64, dtype=torch.float16)
    k, v = k1.expand(2, 4, 2, 64), v1.expand(2, 4, 2, 64)
    table = torch.arange(4, dtype=torch.int32).view(4, 1).cuda()
    c.append(k, v, table, torch.full((4,), 3, dtype=torch.int32).cuda())
    assert torch.equal(c.k_pages[:, :4, :, 3], k) and torch.equal(c.v_pages[:, :4, :, 3], v)
    c.k_pages[:, :4, :, :3], c.v_pages[:, :4, :, :3] = 0.5, 0.25
    q = randn(g, 2, 4, 6, 128, dtype=torch.float16)[..., ::1][:, :, ::3, 64:]     # every third head, upper halves
    n = torch.full((4,), 4, dtype=torch.int32).cuda()
    check_attend(c.attend(q, table, n), *attend_ref(c, q, table, n))


# ------------------------------------------------------------------ calls side by side, and waits that run out
def test_two_streams_and_two_graphs_at_once(pk):
    """Calls that may overlap have workspaces of their own: eager calls per stream, captured graphs per graph."""
    c, table, n = make_cache(pk, [7194, 33, 2000], 16, 1, 2, 128, torch.bfloat16, seed=41, bounds=True)
    fill_bounds(c, table, n)
    qs = [randn(torch.Generator().manual_seed(s), 1, 3, 8, 128, dtype=torch.bfloat16) for s in (1, 2)]

    def step(q):
        sel = c.select(q, table, n, 40)
        return c.attend(q, table, n), sel, c.attend(q, table, n, selected=sel)

    want = [[x.clone() for x in step(q)] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(10):
        got = []
        for q, st in zip(qs, streams):
            with torch.cuda.stream(st):
                got.append(step(q))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    graphs, outs = [], []
    for q in qs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(q))
        graphs.append(graph)
    for _ in range(10):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert c.status() == 0


def test_other_head_counts_and_shapes_reuse_a_streams_workspace(pk):
    """Calls of different shapes in turn on one stream: the counts they share are back at zero after each."""
    g = torch.Generator().manual_seed(43)
    c, table, n = make_cache(pk, [3000, 5], 16, 1, 2, 64, torch.float16, seed=42, bounds=True)
    fill_bounds(c, table, n)
    for G in (4, 1, 16, 9, 2) * 2:
        q = randn(g, 1, 2, 2 * G, 64, dtype=torch.float16)
        check_attend(c.attend(q, table, n), *attend_ref(c, q, table, n))
        for k in (3, 100):
            assert torch.equal(c.select(q, table, n, k).cpu(), select_ref(c, q, table, n, k, 0, 1))
        one = c.select(q[:, :1].contiguous(), table[:1], n[:1], 7)
        assert torch.equal(one.cpu(), select_ref(c, q[:, :1], table[:1], n[:1], 7, 0, 1))


def test_many_sequences(pk):
    """As many sequences as one call takes, most of them idle."""
    A = 4096
    lens = [0] * A
    for s, x in ((0, 40), (1, 1), (17, 300), (4000, 65), (4095, 129)):
        lens[s] = x
    c, table, n = make_cache(pk, lens, 16, 1, 1, 64, torch.bfloat16, seed=44, bounds=True)
    fill_bounds(c, table, n)
    q = randn(torch.Generator().manual_seed(45), 1, A, 12, 64, dtype=torch.bfloat16)
    ref, tol = attend_ref(c, q, table, n)
    check_attend(c.attend(q, table, n), ref, tol)
    got = c.select(q, table, n, 3).cpu()
    live = [s for s in range(A) if lens[s]]
    assert torch.equal(got[:, live], select_ref(c, q[:, live], table[live], n[live], 3, 0, 1))
    got[:, live] = -1
    assert (got == -1).all()
    # appends: the last rows of the batch belong to the last sequence
    k = randn(torch.Generator().manual_seed(46), 1, 3, 1, 64, dtype=torch.bfloat16)
    starts = torch.zeros(A + 1, dtype=torch.int32)
    starts[18:] = 1
    starts[4096] = 3
    before = n.clone()
    c.append(k, k, table, n, starts=starts.cuda())
    assert torch.equal(c.v_pages[0, table[17, 300 // 16].long(), 0, 300 % 16], k[0, 0, 0])
    assert torch.equal(c.v_pages[0, table[4095, 8].long(), 0, 1:3], k[0, 1:, 0]) and torch.equal(n, before)
    assert c.status() == 0


def test_stalled_wait_times_out_and_context_survives(pk):
    """The producer is told to copy nothing: the consumers' bounded waits give up, the status says so, and the next
    call is right."""
    import os
    c, table, n = make_cache(pk, [100, 7], 16, 1, 2, 128, torch.bfloat16, seed=47)
    q = randn(torch.Generator().manual_seed(48), 1, 2, 8, 128, dtype=torch.bfloat16)
    os.environ["POLYKV_TEST_STALL"] = "1"
    try:
        c.attend(q, table, n)
        torch.cuda.synchronize()
    finally:
        del os.environ["POLYKV_TEST_STALL"]
    with pytest.raises(pk.PolyKVError) as e:
        c.status()
    assert e.value.status == 5
    assert c.status() == 0
    check_attend(c.attend(q, table, n), *attend_ref(c, q, table, n))
    assert c.status() == 0


# ------------------------------------------------------------------ small probabilities
def sink_case(pk, dtype, d, H, G, lens, at, nats, page=16):
    """One token per sequence with a logit `nats` above the others', whose logits scatter by about 0.1, and a value
    of zero: the result is what the others leave. (cache, table, lens, q)"""
    dt = DT[dtype]
    c, table, n = make_cache(pk, lens, page, 1, H, d, dt, seed=d + G + len(lens))
    g = torch.Generator().manual_seed(71)
    c.k_pages.copy_(0.1 * randn(g, *c.k_pages.shape, dtype=dt))
    c.v_pages.copy_(1 + 0.25 * randn(g, *c.v_pages.shape, dtype=dt))
    for s, length in enumerate(lens):
        t = {"first": 0, "last": length - 1, "middle": length // 2}[at]
        c.k_pages[0, int(table[s, t // page]), :, t % page] = nats / math.sqrt(d)
        c.v_pages[0, int(table[s, t // page]), :, t % page] = 0.0
    return c, table, n, torch.ones(1, len(lens), H * G, d, dtype=dt, device="cuda")


def sink_tolerance(c, q, table, lens):
    """Per element, in fp32 relative to sum p |v| / sum p whatever the size of p. A logit is off by d 2^-23 sum|q k| and
    2^-23 of itself, a probability by twice that (its own and the maximum's) and 2^-22 of the exponential; in the value
    product its two or three parts leave at most 2^-22 of it. A row's running sums take at most n / 16 steps (one
    16-token product each) and 64 additions within a step and over warps and pieces, 2^-23 each. Twice, for
    numerator and denominator; the sink's own probability is in the denominator only."""
    ref, _ = attend_ref(c, q, table, lens)
    tol = torch.zeros_like(ref)
    G = q.shape[2] // c.n_kv_heads
    for s in range(q.shape[1]):
        for h in range(c.n_kv_heads):
            k, v = tokens_of(c, table, lens, 0, s, h)
            qq = q[0, s, h * G:(h + 1) * G].double()
            x = qq @ k.T / math.sqrt(q.shape[3])
            dx = (qq.abs() @ k.abs().T / math.sqrt(q.shape[3])).amax(-1) * (q.shape[3] * 2.0**-23) + x.abs().amax(-1) * 2.0**-23
            rel = 2 * (2 * dx[:, None] + 2.0**-22 + 2.0**-22 + (k.shape[0] / 16 + 64) * 2.0**-23)
            tol[0, s, h * G:(h + 1) * G] = rel * (torch.softmax(x, -1) @ v.abs())
    return ref, tol


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nats", [12.0, 17.25, 20.0, 30.0, 60.0])
@pytest.mark.parametrize("d,H,G,at", [(128, 2, 4, "first"), (64, 4, 1, "last"), (64, 1, 11, "middle"), (128, 1, 16, "last")])
def test_attend_keeps_small_probabilities(pk, dtype, nats, d, H, G, at):
    """Many tokens far below one whose value is zero: their probabilities keep fp32's accuracy, as in a short unit of one
    warp, in one of several chunks, and in one cut over many CTAs."""
    c, table, n, q = sink_case(pk, dtype, d, H, G, [2, 16, 33, 100, 700, 9001], at, nats)
    ref, tol = sink_tolerance(c, q, table, n)
    check_attend(c.attend(q, table, n), ref, tol)
    every = torch.arange(table.shape[1], dtype=torch.int32, device="cuda").expand(1, len(n), H, -1).contiguous()
    check_attend(c.attend(q, table, n, selected=every), ref, tol)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_keeps_small_probabilities_of_a_long_context(pk, dtype):
    c, table, n, q = sink_case(pk, dtype, 64, 1, 2, [131072], "first", 18.0, page=64)
    check_attend(c.attend(q, table, n), *sink_tolerance(c, q, table, n))


# ------------------------------------------------------------------ host threads, and the status word
@pytest.mark.parametrize("call", ["select", "attend"])
def test_host_threads_with_calls_of_different_sizes(pk, call):
    """Calls whose kernels take different amounts of shared memory, from several host threads at once."""
    import threading
    L, H, d, A = 1, 4, 64, 20
    c = pk.PageCache.empty(L, H, d, 4, 16, "bf16", bounds=True)
    errors = []

    def work(n_seqs, max_pages):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                table = torch.zeros(n_seqs, max_pages, dtype=torch.int32, device="cuda")
                lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
                q = torch.zeros(L, n_seqs, H, d, dtype=torch.bfloat16, device="cuda")
                seqs = pk.PagesSeqs(table.data_ptr(), lens.data_ptr(), max_pages, n_seqs, 0, L)
                need = pk.polykv_pages_attend_workspace_size(c.handle, H) if call == "attend" else \
                    pk.polykv_pages_select_workspace_size(c.handle, seqs)
                ws = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
                out = torch.full((L, n_seqs, H, 64), 7.0, dtype=torch.float32, device="cuda")
                rs = pk.RowStrides(n_seqs * H * d, H * d, d)
                for _ in range(3000):
                    if call == "attend":
                        pk.polykv_pages_attend(c.handle, seqs, q.data_ptr(), rs, H, None, -1, 0.0, out.data_ptr(), True,
                                               ws.data_ptr(), ws.numel(), st.cuda_stream)
                    else:
                        pk.polykv_pages_select(c.handle, seqs, q.data_ptr(), rs, H, 8, 0, 1, out.data_ptr(), ws.data_ptr(),
                                               ws.numel(), st.cuda_stream)
                st.synchronize()
                want = out.view(torch.int32).flatten()[:n_seqs * H * 8] + 1 if call == "select" else out
                if want.any():
                    raise AssertionError("wrong results")
        except Exception as e:
            errors.append(repr(e))

    sizes = [(A, 32768), (A, 4)] if call == "select" else [(1, 4), (4096, 4)]
    threads = [threading.Thread(target=work, args=s) for s in sizes * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert c.status() == 0


def test_status_loses_no_bit_set_by_another_stream(pk):
    """A bad page met on one stream while status() reads and clears on another is reported by that call or a later one."""
    c = pk.PageCache.empty(1, 1, 64, 2, 16, "bf16")
    k = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    table, zero = torch.full((1, 1), 7, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def flagged():
        try:
            return c.status(stream=a) != 0
        except pk.PolyKVError:
            return True

    for i in range(300):
        with torch.cuda.stream(b):
            torch.cuda._sleep(20000 + 700 * i)
            c.append(k, k, table, zero)
            done = torch.cuda.Event()
            done.record(b)
        seen = False
        while not done.query():
            seen |= flagged()
        b.synchronize()
        assert flagged() or seen, i
    assert c.status() == 0


# ------------------------------------------------------------------ values at the ends of f16, and calls without gradients
@pytest.mark.parametrize("d,G", [(64, 1), (128, 12)])
@pytest.mark.parametrize("value", ["largest", "subnormal"])
def test_attend_f16_values_at_the_ends_of_the_type(pk, d, G, value):
    """f16's largest values stay finite in fp32 output and its smallest ones keep their bits."""
    c, table, n = make_cache(pk, [1, 40, 700, 5000], 16, 1, 2, d, torch.float16, seed=81)
    g = torch.Generator().manual_seed(82)
    steps = torch.randint(1, 1024, c.v_pages.shape, generator=g).cuda()
    v = steps.double() * 2.0**-24 if value == "subnormal" else 65504.0 - 32.0 * (steps % 7).double()
    c.v_pages.copy_(torch.where(torch.rand(c.v_pages.shape, generator=g).cuda() < 0.5, v, -v).half())
    q = randn(g, 1, 4, 2 * G, d, dtype=torch.float16)
    check_attend(c.attend(q, table, n), *attend_ref(c, q.double(), table, n))   # the tolerance of fp32 probabilities


def test_calls_under_no_grad_take_tensors_that_require_one(pk):
    c, table, n = make_cache(pk, [100, 40], 16, 1, 2, 64, torch.bfloat16, seed=83)
    q = randn(torch.Generator().manual_seed(84), 1, 2, 8, 64, dtype=torch.bfloat16)
    want, leaf = c.attend(q, table, n), q.clone().requires_grad_()
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            got = c.attend(leaf, table, n)
        assert torch.equal(got, want) and not got.requires_grad
    with pytest.raises(ValueError, match="gradient"):
        c.attend(leaf, table, n)


@pytest.mark.parametrize("d,H,G,dtype,lens,n_ctx", [(128, 2, 4, "bf16", [70, 0, 333], 300), (64, 4, 1, "f16", [16, 500], 129)])
def test_pool_with_chosen_private_pages(pk, d, H, G, dtype, lens, n_ctx):
    """The pool and some of each agent's pages, another choice per layer and kv head, against the oracle with their tokens as
    the private suffix."""
    import oracle
    import synth
    L, A, page, K = 2, len(lens), 16, 4
    kb, vb = synth.gen_kv(L, H, n_ctx, d, dtype, seed=3)
    qb = synth.gen_q(L, A, H * G, d, dtype, seed=3)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).cuda()  # noqa: E731
    pool = pk.Pool(L, H, d, n_ctx, dtype)
    pool.encode(dev(kb), dev(vb))
    c32, b32 = oracle.codebook.codebook_f32()
    c, table, n = make_cache(pk, lens, page, L, H, d, DT[dtype], seed=85)
    rng = np.random.default_rng(86)
    sel = np.full((L, A, H, K), -1, np.int32)
    for l in range(L):
        for s, length in enumerate(lens):
            pages = -(-length // page)
            for h in range(H):
                pick = np.sort(rng.choice(pages, min(K - 1, pages), replace=False)) if pages else []
                sel[l, s, h, :len(pick)] = pick
    out = pool.attend_with_pages(dev(qb), n_ctx, c, table, n, selected=torch.from_numpy(sel).cuda())
    assert pool.status() == 0 and c.status() == 0
    bits = lambda x: x.half().view(torch.int16) if dtype == "f16" else x.bfloat16().view(torch.int16)  # noqa: E731
    for l in range(L):
        for s in range(A):
            for h in range(H):
                one = oracle.attention.encode_pool(kb[l:l + 1, h:h + 1], vb[l:l + 1, h:h + 1], dtype, b32)
                k, v = (bits(x).cpu().numpy().view(np.uint16)[None, None, None] for x in
                        tokens_of(c, table, n, l, s, h, chosen=sel[l, s, h].tolist()))
                kw = dict(suffix_k_bits=k, suffix_v_bits=v) if k.shape[3] else {}
                ref = oracle.attention.attend_pool(np.ascontiguousarray(qb[l:l + 1, s:s + 1, h * G:(h + 1) * G]), dtype, one, n_ctx, c32, **kw)
                err = np.abs(out[l, s, h * G:(h + 1) * G].cpu().numpy().astype(np.float64) - ref[0, 0]).max()
                assert err <= 2e-3, (l, s, h, err)     # the pool kernels' contract
