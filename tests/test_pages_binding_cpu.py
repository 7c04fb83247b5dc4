"""Refusals of the paged cache's calls, in the C ABI and in the torch binding (no GPU: every one of them
comes before anything is launched)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import serving_q8_encode_gb300 as pk
    return pk


def cache(pk, L=2, P=6, H=2, page=16, d=64, dtype=torch.bfloat16, bounds=True):
    k = torch.zeros(L, P, H, page, d, dtype=dtype)
    b = torch.zeros(L, P, H, 2, d, dtype=dtype) if bounds else None
    return pk.PageCache(k, k.clone(), b)


# ------------------------------------------------------------------ the C ABI
def desc(pk, **kw):
    buf = torch.zeros(1 << 16, dtype=torch.int32)
    base = dict(n_layers=2, n_kv_heads=2, head_dim=64, page_tokens=16, n_pages=6, in_dtype=1, k_pages=buf.data_ptr(),
                v_pages=buf.data_ptr(), key_bounds=None, status=None)
    base.update(kw)
    d = pk.PagesDesc(**base)
    d._keep = buf
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(n_layers=0), 1), (dict(n_kv_heads=0), 1), (dict(n_pages=0), 1), (dict(n_pages=-4), 1), (dict(in_dtype=2), 1),
    (dict(head_dim=96), 2), (dict(page_tokens=8), 2), (dict(page_tokens=48), 2), (dict(page_tokens=256), 2),
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(k_pages=8), 1), (dict(key_bounds=24), 1), (dict(status=2), 1),
    (dict(n_pages=1 << 40), 2), (dict(n_layers=70000), 2),
])
def test_create_refuses(pk, kw, status):
    with pytest.raises(pk.PolyKVError) as e:
        pk.polykv_pages_create(desc(pk, **kw))
    assert e.value.status == status


def seqs(pk, **kw):
    base = dict(block_table=64, lens=64, max_pages=4, n_seqs=3, layer0=0, n_layers=2)
    base.update(kw)
    return pk.PagesSeqs(**base)


BAD_SEQS = [(dict(block_table=None), 1), (dict(lens=None), 1), (dict(lens=66), 1), (dict(block_table=2), 1),
            (dict(n_seqs=0), 1), (dict(max_pages=0), 1), (dict(n_seqs=4097), 2), (dict(layer0=-1), 1),
            (dict(layer0=1), 1), (dict(n_layers=0), 1), (dict(n_layers=3), 1), (dict(layer0=0x7FFFFFFF), 1),
            (dict(max_pages=1 << 32), 2), (dict(n_seqs=4096, max_pages=1 << 20), 2)]


@pytest.mark.parametrize("kw,status", BAD_SEQS)
def test_calls_refuse_bad_sequences(pk, kw, status):
    h = pk.polykv_pages_create(desc(pk, key_bounds=64))
    s, rs = seqs(pk, **kw), pk.RowStrides(512, 256, 64)
    a = pk.PagesAppendArgs(k=64, v=64, k_strides=rs, v_strides=rs, n_rows=3)
    calls = [lambda: pk.polykv_pages_append(h, s, a, None),
             lambda: pk.polykv_pages_attend(h, s, 64, rs, 4, None, -1, 0.0, 64, True, 64, 1 << 40, None),
             lambda: pk.polykv_pages_select(h, s, 64, rs, 4, 2, 0, 1, 64, 64, 1 << 40, None),
             lambda: pk.polykv_pages_select_workspace_size(h, s)]
    for call in calls:
        with pytest.raises(pk.PolyKVError) as e:
            call()
        assert e.value.status == status
    pk.polykv_pages_free(h)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=72), 1), (dict(n_rows=2), 1), (dict(n_rows=-1), 1),
    (dict(k_strides=(1, 4, 8)), 1), (dict(v_strides=(8, 8, 4)), 1), (dict(starts=66), 1), (dict(positions=68), 1),
    (dict(turns=68, rotary_dim=64), 1), (dict(turns=64, rotary_dim=0), 2), (dict(turns=64, rotary_dim=24), 2),
    (dict(turns=64, rotary_dim=80), 2), (dict(q=64, q_out=64, n_q_heads=4), 1),
    (dict(q=64, q_out=None, n_q_heads=4, turns=64, rotary_dim=64), 1),
    (dict(q=64, q_out=64, n_q_heads=3, turns=64, rotary_dim=64), 1),
    (dict(q=64, q_out=64, n_q_heads=0, turns=64, rotary_dim=64), 1),
    (dict(q=68, q_out=64, n_q_heads=4, turns=64, rotary_dim=64), 1),
    (dict(q=64, q_out=64, n_q_heads=8192, turns=64, rotary_dim=64), 2),
])
def test_append_refuses(pk, kw, status):
    h = pk.polykv_pages_create(desc(pk))
    rs = pk.RowStrides(512, 256, 64)
    base = dict(k=64, v=64, k_strides=rs, v_strides=rs, q_strides=rs, q_out_strides=rs, n_rows=3)
    base.update({k: pk.RowStrides(*v) if k.endswith("strides") else v for k, v in kw.items()})
    with pytest.raises(pk.PolyKVError) as e:
        pk.polykv_pages_append(h, seqs(pk), pk.PagesAppendArgs(**base), None)
    assert e.value.status == status
    pk.polykv_pages_free(h)


def test_a_call_of_too_many_heads_and_layers_is_refused(pk):
    h = pk.polykv_pages_create(desc(pk, n_layers=60000, n_kv_heads=1))
    with pytest.raises(pk.PolyKVError) as e:
        pk.polykv_pages_attend(h, seqs(pk, n_layers=60000), 64, pk.RowStrides(512, 256, 64), 100, None, -1, 0.0, 64, True,
                               64, 1 << 40, None)
    assert e.value.status == 2
    pk.polykv_pages_free(h)


def test_append_of_no_rows_does_nothing(pk):
    h = pk.polykv_pages_create(desc(pk))
    pk.polykv_pages_append(h, seqs(pk), pk.PagesAppendArgs(n_rows=0, starts=64), None)
    pk.polykv_pages_free(h)


def test_attend_and_select_refuse(pk):
    h = pk.polykv_pages_create(desc(pk))
    hb = pk.polykv_pages_create(desc(pk, key_bounds=64))
    rs = pk.RowStrides(512, 256, 64)

    def attend(q=64, rs=rs, hq=4, sel=None, n_sel=-1, out=64, ws=64, ws_bytes=1 << 40):
        pk.polykv_pages_attend(h, seqs(pk), q, rs, hq, sel, n_sel, 0.0, out, True, ws, ws_bytes, None)

    def select(handle=hb, q=64, rs=rs, hq=4, n=4, first=0, last=1, out=64, ws=64, ws_bytes=1 << 40, max_pages=4):
        pk.polykv_pages_select(handle, seqs(pk, max_pages=max_pages), q, rs, hq, n, first, last, out, ws, ws_bytes, None)

    for call, kw, status in [
            (attend, dict(q=None), 1), (attend, dict(q=72), 1), (attend, dict(rs=pk.RowStrides(512, 100, 64)), 1),
            (attend, dict(hq=3), 1), (attend, dict(hq=0), 1), (attend, dict(hq=8192), 2), (attend, dict(out=None), 1),
            (attend, dict(out=72), 1), (attend, dict(ws=None), 1), (attend, dict(ws=72), 1), (attend, dict(ws_bytes=100), 3),
            (attend, dict(sel=64, n_sel=0), 1), (attend, dict(sel=66, n_sel=2), 1), (attend, dict(sel=64, n_sel=(1 << 20) + 1), 1),
            (select, dict(handle=h), 6), (select, dict(q=None), 1), (select, dict(n=0), 1), (select, dict(n=-3), 1),
            (select, dict(first=-1), 1), (select, dict(last=-1), 1), (select, dict(first=3, last=2), 1),
            (select, dict(out=None), 1), (select, dict(out=66), 1), (select, dict(max_pages=50000, ws=None), 1),
            (select, dict(max_pages=50000, ws_bytes=4096 + 4 * 2 * 3 * 2 * 50000 - 1), 3)]:
        with pytest.raises(pk.PolyKVError) as e:
            call(**kw)
        assert e.value.status == status, kw
    for x in (h, hb):
        pk.polykv_pages_free(x)


@pytest.mark.parametrize("first,last", [(2**63 - 1, 1), (1, 2**63 - 1), (2**63 - 1, 2**63 - 1), (0x7FFFFFFF00001000, 2**62),
                                        (1 << 32, 0), (0, 1 << 32), (5, 0), (0, 5)])
def test_select_refuses_more_kept_pages_than_selected_ones(pk, first, last):
    """Numbers whose sum passes 64 bits, or whose low 32 bits would fit, too."""
    h = pk.polykv_pages_create(desc(pk, key_bounds=64))
    with pytest.raises(pk.PolyKVError, match="keep_first") as e:
        pk.polykv_pages_select(h, seqs(pk), 64, pk.RowStrides(512, 256, 64), 4, 4, first, last, 64, 64, 1 << 40, None)
    assert e.value.status == 1
    pk.polykv_pages_free(h)


@pytest.mark.parametrize("sel,n_sel", [(None, 0), (None, 7), (64, 0), (64, -1), (64, -(1 << 40)), (64, (1 << 20) + 1), (66, 2)])
def test_attend_refuses_a_choice_that_is_neither_all_nor_some(pk, sel, n_sel):
    """NULL with -1 is attention over all pages; an empty choice must not become that."""
    h = pk.polykv_pages_create(desc(pk))
    with pytest.raises(pk.PolyKVError, match="selected") as e:
        pk.polykv_pages_attend(h, seqs(pk), 64, pk.RowStrides(512, 256, 64), 4, sel, n_sel, 0.0, 64, True, 64, 1 << 40, None)
    assert e.value.status == 1
    pk.polykv_pages_free(h)


def test_attend_pages_refuses_a_cache_of_another_shape(pk):
    raw = torch.zeros((1 << 21) + 256, dtype=torch.uint8)
    pd = pk.PoolDesc(2, 2, 64, 128, 1)
    _, need = pk.polykv_pool_create(pd, None, 0)
    pool, _ = pk.polykv_pool_create(pd, (raw.data_ptr() + 255) // 256 * 256, need)
    pages = pk.polykv_pages_create(desc(pk))
    for n_ctx, status in ((0, 1), (1, 6)):   # nothing is encoded yet
        with pytest.raises(pk.PolyKVError) as e:
            pk.polykv_attend_pages_workspace_size(pool, pages, seqs(pk), 4, n_ctx)
        assert e.value.status == status
    with pytest.raises(pk.PolyKVError) as e:
        pk.polykv_attend_pages(pool, pages, seqs(pk), 64, 64, 3, 1, 0.0, None, -1, 64, 1 << 40, None)
    assert e.value.status == 1
    pk.polykv_pages_free(pages)
    pk.polykv_free(pool)


def test_status_needs_a_word_and_free_takes_null(pk):
    h = pk.polykv_pages_create(desc(pk))
    with pytest.raises(pk.PolyKVError) as e:
        pk.polykv_pages_status(h, None)
    assert e.value.status == 6
    pk.polykv_pages_free(h)
    pk.polykv_pages_free(None)


# ------------------------------------------------------------------ the torch binding
def test_page_cache_refuses_malformed_buffers(pk):
    k = torch.zeros(2, 6, 2, 16, 64, dtype=torch.bfloat16)
    for bad in [(k[0], k[0], None), (k.float(), k.float(), None), (k, k.half(), None), (k, k[:1], None),
                (k.transpose(1, 2), k.transpose(1, 2), None), (k, k, torch.zeros(2, 6, 2, 2, 32, dtype=k.dtype)),
                (k, k, torch.zeros(2, 6, 2, 2, 64))]:
        with pytest.raises(ValueError):
            pk.PageCache(*bad)
    with pytest.raises(pk.PolyKVError):
        pk.PageCache(k[:, :, :, :8].contiguous(), k[:, :, :, :8].contiguous())


def test_binding_refuses_malformed_tensors(pk):
    c = cache(pk)
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    rope = pk.Rope([1.0] * 32, device="cpu")
    for call in [lambda: c.attend(q.half(), t, n), lambda: c.attend(q[0], t, n), lambda: c.attend(q[..., :32], t, n),
                 lambda: c.attend(q.transpose(2, 3), t, n), lambda: c.attend(q, t.long(), n), lambda: c.attend(q, t, n.long()),
                 lambda: c.attend(q, t[:2], n), lambda: c.attend(q, t, n[:2]), lambda: c.attend(q, t[:, ::2], n),
                 lambda: c.attend(q, t, n, out=torch.zeros(2, 3, 4, 32)), lambda: c.attend(q, t, n, out_dtype=torch.float16),
                 lambda: c.attend(q, t, n, out=torch.zeros(2, 3, 4, 64), out_dtype=torch.bfloat16),
                 lambda: c.attend(q, t, n, selected=torch.zeros(2, 3, 4, 5, dtype=torch.int32)),
                 lambda: c.attend(q, t, n, selected=torch.zeros(2, 3, 2, 5)),
                 lambda: c.select(q, t, n, 4, out=torch.zeros(2, 3, 2, 4)), lambda: c.select(q[0], t, n, 4),
                 lambda: c.append(k, k.half(), t, n), lambda: c.append(k, k[:, :2], t, n),
                 lambda: c.append(k[..., ::2], k[..., ::2], t, n), lambda: c.append(k, k, t, n, starts=n),
                 lambda: c.append(k, k, t, n, positions=n), lambda: c.append(k, k, t, n, q=q[:, :2], rope=rope),
                 lambda: c.append(k, k, t, n, q_out=q, rope=rope), lambda: c.append(k, k, t, n, q=q, q_out=q[:, :, :2], rope=rope)]:
        with pytest.raises(ValueError):
            call()


class HostPool:
    """What attend_with_pages looks at before it launches anything."""

    def __init__(self, layers, head_dim, dtype=1):
        from types import SimpleNamespace
        self.handle, self.buf = 64, torch.zeros(16, dtype=torch.uint8)
        self.desc = SimpleNamespace(n_layers=layers, head_dim=head_dim, in_dtype=dtype)


def test_attend_refuses_an_empty_choice(pk):
    c, pool = cache(pk), HostPool(2, 64)
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    for sel in (torch.zeros(2, 3, 2, 5, dtype=torch.int32)[..., :0], torch.zeros(2, 3, 2, 0, dtype=torch.int32)):
        for call in (lambda: c.attend(q, t, n, selected=sel), lambda: pk.Pool.attend_with_pages(pool, q, 1, c, t, n, selected=sel)):
            with pytest.raises(ValueError, match="selected"):
                call()


@pytest.mark.parametrize("dtype,other", [(torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16)])
def test_attend_with_pages_refuses_a_q_of_another_type(pk, dtype, other):
    """The cache's type or its bits as integers: another 16-bit floating type would be read as something else."""
    c, pool = cache(pk, dtype=dtype), HostPool(2, 64, dtype=int(dtype == torch.bfloat16))
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(2, 3, 4, 64, dtype=dtype)
    for bad in (q.to(other), q.float()):
        with pytest.raises(ValueError, match="q must be"):
            pk.Pool.attend_with_pages(pool, bad, 1, c, t, n)
    for good in (q, q.view(torch.int16), q.view(torch.uint16)):
        with pytest.raises(ValueError, match="CUDA"):   # these go on to the next refusal
            pk.Pool.attend_with_pages(pool, good, 1, c, t, n)


def test_gradients_are_refused_not_dropped(pk):
    """The calls have no backward pass: a tensor that requires a gradient is refused while gradients are recorded, and
    taken under no_grad. Selection gives whole numbers, which have none."""
    c, pool = cache(pk), HostPool(2, 64)
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    rope = pk.Rope([1.0] * 32, device="cpu")
    gq, gk = q.clone().requires_grad_(), (k.clone().requires_grad_() * 2)
    calls = [lambda: c.attend(gq, t, n), lambda: c.append(gk, k, t, n), lambda: c.append(k, gk, t, n),
             lambda: c.append(k, k, t, n, q=gq, rope=rope), lambda: c.append(k, k, t, n, q=q, q_out=gq, rope=rope),
             lambda: c.attend(q, t, n, out=torch.zeros(2, 3, 4, 64, requires_grad=True)),
             lambda: pk.Pool.attend_with_pages(pool, gq, 1, c, t, n),
             lambda: pk.Pool.attend_with_pages(pool, q, 1, c, t, n, out=torch.zeros(2, 3, 4, 64, requires_grad=True))]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # goes on to the next refusal
            call()
    with pytest.raises(ValueError, match="CUDA"):
        c.select(gq, t, n, 2)
    buf = torch.zeros(2, 6, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="gradient"):
        pk.PageCache(buf, buf.clone().requires_grad_())
    with torch.no_grad():
        pk.PageCache(buf, buf.clone().requires_grad_())


def test_append_refuses_a_result_whose_rows_overlap(pk):
    c = cache(pk)
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    rope = pk.Rope([1.0] * 32, device="cpu")
    for bad in (q[:1].expand(2, 3, 4, 64), q[:, :1].expand(2, 3, 4, 64), q[:, :, :1].expand(2, 3, 4, 64),
                q.view(-1).as_strided((2, 3, 4, 64), (768, 256, 32, 1)), q.view(-1).as_strided((2, 3, 4, 64), (256, 256, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            c.append(k, k, t, n, q=q, q_out=bad, rope=rope)
    for good in (q, torch.zeros(4, 3, 2, 64, dtype=q.dtype).permute(2, 1, 0, 3), torch.zeros(2, 3, 9, 64, dtype=q.dtype)[:, :, 1::2]):
        with pytest.raises(ValueError, match="CUDA"):   # these go on to the next refusal
            c.append(k, k, t, n, q=q, q_out=good, rope=rope)


def test_binding_refuses_host_memory(pk):
    c = cache(pk)
    t, n = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    for call in [lambda: c.attend(q, t, n), lambda: c.select(q, t, n, 4), lambda: c.append(k, k, t, n), c.status]:
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rope_refuses_and_wraps(pk):
    for bad in ([], [float("nan")] * 8, [float("inf")] * 8, [1.0] * 7):
        with pytest.raises(ValueError):
            pk.Rope(bad, device="cpu")
    import math
    r = pk.Rope([2 * math.pi * x for x in (0.25, 0.5, 0.75, 1.25, -0.25, 0.0, 2.0, 1 / 3)], device="cpu")
    got = [int(x) % (1 << 64) for x in r.turns]
    want = [0.25, 0.5, 0.75, 0.25, 0.75, 0.0, 0.0, 1 / 3]
    for g, w in zip(got, want):
        assert min(abs(g - w * 2**64), 2**64 - abs(g - w * 2**64)) <= 2**64 * 2**-50
    assert pk.Rope.from_theta(64, 10000.0, device="cpu").rotary_dim == 64


@pytest.mark.parametrize("dim", [0, -16, 8, 17, 33, 40])
def test_rope_from_theta_refuses_a_width_that_it_cannot_rotate(pk, dim):
    """17 dimensions must not become 8 frequencies that rotate 16 of them."""
    with pytest.raises(ValueError, match="rotary_dim"):
        pk.Rope.from_theta(dim, device="cpu")


def test_rope_keeps_the_nearest_turns(pk):
    """f / (2 pi) modulo 1 in units of 2^-64, off by at most half a unit, for frequencies of any size and sign."""
    import random
    from fractions import Fraction
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")   # to 2^-206
    rng = random.Random(5)
    freq = [500000.0 ** (-j / 64) for j in range(64)] + [0.0, 1.0 / 3, -1.0, 1e-300, 123456.789, -2.0**40] + \
        [rng.uniform(-10, 10) * 10.0 ** rng.uniform(-12, 12) for _ in range(58)]
    for f, got in zip(freq, pk.Rope(freq, device="cpu").turns.tolist()):
        off = (Fraction(f) / two_pi * 2**64 - got) % 2**64
        assert min(off, 2**64 - off) <= Fraction(1, 2) + Fraction(1, 2**60), f
    assert len(pk.Rope([1e300] * 8, device="cpu").turns) == 8
