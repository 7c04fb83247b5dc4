"""Window arithmetic of the paged cache compiled for the host, and the refusals of the calls over windows, rows, codes and
block tables (no GPU: every one of them comes before anything is launched)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "serving_q8_encode_gb300", "csrc")
SHIM = r"""
#include "pages_index.cuh"
using namespace polykv;
extern "C" {
uint32_t t_steps(int64_t len, int page, int window, int sinks) { return window_steps(len, page, window_of(len, page, window, sinks)); }
int64_t t_page(uint32_t step, int64_t len, int page, int window, int sinks, int* slot, uint32_t* mask) {
    return window_page(step, page, window_of(len, page, window, sinks), len, slot, mask);
}
}
"""


@pytest.fixture(scope="module")
def ix(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("window_index")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run([cxx, "-shared", "-fPIC", "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    so = ctypes.CDLL(str(lib))
    so.t_steps.restype = ctypes.c_uint32
    so.t_steps.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    so.t_page.restype = ctypes.c_int64
    so.t_page.argtypes = [ctypes.c_uint32, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                          ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_uint32)]
    return so


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_a_windows_steps_cover_what_it_sees_once(ix, page):
    rng = random.Random(page)
    cases = [(0, 5, 5), (1, 1, 0), (16, 16, 16), (1000, 0, 700), (1000, 1, 0), (1000, 999, 0), (1000, 1000, 3), (1000, 5, 2000)]
    cases += [(rng.randint(0, 1500), rng.choice([0, rng.randint(1, 1600)]), rng.choice([0, rng.randint(0, 300)])) for _ in range(300)]
    for length, window, sinks in cases:
        want = [t for t in range(length) if not window or t >= length - window or t < sinks]
        seen, pages = [], []
        for s in range(ix.t_steps(length, page, window, sinks)):
            slot, mask = ctypes.c_int(), ctypes.c_uint32()
            lp = ix.t_page(s, length, page, window, sinks, slot, mask)
            assert 0 <= lp < -(-length // page) and slot.value % 16 == 0 and slot.value + 16 <= page and mask.value <= 0xFFFF
            seen += [lp * page + slot.value + i for i in range(16) if mask.value >> i & 1]
            pages.append(lp)
        assert seen == want, (length, window, sinks)
        # no page but those that hold something to see
        assert set(pages) == {t // page for t in want}


def test_a_window_of_a_sequence_near_two_to_the_31(ix):
    length, page, window, sinks = (1 << 31) - 200, 128, 1000, 5
    n = ix.t_steps(length, page, window, sinks)
    assert n * 16 <= 128 + 1000 + 2 * 128
    slot, mask = ctypes.c_int(), ctypes.c_uint32()
    assert ix.t_page(0, length, page, window, sinks, slot, mask) == 0 and mask.value == 0b11111
    lp = ix.t_page(n - 1, length, page, window, sinks, slot, mask)
    assert lp * page + slot.value + mask.value.bit_length() == length
    assert ix.t_steps(length, page, (1 << 31) - 1, (1 << 31) - 1) == (length + 15) // 16


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def pk():
    import __graft_entry__
    __graft_entry__.build()
    import serving_q8_encode_gb300 as pk
    return pk


def cache(pk, L=2, P=6, H=2, page=16, d=64, dtype=torch.bfloat16, codes=None):
    if codes is None:
        k = torch.zeros(L, P, H, page, d, dtype=dtype)
        return pk.PageCache(k, k.clone())
    k = torch.zeros(L, P, H, page, d, dtype=codes)
    return pk.PageCache(k, k.clone(), scales=torch.ones(L, P, H, 2), row_dtype=dtype)


def desc(pk, **kw):
    buf = torch.zeros(1 << 16, dtype=torch.int32)
    base = dict(n_layers=2, n_kv_heads=2, head_dim=64, page_tokens=16, n_pages=6, in_dtype=1, k_pages=buf.data_ptr(),
                v_pages=buf.data_ptr(), key_bounds=None, status=None)
    base.update(kw)
    d = pk.PagesDesc(**base)
    d._keep = buf
    return d


@pytest.mark.parametrize("kw,code,scales,status", [
    (dict(), 0, 64, 1), (dict(), 3, 64, 1), (dict(), 1, None, 1), (dict(), 2, 68, 1), (dict(key_bounds=32), 1, 64, 2),
    (dict(head_dim=96), 1, 64, 2), (dict(page_tokens=8), 2, 64, 2), (dict(k_pages=8), 1, 64, 1), (dict(n_pages=0), 1, 64, 1),
])
def test_create_coded_refuses(pk, kw, code, scales, status):
    with pytest.raises(pk.PolyKVError) as e:
        pk.polykv_pages_create_coded(desc(pk, **kw), code, scales)
    assert e.value.status == status


def test_c_calls_refuse(pk):
    h = pk.polykv_pages_create(desc(pk))
    s = pk.PagesSeqs(block_table=64, lens=64, max_pages=4, n_seqs=3, layer0=0, n_layers=2)
    st = pk.RowStrides(512, 128, 64)

    def refused(status, f, *a):
        with pytest.raises(pk.PolyKVError) as e:
            f(*a)
        assert e.value.status == status, e.value

    big = 1 << 31
    for window, sinks in ((-1, 0), (0, -1), (big, 0), (5, big)):
        refused(1, pk.polykv_pages_attend_window, h, s, 64, st, 4, window, sinks, 0.0, 64, 1, 64, 1 << 30, None)
        refused(1, pk.polykv_pages_attend_rows, h, s, 64, st, 4, 9, 64, window, sinks, 0.0, 64, 64, 1 << 30, None)
        refused(1, pk.polykv_pages_attend_rows_workspace_size, h, s, 4, 9, window, sinks)
    refused(3, pk.polykv_pages_attend_window, h, s, 64, st, 4, 5, 1, 0.0, 64, 1, 64, 8, None)
    for args in ((64, st, 4, -1, 64), (64, st, 4, big, 64), (64, st, 4, 9, None), (64, st, 4, 9, 66), (None, st, 4, 9, 64),
                 (72, st, 4, 9, 64), (64, pk.RowStrides(512, 100, 64), 4, 9, 64), (64, st, 3, 9, 64)):
        refused(1, pk.polykv_pages_attend_rows, h, s, *args, 0, 0, 0.0, 64, 64, 1 << 30, None)
    refused(1, pk.polykv_pages_attend_rows, h, s, 64, st, 4, 9, 64, 0, 0, 0.0, None, 64, 1 << 30, None)
    refused(1, pk.polykv_pages_attend_rows, h, s, 64, st, 4, 9, 64, 0, 0, 0.0, 72, 64, 1 << 30, None)
    pk.polykv_pages_attend_rows(h, s, 64, st, 4, 0, 64, 0, 0, 0.0, None, None, 0, None)     # no rows: nothing to do
    for args in ((-1, 64, 64, 64), (9, None, 64, 64), (9, 66, 64, 64), (9, 64, None, 64), (9, 64, 64, 72)):
        refused(1, pk.polykv_pages_gather, h, s, *args, None)
    pk.polykv_pages_gather(h, s, 0, 64, None, None, None)
    refused(1, pk.polykv_pages_gather, h, pk.PagesSeqs(64, 64, 4, 3, 1, 2), 9, 64, 64, 64, None)
    pk.polykv_pages_free(h)


def tables(pk, **kw):
    base = dict(block_table=64, lens=64, first=64, ring=64, counts=64, arrivals=64, status=None, max_pages=4, n_pages=9, window=0,
                sinks=0, n_seqs=3, page_tokens=16)
    base.update(kw)
    return pk.PageTables(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(block_table=None), 1), (dict(lens=None), 1), (dict(first=None), 1), (dict(ring=None), 1), (dict(counts=None), 1),
    (dict(arrivals=None), 1), (dict(counts=68), 1), (dict(ring=66), 1), (dict(status=2), 1), (dict(n_seqs=0), 1),
    (dict(max_pages=0), 1), (dict(n_pages=0), 1), (dict(n_seqs=4097), 2), (dict(n_pages=1 << 31), 2), (dict(page_tokens=48), 2),
    (dict(max_pages=1 << 28), 2), (dict(n_seqs=4096, max_pages=1 << 20), 2), (dict(window=-1), 1), (dict(sinks=1 << 31), 1),
])
def test_tables_refuse(pk, kw, status):
    for f, args in ((pk.polykv_tables_plan, (64, 9, 64, 64, 64, 64, 64, None)), (pk.polykv_tables_cut, (64, None))):
        with pytest.raises(pk.PolyKVError) as e:
            f(tables(pk, **kw), *args)
        assert e.value.status == status
    with pytest.raises(pk.PolyKVError):
        pk.polykv_tables_status(tables(pk, **kw), None)


def test_plan_and_cut_refuse(pk):
    for args in ((None, 9, 64, 64, 64, 64, 64), (64, -1, 64, 64, 64, 64, 64), (64, 1 << 31, 64, 64, 64, 64, 64),
                 (64, 9, None, 64, 64, 64, 64), (64, 9, 64, None, 64, 64, 64), (64, 9, 64, 64, 66, 64, 64),
                 (64, 9, 64, 64, 64, 68, 64), (64, 9, 64, 64, 64, 64, 4)):
        with pytest.raises(pk.PolyKVError) as e:
            pk.polykv_tables_plan(tables(pk), *args, None)
        assert e.value.status == 1
    for keep in (None, 66):
        with pytest.raises(pk.PolyKVError):
            pk.polykv_tables_cut(tables(pk), keep, None)
    with pytest.raises(pk.PolyKVError) as e:
        pk.polykv_tables_status(tables(pk), None)
    assert e.value.status == 6     # no status word


def test_structs_match_the_header(pk):
    hdr = open(os.path.join(ROOT, "include", "polykv.h")).read()
    body = hdr[:hdr.index("} polykv_page_tables;")]
    body = body[body.rindex("typedef struct {"):]
    names = []
    for line in body.splitlines()[1:]:
        line = line.split("/*")[0].strip()
        if line.endswith(";"):
            kind, rest = line[:-1].split(None, 1)
            names += [(x.strip(" *"), kind + ("*" if "*" in kind + x else "")) for x in rest.split(",")]
    assert [n for n, _ in names] == [f[0] for f in pk.PageTables._fields_]
    size = {"int32_t": 4, "int64_t": 8}
    for (n, kind), (_, t) in zip(names, pk.PageTables._fields_):
        assert ctypes.sizeof(t) == (8 if "*" in kind else size[kind]), n


def test_cache_of_codes_refuses(pk):
    k = torch.zeros(2, 6, 2, 16, 64, dtype=torch.int8)
    s = torch.ones(2, 6, 2, 2)
    bf = torch.bfloat16
    for kw in (dict(scales=s), dict(scales=s, row_dtype=torch.float32), dict(row_dtype=bf), dict(scales=s[:, :5], row_dtype=bf),
               dict(scales=s.double(), row_dtype=bf), dict(scales=s.transpose(0, 2), row_dtype=bf),
               dict(scales=s, row_dtype=bf, key_bounds=torch.zeros(2, 6, 2, 2, 64, dtype=bf)),
               dict(scales=torch.ones(2, 6, 2, 2, requires_grad=True), row_dtype=bf)):
        with pytest.raises(ValueError):
            pk.PageCache(k, k.clone(), **kw)
    with pytest.raises(ValueError):
        pk.PageCache(k, k.view(torch.float8_e4m3fn), scales=s, row_dtype=bf)
    with pytest.raises(ValueError):
        pk.PageCache(k.view(torch.uint8), k.view(torch.uint8), scales=s, row_dtype=bf)
    wide = torch.zeros(2, 6, 2, 16, 64, dtype=bf)
    for kw in (dict(scales=s), dict(row_dtype=torch.float16)):
        with pytest.raises(ValueError):
            pk.PageCache(wide, wide.clone(), **kw)
    for kw in (dict(codes="fp8"), dict(codes="int8", bounds=True)):
        with pytest.raises(ValueError):
            pk.PageCache.empty(1, 2, 64, 4, 16, device="cpu", **kw)
    c = pk.PageCache.empty(1, 2, 64, 4, 16, dtype="f16", device="cpu", codes="e4m3")
    assert c.dtype == torch.float16 and c.k_pages.dtype == torch.float8_e4m3fn
    q = torch.zeros(1, 3, 4, 64, dtype=torch.float16)
    t, n = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: c.attend(q, t, n), lambda: c.attend_rows(q, t, n, torch.zeros(4, dtype=torch.int32)),
                 lambda: c.gather(t, n, torch.zeros(4, dtype=torch.int32), 3), lambda: c.append(q[:, :, :2], q[:, :, :2], t, n)):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            call()
    with pytest.raises(ValueError, match="dtype|must be"):
        c.attend(q.bfloat16(), t, n)


def test_bound_calls_refuse(pk):
    c = cache(pk)
    q = torch.zeros(2, 5, 4, 64, dtype=torch.bfloat16)
    t, n, s = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    sel = torch.zeros(2, 3, 2, 1, dtype=torch.int32)
    for call in (lambda: c.attend(q[:, :3], t, n, selected=sel, window=5), lambda: c.attend(q[:, :3], t, n, selected=sel, sinks=5),
                 lambda: c.attend_rows(q, t, n, s[:3]), lambda: c.attend_rows(q, t, n, s.long()),
                 lambda: c.attend_rows(q.float(), t, n, s), lambda: c.attend_rows(q[0], t, n, s),
                 lambda: c.attend_rows(q[..., :32], t, n, s), lambda: c.attend_rows(q, t[0], n, s),
                 lambda: c.attend_rows(q, t, n, s, out=q.float()), lambda: c.attend_rows(q, t, n, s, out=q[:, :4]),
                 lambda: c.attend_rows(q.clone().requires_grad_(), t, n, s), lambda: c.attend_rows(q, t, n, s, layer=1 << 40),
                 lambda: c.gather(t, n, s, -1), lambda: c.gather(t, n, s, 1 << 31), lambda: c.gather(t, n, s[:2], 5),
                 lambda: c.gather(t, n, s, 5, k=q), lambda: c.gather(t, n, s, 5, n_layers=1 << 40)):
        with pytest.raises(ValueError):
            call()


def test_page_table_refuses(pk):
    for a in ((0, 4, 9), (3, 0, 9), (3, 4, 0), (3, 4, 9, 48), (3, 4, 9, 16, -1), (3, 4, 9, 16, 0, 1 << 31)):
        with pytest.raises(ValueError):
            pk.PageTable(*a, device="cpu")
    t = pk.PageTable(3, 4, 9, 16, sinks=17, device="cpu")
    assert t.first.tolist() == [2] * 3 and t.counts.tolist() == [0, 9] and (t.block_table == -1).all()
    new = torch.ones(3, dtype=torch.int32)
    for call in (lambda: t.plan(new, 3), lambda: t.cut(new), lambda: t.status()):
        with pytest.raises(ValueError, match="the tables are on cpu, not on a CUDA device"):
            call()
    for call in (lambda: t.plan(new[:2], 3), lambda: t.plan(new.long(), 3), lambda: t.plan(new, -1), lambda: t.plan(new, 1 << 31),
                 lambda: t.cut(new[:2]), lambda: t.cut(new.float()), lambda: t.plan([1, 1, 1], 3)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        t.restore(t.block_table, t.lens, t.first, t.ring[:4], t.counts)
    t.restore(t.block_table + 1, t.lens, t.first, t.ring, t.counts)
    assert (t.block_table == 0).all()


def test_rows_refuse_a_result_over_their_queries(pk):
    """A row that is not finite is computed again from its query, which a result in its place would have replaced."""
    c = cache(pk)
    t, n, s = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    buf = torch.zeros(2 * 5 * 4 * 64 * 2, dtype=torch.bfloat16)
    q = buf[:2560].view(2, 5, 4, 64)
    for out in (q, buf[8:2568].view(2, 5, 4, 64), buf[2552:5112].view(2, 5, 4, 64)):
        with pytest.raises(ValueError, match="out overlaps q"):
            c.attend_rows(q, t, n, s, out=out)
    wide = buf.view(2, 5, 8, 64)
    with pytest.raises(ValueError, match="out overlaps q"):
        c.attend_rows(wide[:, :, 4:], t, n, s, out=q)
    with pytest.raises(ValueError, match="not on a CUDA device"):      # side by side: all checks passed
        c.attend_rows(q, t, n, s, out=buf[2560:].view(2, 5, 4, 64))
