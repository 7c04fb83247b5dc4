"""The paged cache's index arithmetic (csrc/pages_index.cuh), compiled for the host: the append's work
items, attention's steps, the shares of the work list, and what happens to page ids, lengths, starts and
choices that are wrong. Nothing here needs a GPU."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "serving_q8_encode_gb300", "csrc")

SHIM = r"""
#include "pages_index.cuh"
using namespace polykv;
extern "C" {
int64_t t_clamp_len(int64_t len, int64_t max_pages, int page, uint32_t* bad) { return clamp_len(len, max_pages, page, bad); }
uint32_t t_seq_steps(int64_t len, int page, int n_sel) { return seq_steps(len, page, n_sel); }
int64_t t_step_page(uint32_t step, int page, int n_sel, int64_t chosen, int64_t len, int* slot, int* valid, uint32_t* bad) {
    return step_page(step, page, n_sel, chosen, len, slot, valid, bad);
}
int64_t t_check_page(int64_t id, int64_t n, uint32_t* bad) { return check_page(id, n, bad); }
int64_t t_item_base(int64_t start, int64_t s, int page) { return item_base(start, s, page); }
int t_append_item(int64_t start, int64_t count, int64_t len, int64_t i, int page, int64_t* out) {
    AppendItem it;
    if (!append_item(start, count, len, i, page, &it)) return 0;
    out[0] = it.lp; out[1] = it.row0; out[2] = it.slot0; out[3] = it.n;
    return 1;
}
uint64_t t_share(uint64_t total, uint32_t c, uint32_t n) { return Shares(total, n).first(c); }
uint32_t t_share_of(uint64_t x, uint64_t total, uint32_t n) { return Shares(total, n).of(x); }
}
"""


@pytest.fixture(scope="module")
def ix(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("pages_index")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run([cxx, "-shared", "-fPIC", "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    so = ctypes.CDLL(str(lib))
    i64, i32, u32, u64 = ctypes.c_int64, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64
    P = ctypes.POINTER
    for name, res, args in [("t_clamp_len", i64, [i64, i64, i32, P(u32)]), ("t_seq_steps", u32, [i64, i32, i32]),
                            ("t_step_page", i64, [u32, i32, i32, i64, i64, P(i32), P(i32), P(u32)]),
                            ("t_check_page", i64, [i64, i64, P(u32)]), ("t_item_base", i64, [i64, i64, i32]),
                            ("t_append_item", i32, [i64, i64, i64, i64, i32, P(i64)]), ("t_share", u64, [u64, u32, u32]),
                            ("t_share_of", u32, [u64, u64, u32])]:
        f = getattr(so, name)
        f.restype, f.argtypes = res, args
    return so


def step_page(ix, step, page, n_sel, chosen, length):
    slot, valid, bad = ctypes.c_int(), ctypes.c_int(), ctypes.c_uint32()
    lp = ix.t_step_page(step, page, n_sel, chosen, length, slot, valid, bad)
    return lp, slot.value, valid.value, bad.value


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 31, 63, 64, 127, 128, 129, 500, 1851])
def test_steps_cover_every_token_once(ix, page, length):
    seen = []
    for s in range(ix.t_seq_steps(length, page, -1)):
        lp, slot, valid, bad = step_page(ix, s, page, -1, 0, length)
        assert bad == 0 and lp >= 0 and 1 <= valid <= 16 and slot + 16 <= page
        seen += range(lp * page + slot, lp * page + slot + valid)
    assert seen == list(range(length))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n_sel", [1, 3, 9])
def test_chosen_steps_stay_inside_the_sequence(ix, page, n_sel):
    for length in (0, 1, 63, 64, 65, 200, 513):
        pages = -(-length // page)
        n = ix.t_seq_steps(length, page, n_sel)
        assert n == min(n_sel, pages) * page // 16
        for chosen in (-(1 << 31), -1, 0, pages - 1, pages, pages + 1, (1 << 31) - 1):
            got = []
            for s in range(n):
                if s * 16 // page:
                    break   # the entry under test is the first
                lp, slot, valid, bad = step_page(ix, s, page, n_sel, chosen, length)
                assert bad == (4 if chosen >= pages else 0)
                if valid:
                    assert lp == chosen and 0 <= lp < pages
                    got += range(lp * page + slot, lp * page + slot + valid)
            want = range(chosen * page, min((chosen + 1) * page, length)) if 0 <= chosen < pages and n else []
            assert got == list(want)


def test_lengths_and_page_ids_out_of_range(ix):
    bad = ctypes.c_uint32()
    assert ix.t_clamp_len(-5, 10, 16, bad) == 0 and bad.value == 0
    assert ix.t_clamp_len(160, 10, 16, bad) == 160 and bad.value == 0
    assert ix.t_clamp_len(161, 10, 16, bad) == 160 and bad.value == 2
    bad = ctypes.c_uint32()
    assert ix.t_check_page(0, 7, bad) == 0 and ix.t_check_page(6, 7, bad) == 6 and bad.value == 0
    for wrong in (-1, 7, (1 << 31) - 1, -(1 << 31)):
        bad = ctypes.c_uint32()
        assert ix.t_check_page(wrong, 7, bad) == -1 and bad.value == 1


def find_seq(ix, starts, A, item, page):
    """The kernel's search, lane by lane: the last sequence whose items begin at or before `item`."""
    lo, n = 0, A
    while n > 1:
        stride = (n + 31) // 32
        assert stride < n
        le = [lane * stride < n and ix.t_item_base(starts[lo + lane * stride], lo + lane * stride, page) <= item
              for lane in range(32)]
        cnt = max(1, sum(le))
        lo += (cnt - 1) * stride
        n = min(stride, n - (cnt - 1) * stride)
        assert n >= 1 and 0 <= lo and lo + n <= A
    return lo


def items(ix, starts, lens, A, rows, page):
    out = (ctypes.c_int64 * 4)()
    for it in range(rows // page + 2 * A):
        s = find_seq(ix, starts, A, it, page)
        start, count = starts[s], starts[s + 1] - starts[s]
        if count < 0 or start < 0 or start + count > rows:
            continue   # the kernel flags it
        if ix.t_append_item(start, count, lens[s], it - ix.t_item_base(start, s, page), page, out):
            yield (s, *out)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("A", [1, 2, 5, 33, 70, 1100])
def test_append_items_cover_every_row_once(ix, page, A):
    rng = random.Random(page * A)
    lens = [rng.choice([0, 0, 1, page - 1, page, rng.randrange(500)]) for _ in range(A)]
    new = [rng.choice([0, 0, 1, 1, 2, page, page + 1, rng.randrange(300 if A < 100 else 20)]) for _ in range(A)]
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    got = {}
    for s, lp, row0, slot0, n in items(ix, starts, lens, A, starts[-1] + rng.randrange(40), page):
        assert 0 <= slot0 and slot0 + n <= page and n > 0
        for j in range(n):
            assert row0 + j not in got
            got[row0 + j] = (s, lp * page + slot0 + j)
    want = {starts[s] + i: (s, lens[s] + i) for s in range(A) for i in range(new[s])}
    assert got == want


def test_append_items_of_broken_starts_stay_in_bounds(ix):
    rng = random.Random(3)
    for _ in range(200):
        A, page, rows = rng.choice([1, 2, 7, 40]), rng.choice([16, 64]), rng.randrange(1, 200)
        starts = [rng.randrange(-300, 500) for _ in range(A + 1)]
        lens = [rng.randrange(-10, 300) for _ in range(A)]
        for s, lp, row0, slot0, n in items(ix, starts, lens, A, rows, page):
            assert 0 <= s < A and 0 <= row0 and row0 + n <= rows and 0 <= slot0 and slot0 + n <= page and lp >= 0
            assert lens[s] >= 0


@pytest.mark.parametrize("total,n", [(1, 1), (7, 3), (100, 7), (5, 5), (2, 9), ((1 << 40) + 13, 608), (608 * 4, 608)])
def test_shares_partition_the_list(ix, total, n):
    edges = [ix.t_share(total, c, n) for c in range(n + 1)]
    assert edges[0] == 0 and edges[-1] == total
    sizes = [b - a for a, b in zip(edges, edges[1:])]
    assert max(sizes) - min(sizes) <= 1
    for c in range(n):
        for x in {edges[c], edges[c + 1] - 1}:
            if edges[c] <= x < edges[c + 1]:
                assert ix.t_share_of(x, total, n) == c
