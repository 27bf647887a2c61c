"""What a query sees (csrc/view.cuh), compiled with g++ and held against its definition: the pages a
window's or a tree's row walks hold every token the query sees, in order, and the 64-bit masks of
those pages mark exactly the seen ones."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r'''
#include <stddef.h>
#include "view.cuh"
using namespace mla;
extern "C" int row_len(int kind, int sinks, int window, int L, int n, int plan_sq, int n_q, int j, int page, int max_len) {
    return view_row_len(kind, sinks, window, L, n, plan_sq, n_q, j, page, max_len);
}
// For each virtual token of the row: its token and whether seen() has it; per page the seen64() mask.
extern "C" void walk(int kind, int sinks, int window, int L, int n, unsigned long long mask, int n_q, int j, int page,
                     int len, int *token, int *seen, unsigned long long *bits) {
    View v{};
    v.kind = kind; v.sinks = sinks; v.window = window;
    unsigned long long masks[64];
    for (int i = 0; i < 64; ++i) masks[i] = mask;
    v.n_nodes = &n; v.mask = masks;
    const ItemView iv = item_view(v, &L, 0, j, n_q, page);
    for (int t = 0; t < len; ++t) { token[t] = iv.token(t); seen[t] = iv.seen(token[t]); }
    for (int p = 0; p < (len + 63) / 64; ++p) bits[p] = iv.seen64(iv.token(64 * p));
}
'''
WINDOW, TREE = 1, 2


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("view")
    (d / "probe.cpp").write_text(SRC)
    so = d / "probe.so"
    subprocess.run([gxx, "-x", "c++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "mla_latent_kv_24_b200", "csrc"), str(d / "probe.cpp"), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def _walk(lib, kind, sinks, window, L, n, mask, n_q, j, page, length):
    tok, seen = (ctypes.c_int * length)(), (ctypes.c_int * length)()
    bits = (ctypes.c_uint64 * ((length + 63) // 64))()
    lib.walk(kind, sinks, window, L, n, ctypes.c_uint64(mask), n_q, j, page, length, tok, seen, bits)
    return list(tok), [bool(x) for x in seen], list(bits)


def _check(tok, seen, bits, L, wanted, page):
    assert tok == sorted(set(tok)), "tokens rise"
    assert all(0 <= t < L for t in tok)
    assert {t for t, s in zip(tok, seen) if s} == wanted
    for v in range(0, len(tok), page):                      # a page is never cut
        assert tok[v] % page == 0
        assert tok[v:v + page] == list(range(tok[v], tok[v] + len(tok[v:v + page])))
    if page == 64:
        for p, m in enumerate(bits):
            t0 = tok[64 * p]
            assert {t0 + i for i in range(64) if (m >> i) & 1} == {t for t in wanted if t0 <= t < t0 + 64}


def _window_seen(L, n_q, j, sinks, window):
    p = L - n_q + j
    return {t for t in range(p + 1) if t < sinks or t > p - window}


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_window_rows(lib, page):
    rnd = random.Random(page)
    cases = [(1, 1, 0, 1), (64, 1, 0, 1), (65, 1, 0, 1), (65, 1, 64, 1), (1000, 1, 4, 64), (1000, 2, 64, 65), (129, 4, 1, 2),
             (500, 1, 2 ** 31 - 1, 1), (500, 1, 0, 2 ** 31 - 1), (500, 3, 2 ** 31 - 1, 2 ** 31 - 1), (4, 4, 0, 1)]
    for _ in range(300):
        n_q = rnd.randint(1, 4)
        cases.append((rnd.randint(n_q, 900), n_q, rnd.choice([0, 1, 4, 63, 64, 65, 100, 400]), rnd.choice([1, 2, 63, 64, 65, 200, 1000])))
    for L, n_q, sinks, window in cases:
        for j in range(n_q):
            length = lib.row_len(WINDOW, sinks, window, L, 0, n_q, n_q, j, page, 1 << 20)
            wanted = _window_seen(L, n_q, j, sinks, window)
            tok, seen, bits = _walk(lib, WINDOW, sinks, window, L, 0, 0, n_q, j, page, length)
            _check(tok, seen, bits, L, wanted, page)
            pages = {t // page for t in wanted}
            if len(wanted) < L - n_q + j + 1 and not any(p + 1 in pages or p - 1 in pages for p in pages):
                assert len({t // page for t in tok}) == len(pages)
        # all queries of the request together: every token that one of them sees
        if n_q > 1:
            length = lib.row_len(WINDOW, sinks, window, L, 0, 1, n_q, 0, page, 1 << 20)
            tok, seen, bits = _walk(lib, WINDOW, sinks, window, L, 0, 0, n_q, -1, page, length)
            union = set().union(*(_window_seen(L, n_q, j, sinks, window) for j in range(n_q)))
            assert union <= {t for t, s in zip(tok, seen) if s}


def test_window_rows_leave_out_the_pages_between(lib):
    # 10,000 tokens, 4 sinks, a window of 100: one page of sinks and at most three of the window
    length = lib.row_len(WINDOW, 4, 100, 10000, 0, 1, 1, 0, 64, 1 << 20)
    tok, _, _ = _walk(lib, WINDOW, 4, 100, 10000, 0, 0, 1, 0, 64, length)
    assert {t // 64 for t in tok} == {0} | set(range((10000 - 100) // 64, (9999 // 64) + 1))


def test_tree_rows(lib):
    rnd = random.Random(7)
    for n in [1, 2, 31, 32, 33, 63, 64] + [rnd.randint(1, 64) for _ in range(60)]:
        for ctx in [0, 1, 63, 64, 65, 127, 128, rnd.randint(0, 700)]:
            mask = rnd.choice([0, 1, 1 << 63, (1 << 64) - 1, rnd.getrandbits(64)])
            L = ctx + n
            assert lib.row_len(TREE, 0, 0, L, n, 64, 64, n - 1, 64, 1 << 20) == L
            if n < 64:
                assert lib.row_len(TREE, 0, 0, L, n, 64, 64, n, 64, 1 << 20) == 0     # a slot without a node
            tok, seen, bits = _walk(lib, TREE, 0, 0, L, n, mask, 64, 0, 64, L)
            _check(tok, seen, bits, L, set(range(ctx)) | {ctx + i for i in range(n) if (mask >> i) & 1}, 64)


def test_lengths_that_cannot_be(lib):
    assert lib.row_len(TREE, 0, 0, 3, 4, 8, 8, 0, 64, 1 << 20) == -1        # more nodes than tokens
    assert lib.row_len(TREE, 0, 0, 30, 9, 8, 8, 0, 64, 1 << 20) == -1       # more nodes than slots
    assert lib.row_len(TREE, 0, 0, 30, -1, 8, 8, 0, 64, 1 << 20) == -1
    assert lib.row_len(TREE, 0, 0, 65, 1, 8, 8, 0, 64, 64) == -1            # longer than the page table
    assert lib.row_len(TREE, 0, 0, 0, 0, 8, 8, 0, 64, 64) == 0              # an idle request
    assert lib.row_len(WINDOW, 4, 8, 1, 0, 2, 2, 0, 64, 1 << 20) == -1      # shorter than its queries
    assert lib.row_len(WINDOW, 4, 8, 65, 0, 1, 1, 0, 64, 64) == -1
