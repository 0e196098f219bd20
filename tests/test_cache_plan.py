"""Index arithmetic of the paged token cache (cache_plan.cuh), compiled here as
plain C++ (CPU only): spans cover the work once, what device memory says is
clamped into range, an append's page numbers do not meet."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "latent_query_split_gb300", "csrc")

SOURCE = r"""
#include "cache_plan.cuh"
using namespace flare::cache;
extern "C" {
void seq(const int32_t *cu, int n, long long T, const int32_t *lens, int cap, int b, long long *out) {
    Seq s = sequence(cu, n, T, lens, cap, b);
    out[0] = s.t0; out[1] = s.n; out[2] = s.len; out[3] = s.ok;
}
static Seq make(int n, int len) { Seq s; s.t0 = 0; s.n = n; s.len = len; s.ok = true; return s; }
int row_tiles_(int n, int len, int G, int rows) { return row_tiles(make(n, len), G, rows); }
int visible_(int n, int len, int G, int rows, int rt, int c) { return visible(make(n, len), G, rows, rt, c); }
int limit_(int n, int len, int i, int c) { return limit_of(make(n, len), i, c); }
int item_(int n, int len, int G, int rows, int rt, int c) { return item_tiles(make(n, len), G, rows, rt, c); }
long long seq_tiles_(int n, int len, int G, int rows, int c) { return seq_tiles(make(n, len), G, rows, c); }
long long span_begin_(long long total, int parts, int c) { return span_begin(total, parts, c); }
int part_of_(long long total, int parts, long long t) { return part_of(total, parts, t); }
long long first_slot_(long long t0, int b, int page) { return first_slot(t0, b, page); }
long long slot_bound_(long long T, int B, int page) { return slot_bound(T, B, page); }
int touched_(int len, int n, int page) { return touched_pages(len, n, page); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-o", str(so), str(src)], check=True)
    x = ctypes.CDLL(str(so))
    for name in ("seq_tiles_", "span_begin_", "first_slot_", "slot_bound_"):
        getattr(x, name).restype = ctypes.c_longlong
    L = ctypes.c_longlong
    x.span_begin_.argtypes = [L, ctypes.c_int, ctypes.c_int]
    x.part_of_.argtypes = [L, ctypes.c_int, L]
    x.first_slot_.argtypes = [L, ctypes.c_int, ctypes.c_int]
    x.slot_bound_.argtypes = [L, ctypes.c_int, ctypes.c_int]
    x.seq.argtypes = [ctypes.c_void_p, ctypes.c_int, L, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return x


def _seq(lib, cu, n, T, lens, cap, b):
    out = (ctypes.c_longlong * 4)()
    arr = (ctypes.c_int32 * len(cu))(*cu) if cu is not None else None
    lib.seq(arr, n, T, (ctypes.c_int32 * len(lens))(*lens), cap, b, out)
    return tuple(out)


def test_sequences_are_clamped_into_range(lib):
    assert _seq(lib, [0, 3, 3, 10], 0, 10, [5, 0, 64], 64, 0) == (0, 3, 5, 1)
    assert _seq(lib, [0, 3, 3, 10], 0, 10, [5, 0, 64], 64, 1) == (3, 0, 0, 1)
    assert _seq(lib, None, 4, 12, [5, 0, 64], 64, 2) == (8, 4, 64, 1)
    rng = random.Random(0)
    wild = [-2 ** 31, -7, -1, 0, 1, 9, 10, 11, 2 ** 31 - 1]
    for _ in range(2000):
        cu, lens = [rng.choice(wild) for _ in range(4)], [rng.choice(wild) for _ in range(3)]
        for b in range(3):
            t0, n, length, ok = _seq(lib, cu, 0, 10, lens, 9, b)
            assert 0 <= t0 <= 10 and 0 <= n and t0 + n <= 10 and 0 <= length <= 9
            fine = 0 <= cu[b] <= cu[b + 1] <= 10 and 0 <= lens[b] <= 9
            assert bool(ok) == fine
            if fine:
                assert (t0, n, length) == (cu[b], cu[b + 1] - cu[b], lens[b])


@pytest.mark.parametrize("causal", [0, 1])
def test_row_tiles_and_what_they_see(lib, causal):
    rng = random.Random(causal)
    for _ in range(400):
        n, length, G, rows = rng.randint(0, 40), rng.randint(0, 700), rng.randint(1, 9), rng.choice([8, 16, 32, 128])
        m = lib.row_tiles_(n, length, G, rows)
        assert m == -(-n * G // rows)
        total = 0
        for rt in range(m):
            tokens = [r // G for r in range(rt * rows, min(n * G, (rt + 1) * rows))]
            want = max((max(0, length - n + i + 1) if causal else length) for i in tokens)
            assert lib.visible_(n, length, G, rows, rt, causal) == want
            for i in tokens:
                assert lib.limit_(n, length, i, causal) == (max(0, length - n + i + 1) if causal else length)
            tiles = lib.item_(n, length, G, rows, rt, causal)
            assert tiles == max(1, -(-want // 128))
            total += tiles
        assert lib.seq_tiles_(n, length, G, rows, causal) == total


def test_spans_cover_the_tiles_once(lib):
    rng = random.Random(2)
    for _ in range(500):
        total = rng.choice([1, 2, 7, 151, 152, 153, 1000, rng.randint(1, 10 ** 9), 3 * 10 ** 11])
        parts = min(rng.choice([1, 2, 152, 304, 608]), total)
        begins = [lib.span_begin_(total, parts, c) for c in range(parts + 1)]
        assert begins[0] == 0 and begins[-1] == total
        assert all(x < y for x, y in zip(begins, begins[1:]))              # no span is empty
        for t in {0, total - 1, rng.randrange(total), rng.randrange(total)}:
            c = lib.part_of_(total, parts, t)
            assert begins[c] <= t < begins[c + 1]


def test_append_slots_do_not_meet(lib):
    rng = random.Random(3)
    for _ in range(300):
        page = rng.choice([16, 32, 64, 128])
        B = rng.randint(1, 12)
        counts = [rng.choice([0, 0, 1, 2, page - 1, page, page + 1, rng.randint(0, 400)]) for _ in range(B)]
        T, t0, used = sum(counts), 0, set()
        for b, n in enumerate(counts):
            length = rng.choice([0, 1, page - 1, page, rng.randint(0, 10 ** 6)])
            touched = lib.touched_(length, n, page)
            assert touched == len({(length + i) // page for i in range(n)})
            for i in range(touched):
                slot = lib.first_slot_(t0, b, page) + i
                assert 0 <= slot < lib.slot_bound_(T, B, page) and slot not in used
                used.add(slot)
            t0 += n
