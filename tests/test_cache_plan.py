"""The cache's places and the division of its reading (csrc/cache_plan.hpp)
compiled for the host (CPU only): what a kernel would read or write for tables,
positions and lengths in and out of range."""
import ctypes
import os
import random
import subprocess

import pytest

import implicit_gemm_nhwc_amd as igc

CSRC = os.path.join(os.path.dirname(igc.__file__), "csrc")
SRC = r"""
#include "cache_plan.hpp"
extern "C" {
int page(const int32_t* row, int64_t p, int shift, int entries, int pages) {
    return igc::cache_page(row, p, shift, entries, pages);
}
int64_t row(int id, int heads, int head, int64_t p, int shift) {
    return igc::cache_row(id, heads, head, p, shift);
}
int len(int n, int64_t capacity) { return igc::cache_len(n, capacity); }
int splits(int64_t slots, int64_t b) { return igc::cache_splits(slots, b); }
uint32_t units(int n) { return igc::cache_units(n); }
uint32_t chunk(uint32_t total, uint32_t per) { return igc::cache_chunk(total, per); }
int bisect() { return igc::kCacheBisect; }
int unit() { return igc::kCacheUnit; }
int least() { return igc::kCacheLeast; }
uint32_t parts(int n, uint32_t chunk) { return igc::cache_parts(n, chunk); }
int fixed(int64_t slots, int64_t b, int64_t cap) { return igc::cache_fixed(slots, b, cap); }
int64_t most(int64_t cap) { return igc::cache_most(cap); }
int64_t bound(int64_t slots, int64_t b, int64_t cap) { return igc::cache_slots_bound(slots, b, cap); }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(SRC)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC,
                    str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    i64 = ctypes.c_int64
    L.page.argtypes = [ctypes.POINTER(ctypes.c_int32), i64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    L.row.argtypes, L.row.restype = [ctypes.c_int] * 3 + [i64, ctypes.c_int], i64
    L.len.argtypes = [ctypes.c_int, i64]
    L.splits.argtypes = [i64, i64]
    u32 = ctypes.c_uint32
    L.units.argtypes, L.units.restype = [ctypes.c_int], u32
    L.chunk.argtypes, L.chunk.restype = [u32] * 2, u32
    L.fixed.argtypes, L.most.argtypes, L.most.restype = [i64] * 3, [i64], i64
    L.bound.argtypes, L.bound.restype = [i64] * 3, i64
    L.parts.argtypes, L.parts.restype = [ctypes.c_int, u32], u32
    return L


def test_places(plan):
    table = (ctypes.c_int32 * 4)(3, -1, 7, 0)
    for shift in (4, 7):
        t = 1 << shift
        want = {0: 3, t - 1: 3, t: -1, 2 * t: -1, 3 * t: 0, 4 * t - 1: 0, 4 * t: -1, -1: -1,
                -(1 << 31): -1, (1 << 31) - 1: -1, 1 << 31: -1}
        for p, id in want.items():
            assert plan.page(table, p, shift, 4, 7) == id, p   # page 7 is past a pool of 7
        assert plan.page(table, 2 * t, shift, 4, 8) == 7
        assert plan.page(table, 0, shift, 0, 8) == -1
    for id, heads, head, p, shift in ((0, 1, 0, 5, 4), (3, 8, 7, 1000, 4), ((1 << 31) - 2, 4, 3, 77, 6),
                                      (5, 10, 9, (1 << 31) - 5000, 10)):
        t = 1 << shift
        assert plan.row(id, heads, head, p, shift) == (id * heads + head) * t + p % t
    for n, cap, want in ((-1, 10, 0), (0, 10, 0), (11, 10, 10), (10, 10, 10), (9, 10, 9),
                         ((1 << 31) - 1, (1 << 31) - 5000, (1 << 31) - 5000), (5, 0, 0)):
        assert plan.len(n, cap) == want


def test_division(plan):
    """Every key is read once, no more workgroups are used than there is room
    for, and the splits are even."""
    rng = random.Random(1)
    for _ in range(400):
        b = rng.choice([1, 1, 2, 3, 17, 64, 65, 200])
        cap = rng.choice([16, 1040, 4096, 65536, 1 << 20, (1 << 31) - 5000])
        cap -= cap % 16
        lens = [plan.len(rng.choice([0, 1, cap, rng.randint(0, cap), 255, 257]), cap)
                for _ in range(b)]
        slots = rng.choice([1, 2, 5, 16, 64, 512])
        room = plan.bound(slots, b, cap)
        if not plan.splits(slots, b):
            assert room == b
            continue
        if plan.fixed(slots, b, cap):
            # slots of their own hold every sequence's smallest splits
            assert room == b * plan.most(cap) <= slots
            assert all(plan.parts(n, plan.least()) <= plan.most(cap) for n in lens + [cap])
        else:
            assert room == slots < b * plan.most(cap)
        total = sum(plan.units(n) for n in lens)
        assert total < 1 << 32
        c, low = plan.chunk(total, slots - b), plan.chunk(total, slots)
        for _ in range(plan.bisect()):
            if low < c:
                mid = low + (c - low) // 2
                if sum(plan.parts(n, mid) for n in lens) <= slots:
                    c = mid
                else:
                    low = mid + 1
        parts = [plan.parts(n, c) for n in lens]
        assert c >= plan.least() and sum(parts) <= room
        for n, k in zip(lens, parts):
            assert k >= 1
            at = 0
            for i in range(k):
                lo, hi = i * c * plan.unit(), min((i + 1) * c * plan.unit(), n)
                assert lo == at and (hi > lo or n == 0)
                at = max(hi, at)
            assert at == n
