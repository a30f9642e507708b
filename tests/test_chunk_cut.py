"""The cut of a chunk-attention call into ranges per CTA, on the CPU: the
kernel's own arithmetic (csrc/chunk_cut.h) compiled for the host, walked CTA by
CTA as the kernel walks it."""
import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_verification_isd_b200", "csrc")

DRIVER = r"""
#include <vector>
#include "chunk_cut.h"
using namespace isd;

// Walks every CTA's range; 0 if each item's tiles are covered once, in order,
// its parts lie in consecutive CTAs and their number is what the first one
// works out, else the number of the check that failed.
extern "C" int walk(int B, const int* n, const int* kv, int Hkv, int tpq, int P, int max_pages, int two, int grid,
                    long long* total_out, long long* pieces) {
    CutShape a;
    a.P = P, a.max_pages = max_pages, a.tpq = tpq, a.two = two;
    std::vector<Request> req;
    std::vector<long long> head, before;
    long long total = 0;
    for (int b = 0, start = 0; b < B; start += n[b++]) {
        req.push_back(request_of(a, start, start + n[b], kv[b]));
        head.push_back(head_cost(a, req[b]));
        before.push_back(total);
        total += head[b] * Hkv;
    }
    *total_out = total;
    *pieces = 0;
    const int G = cut_ctas(a, total, grid);
    // the tile that has to come next, and where its item began
    int nb = 0, ng = 0, nq = 0, nt = 0, began = -1, parts = 0, last_cta = -1;
    auto skip_empty = [&] { while (nb < B && req[nb].items == 0) ++nb; };
    skip_empty();
    for (int cta = 0; cta < grid; ++cta) {
        const long long my0 = cta < G ? cut_start(total, G, cta) : 0, my1 = cta < G ? cut_start(total, G, cta + 1) : 0;
        if (my0 > my1 || my0 < 0 || my1 > total) return 1;
        if (my0 == my1) continue;
        int b = 0;
        while (b < B && !(my0 >= before[b] && my0 < before[b] + head[b] * Hkv)) ++b;
        if (b == B) return 2;
        int g, q;
        long long rel = -cut_item(a, req[b], head[b], my0 - before[b], g, q);
        const long long len = my1 - my0;
        while (b < B && rel < len) {
            const Item it = item_of(a, req[b], q);
            const long long start = rel;
            int t0, t1;
            cut_tiles(it, start, len, t0, t1);
            if (t0 < t1) {
                ++*pieces;
                if (b != nb || g != ng || q != nq || t0 != nt) return 3;
                if (t0 == 0) {
                    began = cta;
                    parts = 1;
                    if (t1 < it.nt) parts = cut_owner(total, G, my0 + start + (long long)(it.nt - 1) * it.w) - cta + 1;
                } else if (cta != last_cta + 1) {
                    return 4;
                }
                last_cta = cta;
                nt = t1;
                if (t1 == it.nt) {
                    if (cta - began + 1 != parts) return 5;
                    nt = 0;
                    if (++nq >= req[nb].items) {
                        nq = 0;
                        if (++ng >= Hkv) ng = 0, ++nb, skip_empty();
                    }
                }
            }
            rel += it.cost;
            if (++q >= req[b].items) {
                q = 0;
                if (++g >= Hkv) {
                    g = 0;
                    do ++b;
                    while (b < B && req[b].items == 0);
                }
            }
        }
    }
    return nb == B ? 0 : 6;
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("cut")
    (at / "walk.cpp").write_text(DRIVER)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, "-o", str(at / "walk.so"),
                    str(at / "walk.cpp")], check=True)
    return ctypes.CDLL(str(at / "walk.so"))


def ceil(a, b):
    return -(-a // b)


def cost(n, kv, tpq):
    """Cost of a request's items of one KV head, in whole numbers: 4 a tile and
    13 the ends of an item of two row tiles, 2 and 7 of one."""
    items, tiles = ceil(n, 2 * tpq), ceil(kv, 128)
    merged = n <= 16 and n <= tiles * 128 - kv
    ends = np.minimum((np.arange(items, dtype=object) + 1) * (2 * tpq), n)
    keys = tiles + (np.zeros_like(ends) if merged else (ends + 127) // 128)
    two = np.array([e - 2 * tpq * i > tpq for i, e in enumerate(ends)], dtype=bool)
    return int(np.where(two, 4 * keys + 13, 2 * keys + 7).sum())


def check(cut, n, kv, Hkv, grp, P, grid=148):
    tpq = 128 // grp
    cols = max(ceil(a + b, P) for a, b in zip(n, kv)) + 1
    total, pieces = ctypes.c_longlong(), ctypes.c_longlong()
    ints = ctypes.c_int * len(n)
    bad = cut.walk(len(n), ints(*n), ints(*kv), Hkv, tpq, P, cols, int(sum(n) > tpq), grid, ctypes.byref(total),
                   ctypes.byref(pieces))
    assert total.value == Hkv * sum(cost(a, b, tpq) for a, b in zip(n, kv) if a)
    assert bad == 0
    return total.value


def test_cut_random(cut):
    rng = random.Random(0)
    for _ in range(300):
        B = rng.choice([1, 1, 2, 5, 40])
        grp = rng.choice([1, 3, 4, 7, 8, 100, 128])
        top, far = rng.choice([1, 4, 40, 700]), rng.choice([0, 100, 5000, 100000])
        n = [rng.randint(0, top) for _ in range(B)]
        n[rng.randrange(B)] = top
        check(cut, n, [rng.randint(0, far) for _ in range(B)], rng.choice([1, 2, 8]), grp, rng.choice([1, 16, 24]),
              rng.choice([1, 2, 7, 132, 148, 192]))


@pytest.mark.parametrize("kv", [0, 1, 16383])
def test_cut_around_the_border_of_32_bits(cut, kv):
    """The starts of the ranges are taken in 32 bits up to a total of 2^23."""
    below = above = 0
    for n in range(30000, 90000, 3001):
        total = check(cut, [n, 3], [kv, kv], 8, 4, 16)
        below, above = below + (total < 1 << 23), above + (total >= 1 << 23)
    assert below and above


@pytest.mark.parametrize("n,Hkv,grp", [(6_100_000, 1, 4), (4_300_000, 2, 8), (1_070_000, 1, 128), (12_000_000, 1, 1)])
def test_cut_of_millions_of_new_tokens(cut, n, Hkv, grp):
    """More than 2^31 tiles of new tokens over a request's items."""
    assert check(cut, [5, n, 1], [0, 70, 9], Hkv, grp, 16) > 4 << 31


def test_cut_of_ranges_past_32_bits(cut):
    """A CTA's range longer than 2^31."""
    assert check(cut, [1 << 27], [1 << 26], 16, 1, 64) > 148 << 31
