"""The paged kernels' index arithmetic on the CPU: the checks of a sequence's
numbers, the keys and tiles a unit visits, and the split of the line of tiles
over CTAs, compiled from the kernels' own header and compared with brute force.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r'''
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>
#include "paged.cuh"
using namespace fa;
static int bad = 0;
#define CHECK(x) do { if (!(x) && bad++ < 10) printf("line %d: %s\n", __LINE__, #x); } while (0)

int main() {
    std::mt19937 rng(7);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    // numbers of every kind: only sequences that fit come through
    const int odd[] = {INT_MIN, INT_MIN + 1, -5, -1, 0, 1, 2, 7, 16, 31, 32, 33, 64, 100, INT_MAX - 1, INT_MAX};
    PagedView c{};
    c.B = 3; c.Hkv = 2; c.num_pages = 9; c.page_size = 16; c.page_shift = 4; c.max_pages = 4; c.total_q = 33;
    for (int b = 0; b < 2; ++b)
        for (int q0 : odd) for (int q1 : odd) for (int kv : odd) for (int mq : {1, 16, INT_MAX}) for (int sh : {0, 32}) {
            SeqInfo s;
            const bool ok = check_sequence(c, b, q0, q1, kv, mq, sh, s);
            const bool empty = q0 == q1 && q0 >= 0 && q1 <= 33 && (b > 0 || q0 == 0);
            const long long n = (long long)q1 - q0;
            const bool fits = q0 >= 0 && n > 0 && q1 <= 33 && (b > 0 || q0 == 0) && n <= mq && kv >= n && kv <= 64 && kv >= sh;
            CHECK(ok == (empty || fits));
            CHECK(s.n == (fits ? n : 0));
        }
    // a unit's hull against its rows, one by one
    for (int it = 0; it < 60000; ++it) {
        PagedMask m{pick(0, 1), -1, 0};
        if (m.causal && pick(0, 2)) { m.window = pick(0, 3) ? pick(0, 400) : 0; if (pick(0, 1)) m.sinks = pick(0, 300); }
        const int kv = pick(1, 900), n = pick(1, kv < 40 ? kv : 40);
        int i0 = kv - n + pick(0, n - 1), i1 = i0 + pick(0, kv - 1 - i0);
        const int cut = pick(0, 2) ? 0 : pick(0, kv);
        const bool prefix = cut > 0 && pick(0, 1);
        const int jlo = prefix ? 0 : cut, jhi = prefix ? cut : kv;
        const int sh = pick(6, 7), T = 1 << sh;
        const Hull u = make_hull(m, i0, i1, jlo, jhi, sh);
        std::set<int> tiles;
        for (int k = 0; k < u.tiles; ++k) {
            const int kb = u.tile(k);
            CHECK(kb >= 0 && (k == 0 || kb > u.tile(k - 1)));
            tiles.insert(kb);
            // what is read lies inside the sequence
            for (int a = kb * T; a < kb * T + T; a += 16)
                if (u.any(a, a + 16)) CHECK(a < kv);
            bool every = true, open = true;
            for (int j = kb * T; j < kb * T + T; ++j) {
                every &= u.live(j);
                for (int i = i0; i <= i1; ++i) open &= paged_visible(m, i, j, jlo, jhi);
            }
            CHECK(u.all(kb * T, kb * T + T) <= every);
            CHECK(tile_open(m, kb, i0, i1, jlo, jhi, sh) <= open);
            CHECK(open <= every);
        }
        for (int j = -130; j < kv + 200; ++j) {
            bool seen = false;
            for (int i = i0; i <= i1; ++i) seen |= paged_visible(m, i, j, jlo, jhi);
            CHECK(seen <= u.live(j));                                   // nothing that is seen is left out
            if (seen) CHECK(tiles.count(j >> sh));
            if (u.live(j)) CHECK(j >= jlo && j < jhi && u.any(j, j + 1) && tiles.count(j >> sh));
            if (j >= 0 && j % 16 == 0) {
                bool any = false;
                for (int e = 0; e < 16; ++e) any |= u.live(j + e);
                CHECK(any == u.any(j, j + 16));
            }
        }
    }
    // partials: what lies in the slots, row by row
    for (int it = 0; it < 20000; ++it) {
        const RowParts a{nullptr, nullptr, pick(0, 4) ? pick(-3, 400) : (pick(0, 1) ? INT_MAX : INT_MIN),
                         pick(0, 4) ? pick(-2, 9) : (pick(0, 1) ? INT_MAX : INT_MIN), pick(0, 1) ? 16 : 256};
        const long long rows = pick(1, 12) * 2LL * a.stride;
        bool in = a.count >= 1;
        for (int k = 0; in && k < a.count && k < 100; ++k) in = a.at(k) >= 0 && a.at(k) < rows;
        CHECK(a.within(rows) == in);
    }
    // the division by the group size
    for (uint32_t d : {1u, 2u, 3u, 5u, 6u, 7u, 8u, 12u, 31u, 64u, 100u, 255u, 65537u, 2147483647u}) {
        const FastDiv f = fast_div(d);
        auto q = [&](uint32_t n) { return (uint32_t)((((unsigned long long)f.m * n) >> 32) + n) >> f.s; };
        for (uint32_t n : {0u, 1u, d - 1, d, d + 1, 2147483646u, 2147483647u}) CHECK((int)n < 0 || q(n) == n / d);
        for (int it = 0; it < 20000; ++it) { const uint32_t n = rng() >> 1; CHECK(q(n) == n / d); }
    }
    printf("%d\n", bad);
    return bad != 0;
}
'''


@pytest.fixture(scope="module")
def nvcc():
    nv = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nv):
        pytest.skip("no CUDA toolkit")
    return nv


def test_units(nvcc, tmp_path):
    src, exe = tmp_path / "units.cu", tmp_path / "units"
    src.write_text(SOURCE)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "block_sparse_attention_fa_gb300", "csrc"),
                    "-gencode", "arch=compute_103a,code=sm_103a", "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
