"""The split of the paged kernels' work over their CTAs, on the CPU: every CTA's
stretch of the line of tiles is walked with the kernels' own code
(csrc/paged_line.cuh) and compared with a plain enumeration of the units.

Each tile of each unit has to come up once, in order; only a stretch's first
and last unit may be shared; and a shared unit's partials have to lie where the
joining kernels look for them.  (Only the warp-wide search for a stretch's
first unit in a long prompt is not part of this: the walk finds it alone.)
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
#include <tuple>
#include <vector>
#include "paged_line.cuh"
using namespace fa;
static int bad = 0;
#define CHECK(x) do { if (!(x) && bad++ < 10) printf("line %d: %s\n", __LINE__, #x); } while (0)

static std::mt19937 rng(11);
static int pick(int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); }

struct Batch {
    std::vector<int> q_start, kv_len;
    PagedParams p{};
    void make(int B, int most_new, int most_kv, int group, int shared, bool contradict) {
        q_start.assign(1, 0);
        kv_len.clear();
        for (int b = 0; b < B; ++b) {
            const int n = pick(0, 4) ? pick(0, most_new) : 0;
            q_start.push_back(q_start.back() + n);
            kv_len.push_back(shared + n + pick(0, 3) * pick(0, most_kv) / 3);
            if (contradict && pick(0, 5) == 0) kv_len.back() = pick(0, 1) ? n - 1 : 1 << 28;
        }
        p.c.B = B;
        p.c.Hkv = pick(1, 4);
        p.c.page_size = 64;
        p.c.page_shift = 6;
        p.c.max_pages = 1 << 20;
        p.c.total_q = q_start.back() + pick(0, 3);
        p.c.q_start = q_start.data();
        p.c.kv_len = kv_len.data();
        p.mask = PagedMask{pick(0, 1), -1, 0};
        if (p.mask.causal && pick(0, 1)) { p.mask.window = pick(0, 500); p.mask.sinks = pick(0, 1) * pick(0, 300); }
        p.group = group;
        p.Hq = group * p.c.Hkv;
        p.by_group = fast_div(group);
        p.max_q = most_new;
        p.shared = shared;
        p.join_rows = shared > 0;
        p.ctas = pick(0, 2) ? pick(1, 60) : 304;
    }
};

// a unit in the order of the line, and the part of one in a CTA
struct Unit { int b, h, row0, rows, tiles; };
struct Part { int cta, b, h, row0, rows, tiles, k0, k1, count; };

static void compare(const std::vector<Unit>& units, const std::vector<Part>& parts, int ctas) {
    size_t at = 0;
    for (const Unit& u : units) {
        int k = 0, first = -1, count = 0;
        for (size_t n = 0; k < u.tiles; ++n, ++at) {
            if (at >= parts.size()) { CHECK(!"a part is missing"); return; }
            const Part& x = parts[at];
            CHECK(x.b == u.b && x.h == u.h && x.row0 == u.row0 && x.rows == u.rows && x.tiles == u.tiles);
            CHECK(x.k0 == k && x.k1 > k && x.k1 <= u.tiles);
            // one part per CTA, in CTAs one after another; inside a stretch units are whole
            if (n == 0) { first = x.cta; count = x.count; } else CHECK(x.cta == first + (int)n);
            if (x.k0 > 0) CHECK(at == 0 || parts[at - 1].cta != x.cta);
            if (x.k1 < u.tiles) CHECK(at + 1 == parts.size() || parts[at + 1].cta != x.cta);
            // (count is what the first part is asked for)
            if (x.k1 == u.tiles) CHECK(count == (int)n + 1);
            // the slot that the part is written to is the one that the join reads
            const int stride = 256, r = 3;
            const long long slot = (2LL * x.cta + (x.k0 == 0 ? 1 : 0)) * stride + r;
            const RowParts rp = unit_parts(PagedParts{}, first, count, stride, r);
            if (!(x.k0 == 0 && x.k1 == u.tiles)) {
                CHECK(rp.at((int)n) == slot && rp.within(2LL * ctas * stride));
            }
            if (bad > 10) return;
            k = x.k1;
        }
    }
    CHECK(at == parts.size());
}

template <int SHIFT>
static void small(const Batch& t) {
    const PagedParams& p = t.p;
    std::vector<Unit> units;
    int bare = 0;
    for (int b = 0; b < p.c.B; ++b) {
        const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, nullptr);
        if (s.n == 0) continue;
        const Hull u = make_hull(p.mask, s.kv - s.n, s.kv - 1, p.shared, s.kv, SHIFT);
        bare += u.tiles;
        for (int h = 0; h < p.c.Hkv; ++h) units.push_back({b, h, 0, s.n, u.tiles});
    }
    const int shift = group_shift(p.c.B), groups = groups_of(p.c.B);
    std::vector<int> pre(groups + 1, 0);
    for (int g = 0; g < groups; ++g) pre[g + 1] = pre[g] + group_length<SHIFT>(p, shift, g, nullptr);
    CHECK(pre[groups] == bare);
    const int front = p.c.Hkv * pre[groups] >= kManyTiles * p.ctas;
    if (front) {
        std::vector<int> with(groups + 1, 0);
        for (int g = 0; g < groups; ++g)
            with[g + 1] = with[g] + group_length_front<SHIFT>(p, shift, g, pre[g + 1] - pre[g]);
        pre = with;
    }
    std::vector<Part> parts;
    for (int cta = 0; cta < p.ctas; ++cta) {
        Line ln{};
        ln.pre = pre.data();
        ln.shift = shift;
        ln.front = front;
        line_share(p.c.Hkv * pre[groups], p.ctas, cta, ln.per, ln.t, ln.t1);
        if (ln.t >= ln.t1) continue;
        ln.g = line_find(pre.data(), groups, p.c.Hkv, ln.t);
        open_group<SHIFT>(p, ln);
        SmallSeg s;
        while (next_seg<SHIFT>(p, ln, s)) {
            CHECK(s.q0 == t.q_start[s.b] && s.kv == t.kv_len[s.b]);
            parts.push_back({cta, s.b, s.h, 0, s.n, s.tiles, s.k0, s.k1, s.count});
            if (parts.size() > 1000000) { CHECK(!"no end"); return; }
        }
    }
    compare(units, parts, p.ctas);
}

static void tiles(const Batch& t) {
    const PagedParams& p = t.p;
    std::vector<Unit> units;
    std::vector<int> pre(p.c.B + 1, 0), kv(p.c.B), q0(p.c.B + 1);
    for (int b = 0; b < p.c.B; ++b) {
        const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, nullptr);
        int sum = 0;
        for (int rt = 0; rt * kPagedTileRows < s.n * p.group; ++rt) {
            const int row0 = rt * kPagedTileRows, rows = std::min(kPagedTileRows, s.n * p.group - row0);
            const int i0 = s.kv - s.n + row0 / p.group, i1 = s.kv - s.n + (row0 + rows - 1) / p.group;
            const int n = make_hull(p.mask, i0, i1, p.shared, s.kv, 7).tiles;
            for (int h = 0; h < p.c.Hkv; ++h) units.push_back({b, h, row0, rows, n});
            sum += unit_length(p, s.n, s.kv, rt);
            CHECK(unit_length(p, s.n, s.kv, rt) == n + kUnitTiles);
        }
        pre[b + 1] = pre[b] + sum;
        kv[b] = s.kv;
        q0[b] = s.q0;
        q0[b + 1] = s.q0 + s.n;
    }
    std::vector<Part> parts;
    for (int cta = 0; cta < p.ctas; ++cta) {
        TileLine ln{};
        ln.pre = pre.data();
        ln.kv = kv.data();
        ln.q0 = q0.data();
        line_share(p.c.Hkv * pre[p.c.B], p.ctas, cta, ln.per, ln.t, ln.t1);
        if (ln.t >= ln.t1) continue;
        ln.b = line_find(pre.data(), p.c.B, p.c.Hkv, ln.t);
        ln.start = p.c.Hkv * pre[ln.b];
        TileSeg s;
        while (next_seg(p, ln, s)) {
            parts.push_back({cta, s.b, s.h, s.row0, s.rows, s.tiles, s.k0, s.k1, s.count(ln.per)});
            if (parts.size() > 1000000) { CHECK(!"no end"); return; }
        }
    }
    compare(units, parts, p.ctas);
}

static void prefix(Batch t) {
    PagedParams& p = t.p;
    p.prefix = 1;
    int lo = INT_MAX, hi = INT_MIN;
    for (int b = 0; b < p.c.B; ++b) {
        const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, nullptr);
        if (s.n > 0) lo = std::min(lo, s.kv - s.n), hi = std::max(hi, s.kv - 1);
    }
    std::vector<Unit> units;
    std::vector<Part> parts;
    int per = 0, n = 0;
    for (int cta = 0; cta < p.ctas; ++cta) {
        TileLine ln{};
        ln.imin = lo;
        ln.imax = hi;
        const int total = prefix_line(p, ln, t.q_start.back());
        if (cta == 0) {
            const int rows = lo <= hi ? t.q_start.back() * p.group : 0;
            n = ln.prefix_tiles;
            for (int row0 = 0; row0 < rows; row0 += kPagedTileRows)
                for (int h = 0; h < p.c.Hkv; ++h)
                    units.push_back({0, h, row0, std::min(kPagedTileRows, rows - row0), n});
            if (rows) CHECK(n == make_hull(p.mask, lo, hi, 0, p.shared, 7).tiles);
        }
        line_share(total, p.ctas, cta, ln.per, ln.t, ln.t1);
        per = ln.per;
        TileSeg s;
        while (next_seg(p, ln, s)) parts.push_back({cta, s.b, s.h, s.row0, s.rows, s.tiles, s.k0, s.k1, s.count(ln.per)});
    }
    compare(units, parts, p.ctas);
    // where the joining kernel looks for the rows' partials
    for (size_t at = 0; at < parts.size(); ++at) {
        const Part& x = parts[at];
        if (x.k0 > 0) continue;
        for (int r : {0, x.rows / 2, x.rows - 1}) {
            const float2 ml{};
            PagedParts w{};
            w.slot_ml = const_cast<float2*>(&ml);
            const RowParts rp = prefix_parts(w, n, per, p.c.Hkv, x.row0 + r, x.h, 777);
            if (x.k1 == x.tiles) {
                CHECK(rp.ml == nullptr && rp.first == 777 && rp.count == 1);
            } else {
                CHECK(rp.ml == &ml && rp.count == x.count && rp.first == (2LL * x.cta + 1) * kPagedTileRows + r);
                CHECK(rp.within(2LL * p.ctas * kPagedTileRows));
            }
        }
    }
}

int main() {
    for (int it = 0; it < 4000 && !bad; ++it) {
        Batch t;
        const int group = pick(1, 9), shared = pick(0, 1) * 64 * pick(1, 30);
        t.make(pick(1, 20), pick(1, 16 / group), pick(0, 3) ? 300 : 9000, group, shared, pick(0, 3) == 0);
        small<6>(t);
        small<7>(t);
        t.make(pick(1, 20), pick(0, 2) ? pick(1, 90) : 700, pick(0, 3) ? 300 : 9000, pick(0, 5) ? group : 300, shared, pick(0, 3) == 0);
        tiles(t);
        if (shared) prefix(t);
    }
    // an entry of the line's index for 2 and for 4 sequences
    for (int B : {999, 1000, 1001, 1500, 1999, 2000, 2001, 2047, 2048})
        for (int it = 0; it < 12 && !bad; ++it) {
            Batch t;
            t.make(B, 2, it % 3 ? 100 : 2000, 2, it % 2 * 64, it % 4 == 0);
            small<6>(t);
            small<7>(t);
            tiles(t);
            if (t.p.shared) prefix(t);
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


def test_line(nvcc, tmp_path):
    src, exe = tmp_path / "line.cu", tmp_path / "line"
    src.write_text(SOURCE)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "block_sparse_attention_fa_gb300", "csrc"),
                    "-gencode", "arch=compute_103a,code=sm_103a", "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
