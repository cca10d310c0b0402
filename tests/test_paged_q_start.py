"""Offsets (q_start) of any kind in a paged step.

The kernels bound their work by total_q, so offsets that decrease have to be
seen before the work is counted: 0, T, 0, T, .. makes B / 2 sequences of the same
T rows.  On the CPU, with the kernels' own checks: sequences that come through
ordered offsets are disjoint, and what the joining kernel of a shared prefix
computes for the others does lie outside its slots unless it is checked.  On
the GPU: such a batch is reported, and what runs after it is right.
"""
import os
import subprocess

import pytest
import torch

from tests.test_paged import Batch, compare, fa, reference  # noqa: F401  (fa: the fixture)
from tests.test_paged_line import ROOT, nvcc  # noqa: F401  (the fixture)

gpu = pytest.mark.gpu

SOURCE = r'''
#include <cstdio>
#include <random>
#include <vector>
#include "paged_line.cuh"
using namespace fa;
static int bad = 0;
#define CHECK(x) do { if (!(x) && bad++ < 10) printf("line %d: %s\n", __LINE__, #x); } while (0)

int main() {
    std::mt19937 rng(5);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    int seen_more = 0, seen_outside = 0;
    for (int it = 0; it < 20000; ++it) {
        const int B = pick(1, 12), T = pick(1, 400);
        std::vector<int> qs(B + 1), kv(B, 4000);
        const int kind = pick(0, 3);
        for (int b = 0; b <= B; ++b)
            qs[b] = kind == 0 ? (b % 2 ? T : 0) : kind == 1 ? pick(-2, T + 2) : kind == 2 ? (b ? qs[b - 1] + pick(0, T / B + 1) : 0)
                  : (b ? qs[b - 1] + pick(-1, T / B + 1) : pick(0, 1));
        if (kind == 0 && pick(0, 1)) qs[B] = pick(0, 2);
        PagedParams p{};
        p.c = PagedView{B, 2, 100, 64, 6, 1 << 20, T, nullptr, kv.data(), qs.data()};
        p.group = pick(1, 8);
        p.Hq = 2 * p.group;
        p.by_group = fast_div(p.group);
        p.max_q = INT_MAX;
        p.mask = PagedMask{1, -1, 0};
        p.shared = 3000;
        p.prefix = 1;
        p.ctas = pick(1, 20);
        bool ordered = true;
        long long rows = 0;
        int last = 0, lo = INT_MAX, hi = INT_MIN;
        bool disjoint = true;
        for (int b = 0; b < B; ++b) {
            const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, nullptr);
            ordered = ordered && s.ordered;
            if (s.n == 0) continue;
            CHECK(s.q0 >= 0 && s.q0 + s.n <= T);
            rows += s.n;
            disjoint = disjoint && s.q0 >= last;
            last = s.q0 + s.n;
            lo = std::min(lo, s.kv - s.n);
            hi = std::max(hi, s.kv - 1);
        }
        // the work of a batch in order fits what the host has bounded
        if (ordered) CHECK(disjoint && rows <= T);
        if (rows > T) ++seen_more;
        bool order = qs[0] == 0;
        for (int b = 0; b < B; ++b) order = order && qs[b] <= qs[b + 1];
        CHECK(ordered == order);
        // the rows that the joining kernel looks up
        TileLine ln{};
        ln.imin = lo;
        ln.imax = hi;
        const int total = prefix_line(p, ln, qs[B]);
        line_share(total, p.ctas, 0, ln.per, ln.t, ln.t1);
        for (int t = 0; t < T; ++t) {
            int b = 0;
            for (int x = 0; x < B; ++x) b += qs[x + 1] <= t;
            if (b >= B) continue;
            const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, nullptr);
            if (s.n == 0 || t < s.q0 || t >= s.q0 + s.n) continue;
            for (int h = 0; h < 2; ++h) {
                const RowParts a = prefix_parts(PagedParts{}, ln.prefix_tiles, ln.per, 2, t * p.group, h, 0);
                const bool in = a.stride == 0 || a.within(2LL * p.ctas * kPagedTileRows);
                if (ordered && qs[B] <= T) CHECK(in);
                if (!in) ++seen_outside;
            }
        }
    }
    CHECK(seen_more > 100 && seen_outside > 100);      // the cases are among these
    printf("%d\n", bad);
    return bad != 0;
}
'''


def test_checks(nvcc, tmp_path):  # noqa: F811
    src, exe = tmp_path / "q_start.cu", tmp_path / "q_start"
    src.write_text(SOURCE)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "block_sparse_attention_fa_gb300", "csrc"),
                    "-gencode", "arch=compute_103a,code=sm_103a", "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@gpu
@pytest.mark.parametrize("shared", [0, 64])
@pytest.mark.parametrize("n,B", [(1, 6), (40, 6), (40, 40), (300, 300)])
def test_alternating_offsets(fa, n, B, shared):  # noqa: F811
    """Reported; rows behind the last offset and the next call are untouched by it."""
    bt = Batch([n, 1], [shared + n + 50, shared + 200], 2, 64, 16, shared=shared, pad=2)
    kc, vc, table, kv, qs = bt.device()
    q = torch.from_numpy(bt.queries(4)).cuda().to(torch.bfloat16)
    many = (kc, vc, table[:1].expand(B, -1).contiguous(), kv[:1].expand(B).contiguous(),
            torch.tensor([n * (b % 2) for b in range(B + 1)], dtype=torch.int32, device="cuda"))
    out = torch.full((bt.total, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((bt.total, 4), 3.0, device="cuda")
    fa.fwd_paged(q, *many, max_q_len=n, shared_len=shared, out=out, lse=lse)
    with pytest.raises(fa.FAError) as e:
        fa.default_workspace("cuda").check()
    assert e.value.status == fa.ERR_DEVICE_CHECK
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()
    got = fa.fwd_paged(q, kc, vc, table, kv, qs, max_q_len=n, shared_len=shared)
    fa.default_workspace("cuda").check()
    compare(got, reference(bt, bt.queries(4), "causal", 0, 0))
