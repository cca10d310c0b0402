// paged_line.cuh -- the line of tiles that the paged attention kernels split
// over their CTAs: which units there are, which part of which unit a CTA takes,
// and where the partials of a unit lie that several CTAs share.
//
// Everything here runs on the host too, where a test walks all CTAs' stretches
// against a plain enumeration of the units.
#pragma once

#include "paged.cuh"

namespace fa {

// CTA c's stretch of a line of `total` places over `ctas` CTAs: [t, t1), `per`
// places each (the last ones less, or none).
__host__ __device__ __forceinline__ void line_share(int total, int ctas, int c, int& per, int& t, int& t1) {
    per = imax((total + ctas - 1) / ctas, 1);
    const long long at = (long long)c * per, end = at + per;
    t = static_cast<int>(at < total ? at : total);
    t1 = static_cast<int>(end < total ? end : total);
}

// The last of n groups whose first place (Hkv times pre) is at or before t.
__host__ __device__ __forceinline__ int line_find(const int* pre, int n, int Hkv, int t) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (Hkv * pre[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// ---- units of up to 16 rows: a (sequence, kv head) each

// The part of one unit that falls into a CTA's stretch: tiles k0 .. k1 - 1 of
// the unit's list.  The loader finds it, ahead of the consumers, who read it
// from a slot in shared memory (with its rows of Q).
struct SmallSeg {
    int b, h, kv, n, q0;
    int tiles, k0, k1, count;      // count: CTAs that share the unit from here on
    Hull hull;
    __host__ __device__ __forceinline__ bool begins() const { return k0 == 0; }
    __host__ __device__ __forceinline__ bool ends() const { return k1 == tiles; }
};

// The line's index in shared memory has at most 1000 entries, so that two CTAs
// fit on an SM: one per sequence, or per 2, 4 sequences, within which the loader
// counts for itself (1024 sequences of 512 keys, 32 heads on 8 of 128 columns,
// pages of 16: 329 us, 470 with an entry for each and one CTA per SM).
constexpr int kLineEntries = 1000;
__host__ __device__ constexpr int group_shift(int B) { return B <= kLineEntries ? 0 : B <= 2 * kLineEntries ? 1 : 2; }
__host__ __device__ constexpr uint32_t groups_of(int B) { return (B + (1 << group_shift(B)) - 1) >> group_shift(B); }

// A CTA's stretch [t, t1) of the line of tiles.  Once every CTA has some tiles
// a unit counts as one more (`front` places before its first tile): its start
// and end cost about as much, and a CTA whose stretch is all short units would
// end long after the others (32 sequences of 64 keys before 32 of 8192: 166 us,
// 216 without).  With fewer tiles the units' parts are alike, and the work is
// best on the first CTAs (16 x 4 rows after a shared prefix of 5024 keys: 17.7
// us, 20.2 with).
constexpr int kManyTiles = 4;                    // per CTA
struct Line {
    const int* pre;                // [groups + 1] first tile of each group of 2^shift sequences
    int t, t1, per, front, shift;
    int g, b, base, len;           // group, sequence, its first tile (as in pre) and length
};

// The length of sequence b's place in the line, for one kv head.
template <int SHIFT>
__host__ __device__ __forceinline__ int seq_length(const PagedParams& p, int b, int front, uint32_t* ws) {
    const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, ws);
    return s.n == 0 ? 0 : make_hull(p.mask, s.kv - s.n, s.kv - 1, p.shared, s.kv, SHIFT).tiles + front;
}

// The same out of line, for the calls that only many sequences make (the others
// need not fetch their code).
template <int SHIFT>
__host__ __device__ __noinline__ int seq_length_again(const PagedParams& p, int b, int front) {
    return seq_length<SHIFT>(p, b, front, nullptr);
}

// The lengths of group g's 2^shift sequences together, without the fronts (which
// reports contradictions) and with them, `bare` being the first.
template <int SHIFT>
__host__ __device__ __forceinline__ int group_length(const PagedParams& p, int shift, int g, uint32_t* ws) {
    int sum = 0;
#pragma unroll 1
    for (int b = g << shift; b < imin((g + 1) << shift, p.c.B); ++b) sum += seq_length<SHIFT>(p, b, 0, ws);
    return sum;
}
template <int SHIFT>
__host__ __device__ __forceinline__ int group_length_front(const PagedParams& p, int shift, int g, int bare) {
    if (shift == 0) return bare + (bare > 0);
    int sum = 0;
#pragma unroll 1
    for (int b = g << shift; b < imin((g + 1) << shift, p.c.B); ++b) sum += seq_length_again<SHIFT>(p, b, 1);
    return sum;
}

template <int SHIFT>
__host__ __device__ __forceinline__ void open_group(const PagedParams& p, Line& ln) {
    ln.b = ln.g << ln.shift;
    ln.base = ln.pre[ln.g];
    ln.len = ln.shift ? seq_length_again<SHIFT>(p, ln.b, ln.front) : ln.pre[ln.g + 1] - ln.base;
}

template <int SHIFT>
__host__ __device__ __forceinline__ bool next_seg(const PagedParams& p, Line& ln, SmallSeg& s) {
    if (ln.t >= ln.t1) return false;
    while (p.c.Hkv * (ln.base + ln.len) <= ln.t) {
        if (p.c.Hkv * ln.pre[ln.g + 1] <= ln.t) {
            do ++ln.g; while (p.c.Hkv * ln.pre[ln.g + 1] <= ln.t);
            open_group<SHIFT>(p, ln);
        } else {
            ln.base += ln.len;
            ln.len = seq_length_again<SHIFT>(p, ++ln.b, ln.front);
        }
    }
    s.b = ln.b;
    const int length = ln.len, off = ln.t - p.c.Hkv * ln.base;
    s.tiles = length - ln.front;
    s.h = off / length;
    const int a = off - s.h * length, e = imin(length, a + (ln.t1 - ln.t));
    s.k0 = imax(a - ln.front, 0);
    s.k1 = imax(e - ln.front, 0);
    s.kv = load_i32(p.c.kv_len + ln.b);               // (checked when the line was made)
    s.q0 = load_i32(p.c.q_start + ln.b);
    s.n = load_i32(p.c.q_start + ln.b + 1) - s.q0;
    s.hull = make_hull(p.mask, s.kv - s.n, s.kv - 1, p.shared, s.kv, SHIFT);
    // the places of tile k0 and of the unit's last one
    const int here = ln.t + imax(ln.front - a, 0), last = here - s.k0 + s.tiles - 1;
    s.count = last / ln.per - here / ln.per + 1;
    ln.t += e - a;
    return s.k1 > 0;               // (0: the stretch ends before the unit's first tile)
}

// ---- units of 256 rows of a kv head

// What a unit's start and end cost (Q, the pipeline's first and last steps, O)
// beside its tiles, in tiles: its place in the line is that much longer.
// Without it a CTA whose stretch is all short units ends long after the others
// (prompts of 4 x 1024 tokens 92 us, one of 4096 tokens 210); with 2 those
// take 55 and 123, with 4 57 and 126, with 6 61 and 130, and chunks up to 8192
// keys 376 to 385 with any.  (The units of a shared prefix are all alike.)
constexpr int kUnitTiles = 2;

// The part of a unit in a CTA's stretch.
struct TileSeg {
    int b, h, row0, rows, q0, n, kv;
    int jlo, jhi, i0, i1;          // keys of this kernel's part, positions of the unit's rows
    int tiles, k0, k1, t;          // t: the place of tile k0 in the line
    Hull hull;
    __host__ __device__ __forceinline__ bool begins() const { return k0 == 0; }
    __host__ __device__ __forceinline__ bool ends() const { return k1 == tiles; }
    // CTAs that share the unit, from this part on (per: tiles of a CTA)
    __host__ __device__ __forceinline__ int count(int per) const { return (t - k0 + tiles - 1) / per - t / per + 1; }
};

struct TileLine {
    const int *pre, *kv, *q0;           // [B + 1] first tile, [B] length, [B + 1] first row
    int t, t1, per, b, rt, start;       // start: where unit group (b, rt), its Hkv units, begins in the line
    int prefix_tiles, prefix_rows, imin, imax;
};

// The positions of rows 256 rt .. of a sequence of n new tokens.
__host__ __device__ __forceinline__ void unit_rows(const FastDiv& by_group, int n, int kv, int rt, int& i0, int& i1) {
    const int r0 = rt * kPagedTileRows, r1 = imin(r0 + kPagedTileRows, n * static_cast<int>(by_group.d)) - 1;
    i0 = kv - n + quotient(r0, by_group);
    i1 = kv - n + quotient(r1, by_group);
}

// The length of one such unit's place in the line.
__host__ __device__ __forceinline__ int unit_length(const PagedParams& p, int n, int kv, int rt) {
    int i0, i1;
    unit_rows(p.by_group, n, kv, rt, i0, i1);
    return make_hull(p.mask, i0, i1, p.shared, kv, 7).tiles + kUnitTiles;
}

// A shared prefix's line: the rows up to q_end, the batch's tokens, of every kv
// head against the prefix, for positions ln.imin .. ln.imax (none, if these are
// the other way round).  Returns its length.
__host__ __device__ __forceinline__ int prefix_line(const PagedParams& p, TileLine& ln, int q_end) {
    ln.prefix_rows = ln.imin <= ln.imax ? imin(imax(q_end, 0), p.c.total_q) * p.group : 0;
    ln.prefix_tiles = ln.prefix_rows ? make_hull(p.mask, ln.imin, ln.imax, 0, p.shared, 7).tiles : 1;
    return (ln.prefix_rows + kPagedTileRows - 1) / kPagedTileRows * p.c.Hkv * ln.prefix_tiles;
}

__host__ __device__ __forceinline__ bool next_seg(const PagedParams& p, TileLine& ln, TileSeg& s) {
    if (ln.t >= ln.t1) return false;
    int off;
    if (p.prefix) {
        s.tiles = ln.prefix_tiles;
        const int group_tiles = p.c.Hkv * s.tiles, rt = ln.t / group_tiles;
        off = ln.t - rt * group_tiles;
        s.b = s.q0 = s.n = s.kv = 0;
        s.row0 = rt * kPagedTileRows;
        s.rows = imin(kPagedTileRows, ln.prefix_rows - s.row0);
        s.jlo = 0;
        s.jhi = p.shared;
        s.i0 = ln.imin;
        s.i1 = ln.imax;
        s.hull = make_hull(p.mask, s.i0, s.i1, s.jlo, s.jhi, 7);
    } else {
        while (p.c.Hkv * ln.pre[ln.b + 1] <= ln.t) {
            ++ln.b;
            ln.rt = 0;
            ln.start = p.c.Hkv * ln.pre[ln.b];
        }
        s.b = ln.b;
        s.q0 = ln.q0[s.b];
        s.n = ln.q0[s.b + 1] - s.q0;
        s.kv = ln.kv[s.b];
        s.jlo = p.shared;
        s.jhi = s.kv;
        for (;;) {
            unit_rows(p.by_group, s.n, s.kv, ln.rt, s.i0, s.i1);
            s.hull = make_hull(p.mask, s.i0, s.i1, s.jlo, s.jhi, 7);
            const int next = ln.start + p.c.Hkv * (s.hull.tiles + kUnitTiles);
            if (ln.t < next) break;
            ln.start = next;
            ++ln.rt;
        }
        s.tiles = s.hull.tiles;
        off = ln.t - ln.start;
        s.row0 = ln.rt * kPagedTileRows;
        s.rows = imin(kPagedTileRows, s.n * p.group - s.row0);
    }
    const int front = p.prefix ? 0 : kUnitTiles, length = s.tiles + front;
    s.h = off / length;
    const int a = off - s.h * length, b = imin(length, a + (ln.t1 - ln.t));
    s.k0 = imax(a - front, 0);
    s.k1 = imax(b - front, 0);
    s.t = ln.t + imax(front - a, 0);
    ln.t += b - a;
    return s.k1 > 0;               // (0: the stretch ends before the unit's first tile)
}

// ---- partials

// Row r of the unit that starts in CTA `cta` and runs on over `count` CTAs.
__host__ __device__ __forceinline__ RowParts unit_parts(const PagedParts& parts, int cta, int count, int rows_per_unit, int r) {
    return {parts.slot_o, parts.slot_ml, (2LL * cta + 1) * rows_per_unit + r, count, rows_per_unit};
}

// Row R = token x group + query head of kv head h in the line of a shared prefix
// (`tiles` per unit, `per` per CTA); `row` is its place among all rows.
__host__ __device__ __forceinline__ RowParts prefix_parts(const PagedParts& parts, int tiles, int per, int Hkv, int R, int h,
                                                          long long row) {
    const int rt = R / kPagedTileRows, first = (rt * Hkv + h) * tiles, ca = first / per, cb = (first + tiles - 1) / per;
    if (ca == cb) return {parts.row_o, parts.row_ml, row, 1, 0};
    return unit_parts(parts, ca, cb - ca + 1, kPagedTileRows, R - rt * kPagedTileRows);
}

}  // namespace fa
