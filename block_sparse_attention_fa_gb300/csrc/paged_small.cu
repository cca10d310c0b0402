// paged_small.cu -- attention over the paged cache for a few rows per
// (sequence, kv head), and the kernels that join split units.
//
// The definition is fa_fwd's, for rows at position i of their sequence and
// keys on pages.  A unit of work is a (sequence, kv head): its n x Hq / Hkv
// rows (at most 16) against the keys that some row sees.  With one row per
// query head there is nothing to reuse: every K and V byte is read once and
// HBM bounds the kernel.
//
// Split.  The tiles of all units stand in one line, unit after unit; CTA c of
// the grid (two per SM) takes an equal stretch of it, whatever the sequences'
// lengths.  Only the first and the last unit of a stretch can
// be shared with a neighbour; those leave partials (unnormalised O, running
// max and sum) in two slots per CTA, and a second kernel joins them in the
// order of the keys, so that results do not depend on timing.  The loader runs
// over the whole stretch without a stop at unit boundaries.  Every CTA finds
// its stretch by itself: the lengths are on the device, and a prefix sum over
// the sequences costs about a microsecond.
//
// A tile is 32 KB of K and V (128 keys of 64 columns, 64 of 128), three of them
// are in flight per CTA, and two CTAs share an SM: what one CTA waits for (the
// start, the barriers of a tile, the change from one unit to the next) the
// other's work covers.  One CTA of three 64 KB stages per SM read as much at
// once, but its tiles of 64 columns took 1.05 us instead of the 0.73 us that
// HBM needs: 121 us instead of 89 for 64 sequences of 4096 keys, 8 kv heads of
// 64 columns (537 MB; at 128 columns the two are even).
//
// CTA: 8 consumer warps and a loader warp.  The loader's lanes stand for the
// tile's pages: each reads its page's id ahead of time and issues the page's
// TMA boxes into a ring of stages.  Pages without a visible key are neither
// looked up nor read.  Consumer warp w computes S for an eighth of the tile's
// keys (mma.sync m16n8k16; 16 rows are too few for a tcgen05 tile, and
// the tensor pipe is not the bound), the warps exchange their row maxima and
// then P (bf16) through shared memory, and warp w accumulates columns
// w D / 8 .. of O over all the tile's keys: no warp holds a second copy of O, so a
// unit's end needs no merge and costs one barrier.
//
// V rows of keys that no row of the unit sees (past the end of the sequence,
// before the window, on pages that were not read) are cleared in shared
// memory before the product: their P is 0, but 0 x NaN is not.
#include "paged_small.cuh"

namespace fa {
namespace {

// Joins the partials of rows, the parts of `a` and then those of `b`:
//   M = max m_k, L = sum 2^(m_k - M) l_k, O = sum 2^(m_k - M) O_k / L.
// Eight lanes to a row, four rows to a warp.  What it costs is the loads'
// latency, so many are in flight at once: a lane holds the (m, l) of every
// eighth part for the weights, and reads its 4 x D / 32 columns of several
// parts at a time.  SHARE warps, the block, take the parts of the same four
// rows in turn and add up through shared memory (single tokens and shared
// prefixes, where a row has tens of parts); 1: each of four warps has rows of
// its own.  With few rows eight warps share (one token, 520 keys, 8 blocks:
// the call 8.6 us, with four 9.4; 64 rows after a prefix of 5024 keys, 188
// blocks: 17.5 and 18.9); with many, four that need fewer registers together,
// for then all blocks run at once (64 chats after a prefix of 16384 keys, 512
// blocks: 55.5 us, with eight 58.5).  Summing is in a
// fixed order either way.
template <int SHARE>
constexpr int kJoinWarps = SHARE == 1 ? 4 : SHARE;
template <int D, int SHARE>
__device__ __forceinline__ void join_rows(const PagedParams& p, const RowParts& a, const RowParts& b, long long row,
                                          bool valid, float4* sums) {
    constexpr int kC = D / 32;                     // float4 columns per lane, 32 apart
    constexpr bool SPLIT = SHARE > 1;
    constexpr int kHold = SPLIT ? SHARE / 2 : 1;   // weights per lane: 8 kHold parts per pass
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7;
    const int n = valid ? a.count + b.count : 0;
    auto ml_of = [&](int k) {
        if (k >= n) return make_float2(-CUDART_INF_F, 0.f);
        return k < a.count ? __ldcg(a.ml + a.at(k)) : __ldcg(b.ml + b.at(k - a.count));
    };
    const int longest = __reduce_max_sync(0xffffffffu, n);
    float2 ml[kHold];
#pragma unroll
    for (int t = 0; t < kHold; ++t) ml[t] = ml_of(8 * t + sub);
    float m = ml[0].x;
#pragma unroll
    for (int t = 1; t < kHold; ++t) m = fmaxf(m, ml[t].x);
    for (int k0 = 8 * kHold; k0 < longest; k0 += 8) m = fmaxf(m, ml_of(k0 + sub).x);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == -CUDART_INF_F ? 0.f : m;
    float l = 0.f;
    float4 o[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < longest; k0 += 8 * kHold) {
        float w[kHold];
#pragma unroll
        for (int t = 0; t < kHold; ++t) {
            if (k0) ml[t] = ml_of(k0 + 8 * t + sub);
            w[t] = ml[t].y == 0.f ? 0.f : ex2_approx(ml[t].x - ref);   // 0: the part has no visible key for this row
            l += ml[t].y * w[t];
        }
        // this warp's parts of the pass
#pragma unroll
        for (int e = 0; e < 8 * kHold; e += SHARE) {
            const int k = k0 + e + (SPLIT ? warp : 0);
            const float we = __shfl_sync(0xffffffffu, w[e >> 3], (lane & 24) + (e & 7) + (SPLIT ? warp : 0));
            if (k >= n) continue;
            const float4* src = reinterpret_cast<const float4*>(
                k < a.count ? a.o + a.at(k) * D : b.o + b.at(k - a.count) * D) + sub;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const float4 v = __ldcg(src + 8 * c);
                o[c].x = fmaf(we, v.x, o[c].x);
                o[c].y = fmaf(we, v.y, o[c].y);
                o[c].z = fmaf(we, v.z, o[c].z);
                o[c].w = fmaf(we, v.w, o[c].w);
            }
        }
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (SPLIT) {
        if (warp > 0) {
#pragma unroll
            for (int c = 0; c < kC; ++c) sums[((warp - 1) * kC + c) * 32 + lane] = o[c];
        }
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 0; w < SHARE - 1; ++w) {
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const float4 v = sums[(w * kC + c) * 32 + lane];
                o[c].x += v.x;
                o[c].y += v.y;
                o[c].z += v.z;
                o[c].w += v.w;
            }
        }
    }
    if (!valid) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
        const long long at = row * D + 32 * c + 4 * sub;
        if (p.flags & FA_OUT_FP32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) =
                make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv);
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + at) =
                make_uint2(pack_bf16x2(o[c].x * inv, o[c].y * inv), pack_bf16x2(o[c].z * inv, o[c].w * inv));
    }
    if (sub == 0) p.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kPagedLn2;
}

// Without a shared prefix: block (c, y) joins rows of the unit that starts in
// CTA c of the attention kernel and runs on into the next ones.
template <int D, int SHARE>
__global__ void __launch_bounds__(32 * kJoinWarps<SHARE>) paged_join_units_kernel(const PagedParams p, int rows_per_unit) {
    __shared__ float4 sums[SHARE > 1 ? (SHARE - 1) * (D / 32) * 32 : 1];
    pdl_launch_next();
    pdl_wait_previous();
    const PagedMeta t = p.meta[blockIdx.x];
    const int r = (SHARE > 1 ? blockIdx.y : blockIdx.y * kJoinWarps<SHARE> + (threadIdx.x >> 5)) * 4 + ((threadIdx.x & 31) >> 3);
    if (t.count == 0 || (r & ~3) >= t.rows) return;        // (uniform: four rows to a warp, and to a block that shares them)
    const bool valid = r < t.rows;
    const RowParts a = unit_parts(p.parts, blockIdx.x, t.count, rows_per_unit, r);
    const RowParts none{nullptr, nullptr, 0, 0, 0};
    if (!a.within(2LL * gridDim.x * rows_per_unit)) return;     // (the same for all rows of a unit)
    const int R = t.row0 + r, tok = quotient(R, p.by_group);
    join_rows<D, SHARE>(p, a, none, (long long)(t.q0 + tok) * p.Hq + t.h * p.group + R - tok * p.group, valid, sums);
}

// With a shared prefix: block (t, h, y) joins four rows of token t and kv head
// h, the prefix's partials first, then those of the sequence's own keys.
template <int D, int SHARE>
__global__ void __launch_bounds__(32 * SHARE) paged_join_rows_kernel(const PagedJoin j) {
    constexpr int kThreads = 32 * SHARE;
    __shared__ float4 sums[(SHARE - 1) * (D / 32) * 32];
    const PagedParams& p = j.own;
    pdl_launch_next();
    pdl_wait_previous();
    const int t = blockIdx.x, h = blockIdx.y;
    const int2 pre = *reinterpret_cast<const int2*>(p.hdr);
    if ((blockIdx.x | blockIdx.y | blockIdx.z | threadIdx.x) == 0) *prefix_mark(p) = 0;
    const int gq = blockIdx.z * 4 + ((threadIdx.x & 31) >> 3);
    const bool valid = gq < p.group;
    const long long row = (long long)t * p.Hq + h * p.group + min(gq, p.group - 1);
    const int2 d = __ldcg(p.rowdesc + row);        // (what it says of a row without a unit is not used)
    int b = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += kThreads) {
        const int x = b0 + threadIdx.x;
        b += __syncthreads_count(x < p.c.B && __ldg(p.c.q_start + min(x, p.c.B - 1) + 1) <= t);
    }
    if (b >= p.c.B) return;
    const SeqInfo s = seq_info(p.c, b, p.max_q, p.shared, nullptr);
    if (s.n == 0 || t < s.q0 || t >= s.q0 + s.n) return;
    RowParts a = prefix_parts(j.pre, pre.x, pre.y, p.c.Hkv, t * p.group + min(gq, p.group - 1), h, row);
    RowParts own{p.parts.slot_o, p.parts.slot_ml, d.x, d.y, j.own_rows};
    if (d.x < 0) own = RowParts{p.parts.row_o, p.parts.row_ml, row, 1, 0};
    // (a q_start that decreases can name rows past the prefix's line)
    if (a.stride > 0 && !a.within(2LL * j.pre_ctas * kPagedTileRows)) a.count = 0;
    // (a CTA whose wait ran out leaves its rows' places as the scratch held them)
    if (d.x >= 0 && !own.within(2LL * p.ctas * j.own_rows)) own.count = 0;
    join_rows<D, SHARE>(p, a, own, row, valid, sums);
}

}  // namespace

cudaError_t launch_paged_small(const PagedParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
    return p.D == 64 ? launch_small_d<64, false>(p, tk, tv, s) : launch_small_d<128, false>(p, tk, tv, s);
}

namespace {

// Eight warps to four rows while that is at most one block per SM and a half.
bool few_joins(long long blocks) { return 2 * blocks <= 3 * device_sm_count(); }

template <int D>
cudaError_t launch_join_units(const PagedParams& p, int rows_per_unit, cudaStream_t s) {
    // the blocks that find something to join: at most the units', or one per CTA
    const long long rows = std::min((long long)p.max_q * p.group, (long long)rows_per_unit);
    const long long units = ((long long)p.c.B + (long long)p.c.total_q * p.group / rows_per_unit) * p.c.Hkv;
    const dim3 grid(p.ctas, (unsigned)((rows + 3) / 4));
    if (few_joins(std::min<long long>(units, p.ctas) * grid.y))
        return paged_launch(paged_join_units_kernel<D, 8>, grid, 32 * 8, 0, true, s, p, rows_per_unit);
    if (rows_per_unit == kPagedSmallRows)
        return paged_launch(paged_join_units_kernel<D, 4>, grid, 32 * 4, 0, true, s, p, rows_per_unit);
    return paged_launch(paged_join_units_kernel<D, 1>, dim3(p.ctas, (grid.y + kJoinWarps<1> - 1) / kJoinWarps<1>),
                        32 * kJoinWarps<1>, 0, true, s, p, rows_per_unit);
}

template <int D>
cudaError_t launch_join_rows(const PagedJoin& j, cudaStream_t s) {
    const dim3 grid(j.own.c.total_q, j.own.c.Hkv, (j.own.group + 3) / 4);
    return few_joins((long long)grid.x * grid.y * grid.z)
               ? paged_launch(paged_join_rows_kernel<D, 8>, grid, 32 * 8, 0, true, s, j)
               : paged_launch(paged_join_rows_kernel<D, 4>, grid, 32 * 4, 0, true, s, j);
}

}  // namespace

cudaError_t launch_paged_join_units(const PagedParams& p, int rows_per_unit, cudaStream_t s) {
    return p.D == 64 ? launch_join_units<64>(p, rows_per_unit, s) : launch_join_units<128>(p, rows_per_unit, s);
}

cudaError_t launch_paged_join_rows(const PagedJoin& p, cudaStream_t s) {
    return p.own.D == 64 ? launch_join_rows<64>(p, s) : launch_join_rows<128>(p, s);
}

}  // namespace fa
