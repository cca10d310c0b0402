// paged_eight_scaled.cu -- attention over a cache held in 8 bits (e4m3 codes, a
// scale for each page and kv head) for up to 8 rows per (sequence, kv head).
//
// The split of the work and the partials are paged_small.cu's: the tiles (128
// keys) of all units stand in one line, every CTA (two per SM) takes an equal
// stretch, and a second kernel joins the units that two CTAs share.  With half
// the bytes per key what a key costs beside its bytes counts twice, so the
// consumers work differently.
//
// Each of the 4 consumer warps keeps 32 keys of a tile to itself, from S to
// P V, with a running maximum, a sum and all columns of O of its own: no barrier
// between the warps and no exchange through shared memory within a unit; at its
// end the four are added up.  The products are transposed, S^T = K Q^T and
// O^T = V^T P^T (mma.sync m16n8k16: 16 keys, then 16 columns, by 8 rows of Q), so
// that 8 rows fill them.
//   - K: ldmatrix gives a thread 32 bits of a key's row: four adjacent columns,
//     where the product wants two and two, 8 apart.  The columns of 16 go to the
//     product in that order, Q's with them.
//   - P^T is S^T's result with keys and rows exchanged: movmatrix.
//   - V: ldmatrix.trans gives two keys of two adjacent columns; the even columns
//     are the product's rows 0-7, the odd ones 8-15.
// A code is converted once, to f16, which holds it exactly; so does it a row of Q
// scaled by a power of two, and P is rounded to f16's 11 bits.  k's scale is applied
// to S in fp32.  v's is part of P's exponent: with x the score in base 2,
// lv = log2(v's scale), one for 16 keys (of a page), and M a reference below the
// largest x + lv (kPHead),
//     P = 2^(x + lv - M),   l = sum of P / (v's scale),
// so that O accumulates in the products, P's roundings are relative to the largest
// share that any key has in O, and O / l and M + log2 l are what they are without
// scales.  M is raised (and O and l rescaled) only when an x + lv is past it by kPTop,
// which one vote of the warp tells.
//
// DRAM bounds long contexts; ragged batches on pages of 16 keys the chain of a tile
// in each warp, some 1800 cycles of 2500, and the two loader warps' issue
// (paged_codes.cuh), evenly.  8 sequences of 32768 tokens, 8 kv heads of 128
// columns: 89.5 us, 79.1 at the copy rate (bf16 cache: 163).  128 of up to 4096, 8
// kv heads of 64 columns, pages of 16: 75.5 us, 41.0 at the copy rate.  One of 520
// tokens: 9.6, most of it the first run through the code.
//
// V rows of keys that no row of the unit sees are cleared in shared memory before
// the product: their P is 0, but 0 x NaN is not.
#include "paged_codes.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;                        // consumers, 32 keys each; warps 4 and 5 load
constexpr int kRows = 8;
static_assert(kKeys == 32 * kWarps, "32 keys to a warp");

// Beside the ring and the queues: two warps' O, every warp's [rows] maximum and sum.
template <int D>
struct Eight : CodeLayout<D, kWarps, 2, kRows, 8u * kRows * D + 8u * kWarps * kRows> {
    static constexpr uint32_t kMerge = Eight::kExtra, kMl = kMerge + 8u * kRows * D;
};

// An 8 x 8 matrix of 16-bit elements, two of a row to a thread, transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// c += a b, one m16n8k16 tile of f16, fp32 sums
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same barrier with a vote: whether `ok` holds in every thread.
__device__ __forceinline__ bool consumers_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(ok))
        : "memory");
    return r != 0;
}

// Two CTAs per SM, at no more registers than 128: an SM's quarters hold 16384
// each, and four warps where each of the CTAs has put two there.  (Three CTAs of
// five warps, of which that left room for only by chance: 66 us or 110 for the
// chats, depending on what ran before.)
template <int D, int SCORE>
__global__ void __maxnreg__(128)
paged_eight_scaled_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const PagedScaledParams p) {
    using L = Eight<D>;
    constexpr int ST = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
    SmallSeg* const seg_s = reinterpret_cast<SmallSeg*>(smem + L::kSeg);
    volatile int* const info_s = reinterpret_cast<volatile int*>(smem + L::kInfo);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    if (threadIdx.x == 0) {
        L::init(sbase);
        *abort_flag = 0;
        mbar_fence_init();
    }
    // (a shared prefix's kernel is no input of this one: it is waited for at the end)
    if (p.join_rows)
        wait_before_prefix(p);
    else
        pdl_wait_previous();
    pdl_launch_next();
    const Line line = code_line<L>(p, smem, cta, warp >= kWarps);
    const WaitCtl wc{abort_flag, p.ws, p.timeout_ns};

    if (warp >= kWarps) {
        if (warp == kWarps)
            load_codes<L, kLoadK>(p, tmK, tmV, line, smem, sbase, wc, lane);
        else
            load_codes<L, kLoadV>(p, tmK, tmV, line, smem, sbase, wc, lane);
        if (p.join_rows) pdl_wait_previous();
        return;
    }

    // --------------------------------------------------------------- consumers
    const int gr = lane >> 2, tq = lane & 3, mi = lane >> 3, l8 = lane & 7;
    float2* const ml_s = reinterpret_cast<float2*>(smem + L::kMl);
    // score_mod, to base 2
    const float sl2 = p.scale * kPagedLog2e;
    const SoftCap cap = soft_cap(p.score.softcap, SCORE == FA_SCORE_SOFTCAP ? p.scale : 1.f);
    const int by_page = min(p.c.page_shift, kShift);       // 2^by_page keys of a tile share a page
    constexpr int kChunks = D / 16;                        // 16 columns each
    int g = 0;
    bool ok = true;
    PagedMeta meta{};
    for (int nu = 0;; ++nu) {
        const bool q_here = mbar_wait_warp(L::q_full(sbase, nu), (nu >> 1) & 1, wc, S_PC_Q);
        // (the vote keeps the warps together where a wait has run out)
        if (!consumers_all(q_here)) { ok = false; break; }
        const SmallSeg& s = seg_s[nu % kSegs];
        if (s.b < 0) break;
        const int rows = s.n * p.group, i0 = s.kv - s.n;
        // Q's fragments in f16: a row times a power of two, so that its largest
        // element is 2^14 .. 2^15 and those below f16's normal numbers are 2^28
        // times smaller.  (Rows past the unit's are 0.)
        uint32_t qb[kChunks][2];
        float unscale[2], slope[2];
        int tok[2];
        const int r = gr;
        const uint8_t* const q_row = smem + L::kQ + ((nu & 1) * L::kRows + r) * L::kQRow + 8 * tq;
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const uint2 w = r < rows ? *reinterpret_cast<const uint2*>(q_row + 32 * c) : make_uint2(0u, 0u);
            qb[c][0] = w.x;
            qb[c][1] = w.y;
            top = fmaxf(top, fmaxf(fmaxf(fabsf(bf_low(w.x)), fabsf(bf_high(w.x))),
                                   fmaxf(fabsf(bf_low(w.y)), fabsf(bf_high(w.y)))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int at = max(__float_as_int(top) >> 23, 15);
        const float up = __int_as_float((268 - at) << 23), down = __int_as_float((at - 14) << 23);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                qb[c][e] = pack_f16x2(bf_low(qb[c][e]) * up, bf_high(qb[c][e]) * up);
        }
        // this thread's columns of S^T: rows 2 tq and the next one
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            unscale[e] = __shfl_sync(0xffffffffu, down, 4 * (2 * tq + e));
            const int row = min(2 * tq + e, rows - 1);
            tok[e] = quotient(row, p.by_group);
            slope[e] = 0.f;
            if (SCORE == FA_SCORE_ALIBI || SCORE == FA_SCORE_ALIBI_SOFTCAP)
                slope[e] = p.score.slopes[s.h * p.group + row - tok[e] * p.group] *
                               (SCORE == FA_SCORE_ALIBI ? kPagedLog2e : 1.f);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(L::q_empty(sbase, nu));
        float m[2], l[2], o[kChunks][4];
        m[0] = m[1] = -CUDART_INF_F;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;

        const int tiles = s.k1 - s.k0;
        for (int k = 0; k < tiles; ++k, ++g) {
            const int st = g % ST;
            const uint32_t kbase = sbase + st * L::kStage, vbase = kbase + L::kTile;
            if (!mbar_wait_warp(L::full(sbase, st), (g / ST) & 1, wc, S_PC_FULL)) { ok = false; break; }
            const int info = info_s[st], j0 = (info >> 2) * kKeys + 32 * warp;
            const float* const sc = reinterpret_cast<const float*>(smem + L::kScale + st * L::kScaleStage);
            const int page[2] = {32 * warp >> by_page, (32 * warp + 16) >> by_page};
            const float lv[2] = {sc[2 * (kKeys / 16) + page[0]], sc[2 * (kKeys / 16) + page[1]]};
            const bool open = (info & kTileOpen) != 0;
            bool cleared = false;
            // S^T, 16 keys at a time
            float x[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t kf[4], a[4], b[4];
                    ldsm4(kbase + swz8<D>(32 * warp + 16 * u + 8 * (mi & 1) + l8, c + (mi >> 1)), kf);
                    codes_to_f16(kf[0], a[0], a[2]);
                    codes_to_f16(kf[1], a[1], a[3]);
                    codes_to_f16(kf[2], b[0], b[2]);
                    codes_to_f16(kf[3], b[1], b[3]);
                    mma_f16(x[u], a, qb[c]);
                    mma_f16(x[u], b, qb[c + 1]);
                }
            }
            if (info & kTileClear) {
                // V rows that no row of the unit sees
                cleared = true;
                const uint32_t live = __ballot_sync(0xffffffffu, s.hull.live(j0 + lane));
#pragma unroll
                for (int e = 0; e < kChunks; ++e) {
                    const int r = (32 * e + lane) / kChunks;
                    if (!((live >> r) & 1u))
                        *reinterpret_cast<uint4*>(smem + st * L::kStage + L::kTile + swz8<D>(32 * warp + r, lane % kChunks)) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            // x: the score in base 2, and log2 of v's scale
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float k_scale = sc[page[u]] * (SCORE == FA_SCORE_NONE || SCORE == FA_SCORE_REL_BIAS ? sl2 : 1.f);
                const float f[2] = {unscale[0] * k_scale, unscale[1] * k_scale};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int e = c & 1, j = j0 + 16 * u + gr + 8 * (c >> 1), i = i0 + tok[e];
                    float v = SCORE == FA_SCORE_NONE ? fmaf(x[u][c], f[e], lv[u]) : x[u][c] * f[e];
                    const float far = fabsf(static_cast<float>(i - j));
                    if (SCORE == FA_SCORE_SOFTCAP) v = softcap_one(v, cap);
                    if (SCORE == FA_SCORE_ALIBI) v = fmaf(-slope[e], far, v * sl2);
                    if (SCORE == FA_SCORE_ALIBI_SOFTCAP) v = softcap_one(fmaf(-slope[e], far, v * p.scale), cap);
                    if (SCORE == FA_SCORE_REL_BIAS) {
                        const int R = p.score.rel_max, d = min(max(i - j, -R), R);
                        const int hq = s.h * p.group + min(2 * tq + e, rows - 1) - tok[e] * p.group;
                        v = fmaf(p.score.rel_bias[(size_t)hq * (2 * R + 1) + d + R], kPagedLog2e, v);
                    }
                    if (!open && !paged_visible(p.mask, i, j, p.shared, s.kv)) v = -CUDART_INF_F;
                    x[u][c] = SCORE == FA_SCORE_NONE ? v : v + lv[u];
                }
            }
            const float top[2] = {fmaxf(fmax3(x[0][0], x[0][2], x[1][0]), x[1][2]), fmaxf(fmax3(x[0][1], x[0][3], x[1][1]), x[1][3])};
            if (__any_sync(0xffffffffu, top[0] > m[0] + kPTop || top[1] > m[1] + kPTop)) {
                float alpha[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float to = top[e];
                    to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 4));
                    to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 8));
                    to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 16));
                    to = fmaxf(to - kPHead, m[e]);
                    alpha[e] = to == m[e] ? 1.f : ex2_approx(m[e] - to);
                    l[e] = alpha[e] == 0.f ? times_2_to(l[e], m[e] - to) : l[e] * alpha[e];
                    m[e] = to;
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    o[c][0] *= alpha[0];
                    o[c][1] *= alpha[1];
                    o[c][2] *= alpha[0];
                    o[c][3] *= alpha[1];
                }
            }
            // P^T, rows of Q along the threads
            uint32_t pb[2][2];
            const float ref[2] = {m[0] == -CUDART_INF_F ? 0.f : m[0], m[1] == -CUDART_INF_F ? 0.f : m[1]};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) w[c] = ex2_approx(x[u][c] - ref[c & 1]);
                const float iv = sc[3 * (kKeys / 16) + page[u]];
                l[0] = fmaf(w[0] + w[2], iv, l[0]);
                l[1] = fmaf(w[1] + w[3], iv, l[1]);
                pb[u][0] = transpose_8x8(pack_p(w[0], w[1]));
                pb[u][1] = transpose_8x8(pack_p(w[2], w[3]));
            }
            // O^T += V^T P^T, 16 columns at a time
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t vf[4];
                    ldsm4_t(vbase + swz8<D>(32 * warp + 16 * u + 8 * (mi & 1) + l8, c + (mi >> 1)), vf);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t a[4];
                        codes_to_f16(__byte_perm(vf[2 * e], 0u, 0x3120), a[0], a[1]);
                        codes_to_f16(__byte_perm(vf[2 * e + 1], 0u, 0x3120), a[2], a[3]);
                        mma_f16(o[c + e], a, pb[u]);
                    }
                }
            }
            if (cleared) fence_async_shared();     // the next copy into this stage comes after the clearing
            __syncwarp();
            if (lane == 0) mbar_arrive(L::empty(sbase, st));
        }

        // the unit's end in this CTA: the warps' maxima and sums, then their O
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[e];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            if (gr == 0) ml_s[warp * L::kRows + 2 * tq + e] = make_float2(m[e], sum);
        }
        if (!consumers_all(ok)) { ok = false; break; }
        float sum[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float top = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml_s[w * L::kRows + 2 * tq + e].x);
            const float ref = top == -CUDART_INF_F ? 0.f : top;
            sum[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 t = ml_s[w * L::kRows + 2 * tq + e];
                sum[e] += times_2_to(t.y, t.x - ref);
            }
            const float f = ex2_approx(m[e] - ref);
            m[e] = top;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                o[c][e] *= f;
                o[c][2 + e] *= f;
            }
        }
        // O of warps 2, 3 to 0, 1, and of 1 to 0
#pragma unroll
        for (int half = kWarps / 2; half > 0; half >>= 1) {
            float4* const at = reinterpret_cast<float4*>(smem + L::kMerge) + (warp % half) * kChunks * 32 + lane;
            if (warp >= half && warp < 2 * half) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c) at[32 * c] = make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
            }
            consumers_sync();
            if (warp < half) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const float4 t = at[32 * c];
                    o[c][0] += t.x;
                    o[c][1] += t.y;
                    o[c][2] += t.z;
                    o[c][3] += t.w;
                }
            }
            if (half > 1) consumers_sync();
        }
        if (warp == 0) {
            const bool whole = s.begins() && s.ends();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * tq + e;
                if (r >= rows) continue;
                const int at = quotient(r, p.by_group);
                const long long row = (long long)(s.q0 + at) * p.Hq + s.h * p.group + r - at * p.group;
                const bool last = whole && !p.join_rows;
                const long long slot = whole ? row : (2LL * cta + (s.begins() ? 1 : 0)) * kPagedSmallRows + r;
                const float inv = !last ? even_out(m[e], sum[e]) : sum[e] == 0.f ? 0.f : 1.f / sum[e];      // a NaN stays one
                if (last && !(p.flags & FA_OUT_FP32)) {
                    uint16_t* const dst = static_cast<uint16_t*>(p.o) + row * D + 2 * gr;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        *reinterpret_cast<uint32_t*>(dst + 16 * c) = pack_bf16x2(o[c][e] * inv, o[c][2 + e] * inv);
                } else {
                    float* const dst = (last ? static_cast<float*>(p.o) : whole ? p.parts.row_o : p.parts.slot_o) +
                                       slot * D + 2 * gr;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        *reinterpret_cast<float2*>(dst + 16 * c) = make_float2(o[c][e] * inv, o[c][2 + e] * inv);
                }
                if (gr != 0) continue;
                if (last) {
                    p.lse[row] = sum[e] == 0.f ? -CUDART_INF_F : (m[e] + log2f(sum[e])) * kPagedLn2;
                } else {
                    (whole ? p.parts.row_ml : p.parts.slot_ml)[slot] = make_float2(m[e], sum[e]);
                    if (p.join_rows && s.begins())
                        p.rowdesc[row] = whole ? make_int2(-1, 1)
                                               : make_int2((2 * cta + 1) * kPagedSmallRows + r, s.count);
                }
            }
        }
        if (s.begins() && !s.ends()) {
            meta.count = s.count;
            meta.q0 = s.q0;
            meta.rows = rows;
            meta.h = s.h;
        }
    }
    if (!p.join_rows && threadIdx.x == 0) p.meta[cta] = ok ? meta : PagedMeta{};
    if (p.join_rows) pdl_wait_previous();
}

template <int D, int SCORE>
cudaError_t launch_one(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    auto kern = paged_eight_scaled_kernel<D, SCORE>;
    using L = Eight<D>;
    constexpr size_t most = L::bytes(kCodeEntries);
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return paged_launch(kern, dim3(p.ctas), L::kThreads, L::bytes(p.c.B), true, s, tk, tv, p);
}

template <int D>
cudaError_t launch_score(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    switch (p.score.kind) {
        case FA_SCORE_SOFTCAP: return launch_one<D, FA_SCORE_SOFTCAP>(p, tk, tv, s);
        case FA_SCORE_ALIBI: return launch_one<D, FA_SCORE_ALIBI>(p, tk, tv, s);
        case FA_SCORE_REL_BIAS: return launch_one<D, FA_SCORE_REL_BIAS>(p, tk, tv, s);
        case FA_SCORE_ALIBI_SOFTCAP: return launch_one<D, FA_SCORE_ALIBI_SOFTCAP>(p, tk, tv, s);
        default: return launch_one<D, FA_SCORE_NONE>(p, tk, tv, s);
    }
}

}  // namespace

cudaError_t launch_paged_eight_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s) {
    return p.D == 64 ? launch_score<64>(p, tk, tv, s) : launch_score<128>(p, tk, tv, s);
}

}  // namespace fa
