// paged_small_scaled.cu -- paged_small.cu's attention for 9 to 16 rows per
// (sequence, kv head), over a cache held in 8 bits (e4m3 codes, a scale for each
// page and kv head).  Fewer rows are paged_eight_scaled.cu's, whose loader this
// kernel shares.
//
// What differs from paged_small.cu.  The codes come into shared memory as they are
// and are converted in registers, each once per CTA, to f16, which holds them
// exactly; so does it a row of Q scaled by a power of two, and P, at most 2^15 (kPTop),
// is rounded to f16's 11 bits instead of bf16's 8.  Products and sums are fp32's, k's
// scale is applied to S and v's, with P's 2^15 taken out again, to the product of 16
// keys, which are of one page: any scales will do (below 2^-111 a v scale with the
// 2^-15 is a subnormal number, and keeps 8 bits down to 2^-126).
//
// A thread's 32 bits of a row of codes are four adjacent columns where a matrix
// product's operand has two and two: K's columns go to the product in another
// order, and Q's with them; V's 16-byte chunks come transposed as pairs of
// columns, whose even and odd ones go to two products.  Consumer warp w computes
// S for 16 of a tile's 128 keys; the warps exchange their row maxima and P through
// shared memory, and each has an eighth of O's columns.
//
// 64 sequences of 3 tokens, 4 heads to a kv head of 64 columns, a window of 1024:
// 27.0 us (bf16 cache 23; 5 at the copy rate): start and join, about 9, then the
// warps' two exchanges per tile.  The form for 8 rows, with a warp's keys to itself
// and twice the columns of P, took 38.
#include "paged_codes.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;                        // consumers; warp 8 loads
constexpr int kRows = kPagedSmallRows;
static_assert(kKeys == 16 * kWarps, "16 keys to a warp");
constexpr float kPDown = 1.f / 32768.f;          // 2^-kPTop

// Beside the ring and the queues: P, and every warp's [rows] maximum and sum.
constexpr uint32_t kPRow = 2u * kKeys + 16u;     // 16 bytes of padding: rows on distinct banks
template <int D>
struct Sixteen : CodeLayout<D, kWarps, 1, kRows, kRows * kPRow + 8u * kRows * kWarps> {
    static constexpr uint32_t kP = Sixteen::kExtra, kMax = kP + kRows * kPRow, kSum = kMax + 4u * kRows * kWarps;
};

// c += a b and d = a b, one m16n8k16 tile of f16, fp32 sums
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_from_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The same barrier with a vote: whether `ok` holds in every thread.
__device__ __forceinline__ bool consumers_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(ok))
        : "memory");
    return r != 0;
}

// A thread's columns of row e of O (times inv), as fp32, and to the output:
// 16 (the warp's chunk) + 4 tq + {0, 2} of tile 0, {1, 3} of tile 1; of 64 columns
// two warps share a chunk, a tile each.
template <int D>
__device__ __forceinline__ void store_columns(float* dst, int warp, int tq, const float (&o)[D / 64][4], int e, float inv) {
    if constexpr (D == 128) {
        *reinterpret_cast<float4*>(dst + 16 * warp + 4 * tq) =
            make_float4(o[0][2 * e] * inv, o[1][2 * e] * inv, o[0][2 * e + 1] * inv, o[1][2 * e + 1] * inv);
    } else {
        dst += 16 * (warp >> 1) + 4 * tq + (warp & 1);
        dst[0] = o[0][2 * e] * inv;
        dst[2] = o[0][2 * e + 1] * inv;
    }
}
template <int D>
__device__ __forceinline__ void put_columns(const PagedParams& p, long long at, int warp, int tq,
                                            const float (&o)[D / 64][4], int e, float inv) {
    if (p.flags & FA_OUT_FP32) {
        store_columns<D>(static_cast<float*>(p.o) + at, warp, tq, o, e, inv);
        return;
    }
    if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + at + 16 * warp + 4 * tq) =
            make_uint2(pack_bf16x2(o[0][2 * e] * inv, o[1][2 * e] * inv),
                       pack_bf16x2(o[0][2 * e + 1] * inv, o[1][2 * e + 1] * inv));
    } else {
        uint16_t* const dst = static_cast<uint16_t*>(p.o) + at + 16 * (warp >> 1) + 4 * tq + (warp & 1);
        const uint32_t w = pack_bf16x2(o[0][2 * e] * inv, o[0][2 * e + 1] * inv);
        dst[0] = static_cast<uint16_t>(w);
        dst[2] = static_cast<uint16_t>(w >> 16);
    }
}

template <int D, int SCORE>
__global__ void __launch_bounds__(Sixteen<D>::kThreads, 2)
paged_small_scaled_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const PagedScaledParams p) {
    using L = Sixteen<D>;
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
    const Line line = code_line<L>(p, smem, cta, warp == kWarps);
    const WaitCtl wc{abort_flag, p.ws, p.timeout_ns};

    if (warp == kWarps) {
        load_codes<L, kLoadBoth>(p, tmK, tmV, line, smem, sbase, wc, lane);
        if (p.join_rows) pdl_wait_previous();
        return;
    }

    // --------------------------------------------------------------- consumers
    const int gr = lane >> 2, tq = lane & 3, mi = lane >> 3, l8 = lane & 7;
    float* const smax = reinterpret_cast<float*>(smem + L::kMax);
    float* const ssum = reinterpret_cast<float*>(smem + L::kSum);
    // score_mod, to base 2
    const float sl2 = p.scale * kPagedLog2e;
    const SoftCap cap = soft_cap(p.score.softcap, SCORE == FA_SCORE_SOFTCAP ? p.scale : 1.f);
    constexpr int kNT = D / 64;                    // n8 tiles of O per warp
    const int chunk = D == 128 ? warp : warp >> 1; // the warp's 16 columns of O, or half of their columns
    const uint32_t pick = D == 128 ? 0x3120u : (warp & 1) ? 0x0031u : 0x0020u;
    const int by_page = min(p.c.page_shift, kShift);       // 2^by_page keys of a tile share a page
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
        int tok[2], hq[2];
        float slope[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = min(gr + 8 * e, rows - 1);
            tok[e] = quotient(r, p.by_group);
            hq[e] = s.h * p.group + r - tok[e] * p.group;
            if (SCORE == FA_SCORE_ALIBI) slope[e] = p.score.slopes[hq[e]] * kPagedLog2e;
            if (SCORE == FA_SCORE_ALIBI_SOFTCAP) slope[e] = p.score.slopes[hq[e]];
        }
        // Q's fragments in f16: a row times a power of two, so that its largest
        // element is 2^14 .. 2^15 and those below f16's normal numbers are 2^28
        // times smaller (rows past the unit's are 0); columns 4 tq .. 4 tq + 3 of 16
        // where the product has 2 tq, 2 tq + 1, 2 tq + 8 and 2 tq + 9.
        uint32_t qa[D / 16][4];
        float unscale[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint8_t* const q_row = smem + L::kQ + ((nu & 1) * kRows + gr + 8 * e) * L::kQRow + 8 * tq;
            float top = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint2 w = gr + 8 * e < rows ? *reinterpret_cast<const uint2*>(q_row + 32 * ks) : make_uint2(0u, 0u);
                qa[ks][e] = w.x;
                qa[ks][2 + e] = w.y;
                top = fmaxf(top, fmaxf(fmaxf(fabsf(bf_low(w.x)), fabsf(bf_high(w.x))),
                                       fmaxf(fabsf(bf_low(w.y)), fabsf(bf_high(w.y)))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int at = max(__float_as_int(top) >> 23, 15);
            const float up = __int_as_float((268 - at) << 23);
            unscale[e] = __int_as_float((at - 14) << 23);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                qa[ks][e] = pack_f16x2(bf_low(qa[ks][e]) * up, bf_high(qa[ks][e]) * up);
                qa[ks][2 + e] = pack_f16x2(bf_low(qa[ks][2 + e]) * up, bf_high(qa[ks][2 + e]) * up);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(L::q_empty(sbase, nu));
        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
        float o[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

        const int tiles = s.k1 - s.k0;
        for (int k = 0; k < tiles; ++k, ++g) {
            const int st = g % ST;
            const uint32_t kbase = sbase + st * L::kStage, vbase = kbase + L::kTile;
            const float* const sc = reinterpret_cast<const float*>(smem + L::kScale + st * L::kScaleStage);
            const bool here = mbar_wait_warp(L::full(sbase, st), (g / ST) & 1, wc, S_PC_FULL);
            const int info = info_s[st], j0 = (info >> 2) * kKeys + 16 * warp;
            float x[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
            bool cleared = false;
            if (here) {
                float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                for (int ks = 0; ks < D / 16; ks += 2) {
                    uint32_t kf[4], lo[4], hi[4];
                    ldsm4(kbase + swz8<D>(16 * warp + 8 * (mi >> 1) + l8, ks + (mi & 1)), kf);
#pragma unroll
                    for (int e = 0; e < 4; ++e) codes_to_f16(kf[e], lo[e], hi[e]);
                    mma_f16(x[0], qa[ks], lo[0], hi[0]);
                    mma_f16(x[1], qa[ks], lo[2], hi[2]);
                    mma_f16(x[0], qa[ks + 1], lo[1], hi[1]);
                    mma_f16(x[1], qa[ks + 1], lo[3], hi[3]);
                }
                const float k_scale = sc[16 * warp >> by_page];
                const bool open = (info & kTileOpen) != 0;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int e = c >> 1, j = j0 + 8 * nt + 2 * tq + (c & 1);
                        float v = x[nt][c] * unscale[e] * k_scale;
                        const float far = fabsf(static_cast<float>(i0 + tok[e] - j));
                        if (SCORE == FA_SCORE_NONE || SCORE == FA_SCORE_REL_BIAS) v *= sl2;
                        if (SCORE == FA_SCORE_SOFTCAP) v = softcap_one(v, cap);
                        if (SCORE == FA_SCORE_ALIBI) v = fmaf(-slope[e], far, v * sl2);
                        if (SCORE == FA_SCORE_ALIBI_SOFTCAP) v = softcap_one(fmaf(-slope[e], far, v * p.scale), cap);
                        if (SCORE == FA_SCORE_REL_BIAS) {
                            const int R = p.score.rel_max, d = min(max(i0 + tok[e] - j, -R), R);
                            v = fmaf(p.score.rel_bias[(size_t)hq[e] * (2 * R + 1) + d + R], kPagedLog2e, v);
                        }
                        if (!open && !paged_visible(p.mask, i0 + tok[e], j, p.shared, s.kv)) v = -CUDART_INF_F;
                        x[nt][c] = v;
                        mx[e] = fmaxf(mx[e], v);
                    }
                }
                if (info & kTileClear) {
                    // V rows that no row of the unit sees
                    constexpr int kChunks = D / 16;
                    cleared = true;
                    const uint32_t live = __ballot_sync(0xffffffffu, s.hull.live(j0 + (lane & 15)));
#pragma unroll
                    for (int e = 0; e < kChunks / 2; ++e) {
                        const int r = (32 * e + lane) / kChunks;
                        if (!((live >> r) & 1u))
                            *reinterpret_cast<uint4*>(smem + st * L::kStage + L::kTile + swz8<D>(16 * warp + r, lane % kChunks)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                    if (tq == 0) smax[(gr + 8 * e) * kWarps + warp] = mx[e];
                }
            }
            // (a warp whose wait ran out still comes here, so that all leave together)
            if (!consumers_all(here)) { ok = false; break; }
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 a = *reinterpret_cast<const float4*>(smax + (gr + 8 * e) * kWarps);
                const float4 b = *reinterpret_cast<const float4*>(smax + (gr + 8 * e) * kWarps + 4);
                const float m_new = fmaxf(fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)),
                                                fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w))), m[e]);
                alpha[e] = m_new == m[e] ? 1.f : ex2_approx(m[e] - m_new);
                const float nm = m_new == -CUDART_INF_F ? 0.f : kPTop - m_new;
                m[e] = m_new;
                l[e] *= alpha[e];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const float p0 = ex2_approx(x[nt][2 * e] + nm), p1 = ex2_approx(x[nt][2 * e + 1] + nm);
                    l[e] += p0 + p1;
                    *reinterpret_cast<uint32_t*>(smem + L::kP + (gr + 8 * e) * kPRow + 2 * (16 * warp + 8 * nt + 2 * tq)) =
                        pack_p(p0, p1);
                }
            }
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                o[n][0] *= alpha[0];
                o[n][1] *= alpha[0];
                o[n][2] *= alpha[1];
                o[n][3] *= alpha[1];
            }
            consumers_sync();
            // O's columns of this warp += P V over the tile's keys, 16 at a time,
            // which are of one page, and its scale on their sum
            const uint32_t p_row = sbase + L::kP + (l8 + 8 * (mi & 1)) * kPRow + 16 * (mi >> 1);
#pragma unroll
            for (int ks = 0; ks < kKeys / 16; ks += 2) {
                uint32_t vf[4], lo[4], hi[4];
                ldsm4_t(vbase + swz8<D>(16 * ks + 8 * mi + l8, chunk), vf);
#pragma unroll
                for (int e = 0; e < 4; ++e) codes_to_f16(__byte_perm(vf[e], 0u, pick), lo[e], hi[e]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t pa[4];
                    ldsm4(p_row + 32 * (ks + e), pa);
                    const float v_scale = sc[kKeys / 16 + (16 * (ks + e) >> by_page)] * kPDown;
                    float y[4];
                    mma_f16_from_0(y, pa, lo[2 * e], lo[2 * e + 1]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[0][c] = fmaf(y[c], v_scale, o[0][c]);
                    if constexpr (kNT == 2) {
                        mma_f16_from_0(y, pa, hi[2 * e], hi[2 * e + 1]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[1][c] = fmaf(y[c], v_scale, o[1][c]);
                    }
                }
            }
            if (cleared) fence_async_shared();     // the next copy into this stage comes after the clearing
            __syncwarp();
            if (lane == 0) mbar_arrive(L::empty(sbase, st));
        }
        if (!ok) break;

        // the unit's end in this CTA: row sums over the lanes and warps
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (tq == 0) ssum[(gr + 8 * e) * kWarps + warp] = l[e] * kPDown;
        }
        consumers_sync();
        const bool whole = s.begins() && s.ends();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = gr + 8 * e;
            if (r >= rows) continue;
            const float4 a = *reinterpret_cast<const float4*>(ssum + r * kWarps);
            const float4 b = *reinterpret_cast<const float4*>(ssum + r * kWarps + 4);
            const float sum = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
            const long long row = (long long)(s.q0 + tok[e]) * p.Hq + hq[e];
            if (whole && !p.join_rows) {
                put_columns<D>(p, row * D, warp, tq, o, e, sum == 0.f ? 0.f : 1.f / sum);     // a NaN stays one
                if (warp == 0 && tq == 0) p.lse[row] = sum == 0.f ? -CUDART_INF_F : (m[e] + log2f(sum)) * kPagedLn2;
            } else {
                const long long slot = whole ? row : (2LL * cta + (s.begins() ? 1 : 0)) * kRows + r;
                store_columns<D>((whole ? p.parts.row_o : p.parts.slot_o) + slot * D, warp, tq, o, e, 1.f);
                if (warp == 0 && tq == 0) {
                    (whole ? p.parts.row_ml : p.parts.slot_ml)[slot] = make_float2(m[e], sum);
                    if (p.join_rows && s.begins())
                        p.rowdesc[row] = whole ? make_int2(-1, 1) : make_int2((2 * cta + 1) * kRows + r, s.count);
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
    auto kern = paged_small_scaled_kernel<D, SCORE>;
    using L = Sixteen<D>;
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

cudaError_t launch_paged_small_scaled(const PagedScaledParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      cudaStream_t s) {
    return p.D == 64 ? launch_score<64>(p, tk, tv, s) : launch_score<128>(p, tk, tv, s);
}

}  // namespace fa
