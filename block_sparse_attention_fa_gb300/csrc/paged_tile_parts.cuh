// paged_tile_parts.cuh -- pieces of the two attention kernels for many rows
// (paged_tiles.cu and paged_tiles_scaled.cu).
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "paged_line.cuh"

namespace fa {
namespace {

// x <- the soft-capped score, base 2.  TRY: where no element of the warp is past
// the polynomial's range, two elements to an instruction (4 x 1024 new tokens
// at 8192 keys, cap 30: 529 us).  Otherwise, and always without TRY, the
// exponential form, at two MUFU operations per element (cap 2: 747).  A cap far
// above the scores takes the polynomial where it holds, with or without TRY;
// a warp that needs both forms evaluates both (ALiBi then a cap of 100: 1134 us,
// 1e5, where the polynomial alone does: 771; 30, exponential: 792).
template <bool TRY>
__device__ __forceinline__ void softcap_all(float (&x)[64], const SoftCap& c) {
    bool inner = false;
    if (TRY || c.fine) {
        float am = 0.f;
#pragma unroll
        for (int e = 0; e < 64; e += 2) am = fmax3(am, fabsf(x[e]), fabsf(x[e + 1]));
        inner = !__any_sync(0xffffffffu, !(am * c.in <= kTanhFineRange));
    }
    const float q0 = c.mul * kTanhFineC0, q1 = c.mul * kTanhFineC1, q2 = c.mul * kTanhFineC2, q3 = c.mul * kTanhFineC3,
                q4 = c.mul * kTanhFineC4;
    // u = x in and x mul q(u^2) of a pair
    auto pair = [&](int e, float& u0, float& u1, float& y0, float& y1) {
        float w0, w1;
        ffma2(u0, u1, x[e], x[e + 1], c.in, c.in, -0.f, -0.f);
        ffma2(w0, w1, u0, u1, u0, u1, -0.f, -0.f);
        ffma2(y0, y1, w0, w1, q4, q4, q3, q3);
        ffma2(y0, y1, y0, y1, w0, w1, q2, q2);
        ffma2(y0, y1, y0, y1, w0, w1, q1, q1);
        ffma2(y0, y1, y0, y1, w0, w1, q0, q0);
        ffma2(y0, y1, x[e], x[e + 1], y0, y1, -0.f, -0.f);
    };
    if (inner) {
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
            float u0, u1, y0, y1;
            pair(e, u0, u1, y0, y1);
            x[e] = y0;
            x[e + 1] = y1;
        }
    } else if (c.fine) {
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
            float u0, u1, y0, y1;
            pair(e, u0, u1, y0, y1);
            x[e] = softcap_pick(y0, u0, c);
            x[e + 1] = softcap_pick(y1, u1, c);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 64; ++e) x[e] = softcap_outer(x[e] * c.in, c);
    }
}

__device__ __forceinline__ void exp2_pair(float& p0, float& p1, float x0, float x1, float sc, float nm) {
    float a0, a1;
    ffma2(a0, a1, x0, x1, sc, sc, nm, nm);
    p0 = ex2_approx(a0);
    p1 = ex2_approx(a1);
}

// 16 bytes from global into shared memory, without passing registers; zeros
// where `there` does not hold.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Eight words; `wide`: to a 32-byte boundary (16 otherwise).
__device__ __forceinline__ void store8(void* dst, const uint32_t* w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Bits a .. 31, and bits 0 .. a, of a word (any a).
__device__ __forceinline__ uint32_t bits_from(int a) { return a <= 0 ? 0xffffffffu : a > 31 ? 0u : 0xffffffffu << a; }
__device__ __forceinline__ uint32_t bits_to(int a) { return a < 0 ? 0u : a >= 31 ? 0xffffffffu : 0xffffffffu >> (31 - a); }

// Finds the unit group of ln.b in which the stretch begins: a lane to a group
// of the next 32.
__device__ __forceinline__ void seek(const PagedParams& p, TileLine& ln, int lane) {
    const int q0 = ln.q0[ln.b], n = ln.q0[ln.b + 1] - q0, kv = ln.kv[ln.b];
    for (; ln.rt * kPagedTileRows < n * p.group; ln.rt += 32) {
        int len = 0;
        if ((ln.rt + lane) * kPagedTileRows < n * p.group) len = p.c.Hkv * unit_length(p, n, kv, ln.rt + lane);
        int upto = len;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        const uint32_t behind = __ballot_sync(0xffffffffu, ln.start + upto > ln.t);
        const int at = behind ? __ffs(behind) - 1 : 31;
        ln.start += __shfl_sync(0xffffffffu, behind ? upto - len : upto, at);
        if (behind) {
            ln.rt += at;
            return;
        }
    }
}

// Rows r0 .. r0 + 31 of a unit's Q into their row tile at `tile` (128-byte
// swizzled, zeros past the unit's rows), D / 8 lanes to a row, so that whole
// lines are read.
template <int D>
__device__ __forceinline__ void load_rows(const PagedParams& p, const TileSeg& s, int r0, uint32_t tile, int lane) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;      // lanes per row, rows per copy
    const int ur = r0 + lane, R = s.row0 + min(ur, s.rows - 1), tok = quotient(R, p.by_group);
    const long long mine = ur < s.rows ? (long long)(s.q0 + tok) * p.qs[0] +
                                             (long long)(s.h * p.group + R - tok * p.group) * p.qs[1]
                                       : -1;
    const int c = lane % kLanes;
    tile += (c >> 3) * 16384u;
#pragma unroll 4
    for (int e = 0; e < kLanes; ++e) {
        const long long at = __shfl_sync(0xffffffffu, mine, e * kPer + lane / kLanes);
        const int rr = (r0 & 127) + e * kPer + lane / kLanes;
        copy16(tile + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), p.q + (at >= 0 ? at + 8 * c : 0), at >= 0);
    }
}

}  // namespace
}  // namespace fa
