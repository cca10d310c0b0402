// paged_api.cu -- the C ABI of the paged cache (include/fa_paged.h): argument
// validation, scratch layout and launches.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/fa_paged.h"
#include "fa_internal.h"
#include "ptx.cuh"

namespace {

fa_status fail(fa_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return fa::report(st, buf);
}

fa_status cuda_fail(cudaError_t e, const char* what) {
    return fail(FA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

fa_status check_cache(const fa_paged_kv* c) {
    if (!c) return fail(FA_ERR_INVALID_ARG, "the paged cache is NULL");
    if (c->B < 1 || c->Hkv < 1 || c->num_pages < 1 || c->max_pages < 1 || c->total_q < 0)
        return fail(FA_ERR_INVALID_ARG, "B, Hkv, num_pages and max_pages must be >= 1 and total_q >= 0 "
                    "(got %d, %d, %d, %d, %d)", c->B, c->Hkv, c->num_pages, c->max_pages, c->total_q);
    if (c->D != 64 && c->D != 128) return fail(FA_ERR_UNSUPPORTED, "head dim %d not supported (64 or 128)", c->D);
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return fail(FA_ERR_UNSUPPORTED, "page size %d not supported (16, 32, 64, 128 or 256)", c->page_size);
    if ((long long)c->num_pages * c->Hkv > 2147483647LL)
        return fail(FA_ERR_UNSUPPORTED, "num_pages x Hkv must be below 2^31");
    if ((long long)c->max_pages * c->page_size > 2147483647LL - 1024)
        return fail(FA_ERR_UNSUPPORTED, "max_pages x page_size must be below 2^31 - 1024");
    if (!c->k || !c->v || !c->page_table || !c->kv_len || !c->q_start)
        return fail(FA_ERR_INVALID_ARG, "k, v, page_table, kv_len and q_start must be non-NULL");
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return fail(FA_ERR_INVALID_ARG, "the cache's k and v must be 16-byte aligned");
    if (!aligned(c->page_table, 4) || !aligned(c->kv_len, 4) || !aligned(c->q_start, 4))
        return fail(FA_ERR_INVALID_ARG, "page_table, kv_len and q_start must be 4-byte aligned");
    return FA_OK;
}

// Rows that 16-byte accesses read or write: aligned, strides multiples of 8
// elements (0 repeats a row).
fa_status check_rows(const char* name, const void* p, const int64_t (&st)[2]) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "%s must be non-NULL", name);
    if (!aligned(p, 16)) return fail(FA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (st[0] < 0 || st[1] < 0 || (st[0] & 7) || (st[1] & 7))
        return fail(FA_ERR_INVALID_ARG, "%s: strides must be non-negative multiples of 8 elements (got %lld, %lld)", name,
                    (long long)st[0], (long long)st[1]);
    return FA_OK;
}

fa::PagedView view(const fa_paged_kv* c) {
    fa::PagedView v{};
    v.B = c->B;
    v.Hkv = c->Hkv;
    v.num_pages = c->num_pages;
    v.page_size = c->page_size;
    for (v.page_shift = 4; (1 << v.page_shift) < c->page_size; ++v.page_shift) {}
    v.max_pages = c->max_pages;
    v.total_q = c->total_q;
    v.page_table = c->page_table;
    v.kv_len = c->kv_len;
    v.q_start = c->q_start;
    return v;
}

// The kernel that a call's own keys take: 16-row units (mma.sync) while every
// sequence's rows of a kv head fit in one, 256-row units (tcgen05) beyond, where
// 16-row units would read every key twice.  64 sequences of 4096 (1024) keys, 8
// kv heads of 128 columns, by rows: 4: 169 (52) us in 16-row units, 177 (57) in
// 256-row ones; 16: 173 (53) and 180 (59); beyond, 17: 181 (59), 64: 187 (62).
// One sequence of 4096 keys: 4: 10.9 and 13.7; 16: 12.0 and 19.2.
bool small_rows(const fa_paged_kv* c, const fa_paged_fwd_args* a) {
    return (long long)a->max_q_len * (a->Hq / c->Hkv) <= fa::kPagedSmallRows;
}

fa_status check_fwd(const fa_paged_kv* c, const fa_paged_fwd_args* a) {
    fa_status st = check_cache(c);
    if (st != FA_OK) return st;
    if (!a) return fail(FA_ERR_INVALID_ARG, "the paged forward's args are NULL");
    if (c->B > fa::kPagedMaxSeqs)
        return fail(FA_ERR_UNSUPPORTED, "at most %d sequences per call (got %d)", fa::kPagedMaxSeqs, c->B);
    if (a->Hq < 1 || a->Hq % c->Hkv != 0)
        return fail(FA_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", a->Hq, c->Hkv);
    if (a->max_q_len < 1) return fail(FA_ERR_INVALID_ARG, "max_q_len must be >= 1 (got %d)", a->max_q_len);
    if (a->shared_len < 0) return fail(FA_ERR_INVALID_ARG, "shared_len must be >= 0 (got %d)", a->shared_len);
    const long long cap = (long long)c->max_pages * c->page_size;
    if (a->shared_len > cap)
        return fail(FA_ERR_INVALID_ARG, "shared_len (%d) is past max_pages x page_size (%lld)", a->shared_len, cap);
    if (c->Hkv > 65535) return fail(FA_ERR_UNSUPPORTED, "Hkv must be <= 65535");
    // the line of tiles is counted in 32 bits: units (at most one partly
    // filled one per sequence) x kv heads x tiles (of 64 keys, or of 128 and
    // a few for the unit itself)
    const long long group = a->Hq / c->Hkv, tiles = cap / 64 + 4;
    const double units = (double)c->B + (double)c->total_q * group / fa::kPagedTileRows + 1;
    if (units * c->Hkv * tiles > 2147483647.0 || (long long)c->total_q * a->Hq > 2147483647LL)
        return fail(FA_ERR_UNSUPPORTED, "too much work for one call (%d rows of %d heads against up to %lld keys)",
                    c->total_q, a->Hq, cap);
    return FA_OK;
}

// The scratch in order: the prefix's two numbers and mark, the units to join, the two
// slots per CTA; with a shared prefix the same for it, and partials by row.
struct Scratch {
    size_t hdr, meta, slot_o, slot_ml, row_o, row_ml, desc, pre_slot_o, pre_slot_ml, pre_row_o, pre_row_ml, bytes;
};

// CTAs that share the work of a call's own keys.
int own_ctas(const fa_paged_kv* c, const fa_paged_fwd_args* a) {
    return fa::device_sm_count() * (small_rows(c, a) ? fa::kPagedSmallCtasPerSm : 1);
}

Scratch layout(const fa_paged_kv* c, const fa_paged_fwd_args* a) {
    Scratch s{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) & ~(size_t)255;
        return here;
    };
    const size_t ctas = own_ctas(c, a), D = c->D;
    const size_t own = 2 * ctas * (small_rows(c, a) ? fa::kPagedSmallRows : fa::kPagedTileRows);
    s.hdr = take(256);
    s.meta = take(ctas * sizeof(fa::PagedMeta));
    s.slot_o = take(own * D * 4);
    s.slot_ml = take(own * 8);
    if (a->shared_len > 0) {
        const size_t rows = (size_t)c->total_q * a->Hq, pre = 2 * (size_t)fa::device_sm_count() * fa::kPagedTileRows;
        s.row_o = take(rows * D * 4);
        s.row_ml = take(rows * 8);
        s.desc = take(rows * 8);
        s.pre_slot_o = take(pre * D * 4);
        s.pre_slot_ml = take(pre * 8);
        s.pre_row_o = take(rows * D * 4);
        s.pre_row_ml = take(rows * 8);
    }
    s.bytes = at;
    return s;
}

}  // namespace

extern "C" {

fa_status fa_kv_append(const fa_paged_kv* c, const fa_kv_append_args* a, void* workspace, void* stream) {
    fa_status st = check_cache(c);
    if (st != FA_OK) return st;
    if (!a) return fail(FA_ERR_INVALID_ARG, "the append's args are NULL");
    if (!workspace) return fail(FA_ERR_INVALID_ARG, "workspace is NULL");
    if (a->Hq < 0) return fail(FA_ERR_INVALID_ARG, "Hq must be >= 0 (got %d)", a->Hq);
    if (a->rot_dim < 0 || a->rot_dim > c->D || a->rot_dim % 16)
        return fail(FA_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16 from 0 to D=%d (got %d)", c->D, a->rot_dim);
    if (a->interleaved != 0 && a->interleaved != 1)
        return fail(FA_ERR_INVALID_ARG, "interleaved must be 0 or 1 (got %d)", a->interleaved);
    if ((long long)a->Hq + 2LL * c->Hkv > 1 << 24) return fail(FA_ERR_UNSUPPORTED, "too many heads");
    if (c->total_q == 0) return fa::report(FA_OK, "");     // no rows: their pointers may be NULL
    if ((st = check_rows("k", a->k, a->k_stride)) != FA_OK) return st;
    if ((st = check_rows("v", a->v, a->v_stride)) != FA_OK) return st;
    if (a->Hq > 0) {
        if ((st = check_rows("q", a->q, a->q_stride)) != FA_OK) return st;
        if ((st = check_rows("q_out", a->q_out, a->q_out_stride)) != FA_OK) return st;
        // an output row must not run into another: heads within tokens or
        // tokens within heads
        const int64_t hs = a->Hq > 1 ? a->q_out_stride[1] : c->D, ts = c->total_q > 1 ? a->q_out_stride[0] : c->D;
        if ((double)(a->Hq - 1) * hs + c->D > ts && (double)(c->total_q - 1) * ts + c->D > hs)
            return fail(FA_ERR_INVALID_ARG, "q_out's strides (%lld, %lld) overlap its rows", (long long)ts, (long long)hs);
        if (a->q_out == a->q && ((c->total_q > 1 && ts != a->q_stride[0]) || (a->Hq > 1 && hs != a->q_stride[1])))
            return fail(FA_ERR_INVALID_ARG, "q_out is q with other strides");
    }
    if (a->rot_dim > 0) {
        if (!a->cos || !a->sin || a->rope_len < 1)
            return fail(FA_ERR_INVALID_ARG, "a rotation needs cos, sin and rope_len >= 1");
        if (!aligned(a->cos, 16) || !aligned(a->sin, 16))
            return fail(FA_ERR_INVALID_ARG, "cos and sin must be 16-byte aligned");
    }
    if (!aligned(a->positions, 4)) return fail(FA_ERR_INVALID_ARG, "positions must be 4-byte aligned");
    const uintptr_t kc = reinterpret_cast<uintptr_t>(c->k), vc = reinterpret_cast<uintptr_t>(c->v);
    if ((double)(kc > vc ? kc - vc : vc - kc) < 2.0 * c->num_pages * c->Hkv * c->page_size * c->D)
        return fail(FA_ERR_INVALID_ARG, "the cache's k and v overlap");

    fa::AppendParams p{};
    p.c = view(c);
    p.Hq = a->Hq;
    p.D = c->D;
    p.rot = a->rot_dim;
    p.rope_len = a->rope_len;
    p.interleaved = a->interleaved;
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.q_out = static_cast<uint16_t*>(a->q_out);
    p.kc = static_cast<uint16_t*>(c->k);
    p.vc = static_cast<uint16_t*>(c->v);
    for (int e = 0; e < 2; ++e) {
        p.qs[e] = a->q_stride[e];
        p.ks[e] = a->k_stride[e];
        p.vs[e] = a->v_stride[e];
        p.os[e] = a->q_out_stride[e];
    }
    p.cos = a->cos;
    p.sin = a->sin;
    p.positions = a->positions;
    p.ws = static_cast<uint32_t*>(workspace);
    cudaError_t e = fa::launch_kv_append(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
    return fa::report(FA_OK, "");
}

size_t fa_paged_scratch_bytes(const fa_paged_kv* c, const fa_paged_fwd_args* a) {
    if (check_fwd(c, a) != FA_OK) return 0;
    fa::report(FA_OK, "");
    return layout(c, a).bytes;
}

fa_status fa_fwd_paged(const fa_paged_kv* c, const fa_paged_fwd_args* a, const fa_mask_desc* mask,
                       const fa_score_desc* sc, void* scratch, size_t scratch_bytes, void* workspace, void* stream) {
    fa_status st = check_fwd(c, a);
    if (st != FA_OK) return st;
    if (!mask) return fail(FA_ERR_INVALID_ARG, "the mask is NULL");
    fa::PagedMask m{0, -1, 0};
    switch (mask->kind) {
        case FA_MASK_FULL: break;
        case FA_MASK_CAUSAL: m.causal = 1; break;
        case FA_MASK_SINK_WINDOW:
            if (mask->prefix_len < 0)
                return fail(FA_ERR_INVALID_ARG, "the sink count (prefix_len) must be >= 0 (got %d)", mask->prefix_len);
            m.sinks = mask->prefix_len;
            [[fallthrough]];
        case FA_MASK_SLIDING_WINDOW:
            if (mask->window < 0) return fail(FA_ERR_INVALID_ARG, "sliding window must be >= 0 (got %d)", mask->window);
            m.causal = 1;
            m.window = mask->window;
            break;
        default:
            return fail(FA_ERR_UNSUPPORTED, "mask kind %d: the paged forward takes full, causal, sliding-window and "
                        "sink-window masks", mask->kind);
    }
    fa_score_desc score;
    if ((st = fa::check_score_desc(sc, &score)) != FA_OK) return st;
    if (c->total_q == 0) return fa::report(FA_OK, "");     // no rows: their pointers may be NULL
    if ((st = check_rows("q", a->q, a->q_stride)) != FA_OK) return st;
    if (!a->o || !a->lse) return fail(FA_ERR_INVALID_ARG, "o and lse must be non-NULL");
    if (!aligned(a->o, 16) || !aligned(a->lse, 4))
        return fail(FA_ERR_INVALID_ARG, "o must be 16-byte aligned and lse 4-byte aligned");
    if (!std::isfinite(a->scale)) return fail(FA_ERR_INVALID_ARG, "scale must be finite");
    if (a->flags & ~FA_OUT_FP32) return fail(FA_ERR_INVALID_ARG, "unknown flags 0x%x", a->flags);
    if (!workspace) return fail(FA_ERR_INVALID_ARG, "workspace is NULL");
    if (!scratch || !aligned(scratch, 16))
        return fail(FA_ERR_INVALID_ARG, "scratch must be non-NULL and 16-byte aligned");
    const Scratch lay = layout(c, a);
    if (scratch_bytes < lay.bytes)
        return fail(FA_ERR_INVALID_ARG, "scratch holds %zu bytes, %zu needed", scratch_bytes, lay.bytes);

    uint8_t* base = static_cast<uint8_t*>(scratch);
    fa::PagedParams p{};
    p.c = view(c);
    p.mask = m;
    p.Hq = a->Hq;
    p.group = a->Hq / c->Hkv;
    p.by_group = fa::fast_div(p.group);
    p.D = c->D;
    p.max_q = a->max_q_len;
    p.shared = a->shared_len;
    p.join_rows = a->shared_len > 0;
    p.ctas = own_ctas(c, a);
    p.scale = a->scale > 0.f ? a->scale : 1.0f / std::sqrt((float)c->D);
    p.score = {score.kind, score.softcap, score.alibi_slopes, score.rel_bias, score.rel_max};
    p.q = static_cast<const uint16_t*>(a->q);
    p.qs[0] = a->q_stride[0];
    p.qs[1] = a->q_stride[1];
    p.o = a->o;
    p.lse = a->lse;
    p.meta = reinterpret_cast<fa::PagedMeta*>(base + lay.meta);
    p.hdr = reinterpret_cast<int*>(base + lay.hdr);
    p.parts.slot_o = reinterpret_cast<float*>(base + lay.slot_o);
    p.parts.slot_ml = reinterpret_cast<float2*>(base + lay.slot_ml);
    if (p.join_rows) {
        p.parts.row_o = reinterpret_cast<float*>(base + lay.row_o);
        p.parts.row_ml = reinterpret_cast<float2*>(base + lay.row_ml);
        p.rowdesc = reinterpret_cast<int2*>(base + lay.desc);
    }
    p.ws = static_cast<uint32_t*>(workspace);
    p.timeout_ns = (uint64_t)(a->timeout_ms ? a->timeout_ms : 2000u) * 1000000ull;
    p.flags = a->flags;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool small = small_rows(c, a);
    const long long blocks = (long long)c->num_pages * c->Hkv;
    alignas(64) CUtensorMap tk, tv, sk, sv;       // boxes of the tile kernel, of the small one
    if (!small || p.join_rows) {
        if ((st = fa::page_tensor_map(&tk, c->k, blocks, c->page_size, c->D, fa::kPagedTileKeys)) != FA_OK) return st;
        if ((st = fa::page_tensor_map(&tv, c->v, blocks, c->page_size, c->D, fa::kPagedTileKeys)) != FA_OK) return st;
    }
    if (small) {
        const int keys = fa::paged_small_keys(c->D);
        if ((st = fa::page_tensor_map(&sk, c->k, blocks, c->page_size, c->D, keys)) != FA_OK) return st;
        if ((st = fa::page_tensor_map(&sv, c->v, blocks, c->page_size, c->D, keys)) != FA_OK) return st;
    }
    fa::PagedParams pre = p;
    if (p.join_rows) {
        pre.prefix = 1;
        pre.ctas = fa::device_sm_count();
        pre.parts = {reinterpret_cast<float*>(base + lay.pre_slot_o), reinterpret_cast<float2*>(base + lay.pre_slot_ml),
                     reinterpret_cast<float*>(base + lay.pre_row_o), reinterpret_cast<float2*>(base + lay.pre_row_ml)};
        cudaError_t e = fa::launch_paged_tiles(pre, tk, tv, s);
        if (e != cudaSuccess) return cuda_fail(e, "shared prefix launch");
    }
    cudaError_t e = small ? fa::launch_paged_small(p, sk, sv, s) : fa::launch_paged_tiles(p, tk, tv, s);
    if (e != cudaSuccess) return cuda_fail(e, "paged forward launch");
    const int unit_rows = small ? fa::kPagedSmallRows : fa::kPagedTileRows;
    if (p.join_rows) {
        fa::PagedJoin j{};
        j.own = p;
        j.pre = pre.parts;
        j.own_rows = unit_rows;
        j.pre_ctas = pre.ctas;
        e = fa::launch_paged_join_rows(j, s);
    } else {
        e = fa::launch_paged_join_units(p, unit_rows, s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "joining launch");
    return fa::report(FA_OK, "");
}

}  // extern "C"
