// paged_step.cu -- a step's page tables, offsets and slots from its sequences'
// lengths (fa_paged_step).
//
// With before_b and after_b the entries of sequence b's row of the page table
// before and behind the step (at least the shared ones), three exclusive sums
// over the sequences place everything:
//     Q of new_len, G of max(before - after, 0), T of max(after - before, 0).
// The g-th page given back (sequences and entries ascending) goes to place
// F + R - 1 - g of the stack of free pages (F pages before, R given in all),
// and the k-th page taken is the one at place F + R - 1 - k: of the stack as it
// was, or for k < R the k-th page given back.  Row t of the step belongs to the
// sequence with Q_b <= t < Q_b + new_b.
//
// So every entry and every slot follows from the arguments alone, and one launch
// does it all: each CTA makes the sums for itself (the lengths of 2048 sequences
// are 24 KB) and takes its share of the pages and rows; a row's page comes from
// the table, or from the stack by the same formula, never from another CTA.  The
// last CTA to have read the lengths (a counter in the workspace, 0 between
// launches) writes what may be written in place: the lengths and the count.  One
// CTA does up to kRowsEach rows, whatever pages move: 500000 pages that are given back
// at once are one CTA's where no rows come with them.
//
// What it costs is latency, load after load: 5.1 us for 64 sequences with a token
// each, 8.1 for 256 with 61000 rows, 13.0 for 512 with 1.2 million (2.1 for their 14
// MB at the copy rate).  The ticket is drawn as soon as the lengths are read: at
// the end it took 1 and 2 us more.
#include <algorithm>

#include "paged.cuh"

namespace fa {
namespace {

constexpr int kRowsEach = 2048;          // rows that are worth a CTA (pages that move do not count)
constexpr int kSlotRows = 4;             // rows of a thread, adjacent ones
// The counter's word of the workspace (behind the forward's).
constexpr int kStepTicket = WS_SCHED_DONE + 1;
static_assert(kStepTicket < WS_WORDS, "a word of the workspace");

// The last of the n sequences with pre[b] <= x (pre[0] = 0 <= x < pre[n]): the one whose share holds x.
__device__ __forceinline__ int share_of(const int* pre, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Sequence b's numbers: tokens kept and new, entries before and behind the step.
struct StepSeq {
    int keep, count, before, after;
    bool fits;
};
__device__ __forceinline__ StepSeq step_sequence(const StepParams& p, int b) {
    const int old = p.kv_len[b], up = p.page_size - 1;
    StepSeq s;
    s.keep = p.keep_len[b];
    s.count = p.new_len[b];
    const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
    const long long most = max(static_cast<long long>(old), static_cast<long long>(p.shared_pages) << p.page_shift);
    s.fits = old >= 0 && old <= room && s.keep >= 0 && s.keep <= most && s.count >= 0 &&
             static_cast<long long>(s.keep) + s.count <= room;
    if (!s.fits) {
        s.keep = s.count = s.before = s.after = 0;
        return s;
    }
    s.before = max((old + up) >> p.page_shift, p.shared_pages);
    s.after = max((s.keep + s.count + up) >> p.page_shift, p.shared_pages);
    return s;
}

// Three sums at once, of 64 bits: 2048 sequences' numbers of 31 bits may add up to more than 32.
struct Sums {
    long long q, take, give;
};

template <int THREADS>
__global__ void __launch_bounds__(THREADS) paged_step_kernel(const StepParams p, bool wide) {
    extern __shared__ int step_smem[];
    int* const q_pre = step_smem;
    int* const take = q_pre + p.B + 1;
    int* const give = take + p.B + 1;
    int* const keep_s = give + p.B + 1;
    int* const before_s = keep_s + p.B;
    __shared__ Sums warp_sums[THREADS / 32];
    __shared__ int first_bad;
    __shared__ unsigned ticket;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) first_bad = INT_MAX;
    __syncthreads();
    pdl_wait_previous();
    pdl_launch_next();
    const int F = p.free_count[0];

    // the sums; a thread has `per` sequences
    const int per = (p.B + THREADS - 1) / THREADS, b0 = tid * per, b1 = min(b0 + per, p.B);
    Sums mine{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
        const StepSeq s = step_sequence(p, b);
        if (!s.fits) atomicMin(&first_bad, b);
        keep_s[b] = s.keep;
        before_s[b] = s.before;
        q_pre[b] = s.count;
        take[b] = max(s.after - s.before, 0);
        give[b] = max(s.before - s.after, 0);
        mine.q += s.count;
        mine.take += take[b];
        mine.give += give[b];
    }
    Sums upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long q = __shfl_up_sync(0xffffffffu, upto.q, d), t = __shfl_up_sync(0xffffffffu, upto.take, d),
                        g = __shfl_up_sync(0xffffffffu, upto.give, d);
        if (lane >= d) {
            upto.q += q;
            upto.take += t;
            upto.give += g;
        }
    }
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    Sums base{upto.q - mine.q, upto.take - mine.take, upto.give - mine.give}, all{0, 0, 0};
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const Sums x = warp_sums[w];
        if (w < warp) {
            base.q += x.q;
            base.take += x.take;
            base.give += x.give;
        }
        all.q += x.q;
        all.take += x.take;
        all.give += x.give;
    }
    const bool good = first_bad == INT_MAX && F >= 0 && F <= p.num_pages && all.q <= p.total_q &&
                      F + all.give <= p.num_pages && all.take <= F + all.give;
    // (32 bits hold what follows once it is good)
    for (int b = b0; b < b1; ++b) {
        const int q = q_pre[b], t = take[b], g = give[b];
        q_pre[b] = static_cast<int>(base.q);
        take[b] = static_cast<int>(base.take);
        give[b] = static_cast<int>(base.give);
        base.q += q;
        base.take += t;
        base.give += g;
    }
    if (tid == 0) {
        q_pre[p.B] = good ? static_cast<int>(all.q) : 0;
        take[p.B] = static_cast<int>(all.take);
        give[p.B] = static_cast<int>(all.give);
    }
    __syncthreads();
    // (drawn as soon as the whole CTA has used the lengths and the count; the answer
    // takes a while)
    unsigned drawn = 0;
    if (gridDim.x > 1 && tid == 0) {
        __threadfence();
        drawn = atomicAdd(p.ws + kStepTicket, 1u);
    }
    const int N = good ? static_cast<int>(all.take) : 0, R = good ? static_cast<int>(all.give) : 0, rows = q_pre[p.B];
    auto after_of = [&](int b) {
        return max((keep_s[b] + q_pre[b + 1] - q_pre[b] + p.page_size - 1) >> p.page_shift, p.shared_pages);
    };
    // the g-th page given back, and the k-th taken
    auto given = [&](int g) {
        const int b = share_of(give, p.B, g);
        return p.page_table[static_cast<size_t>(b) * p.max_pages + after_of(b) + g - give[b]];
    };
    auto taken = [&](int k) { return k < R ? given(k) : p.free_pages[F + R - 1 - k]; };

    const int threads = gridDim.x * THREADS, at = blockIdx.x * THREADS + tid;
    for (int g = at; g < R; g += threads) {      // (nobody reads the stack past F)
        const int id = given(g);
        if (id < 0 || id >= p.num_pages) report_sequence(p.ws, share_of(give, p.B, g));
        p.free_pages[F + R - 1 - g] = id;
    }
    for (int k = at; k < N; k += threads) {
        const int b = share_of(take, p.B, k), id = taken(k);
        if (id < 0 || id >= p.num_pages) report_sequence(p.ws, b);
        p.page_table[static_cast<size_t>(b) * p.max_pages + before_s[b] + k - take[b]] = id;
    }
    for (long long t0 = static_cast<long long>(at) * kSlotRows; (p.slots || p.positions) && t0 < p.total_q;
         t0 += static_cast<long long>(threads) * kSlotRows) {
        long long slot[kSlotRows];
        int pos[kSlotRows];
        int b = -1, last = -1, id = -1;          // the entry of the row before, and its page
#pragma unroll
        for (int e = 0; e < kSlotRows; ++e) {
            slot[e] = -1;
            pos[e] = 0;
            if (t0 + e >= rows) continue;
            const int t = static_cast<int>(t0) + e;
            if (b < 0 || t >= q_pre[b + 1]) {
                b = share_of(q_pre, p.B, t);
                last = -1;
            }
            pos[e] = keep_s[b] + (t - q_pre[b]);
            const int entry = pos[e] >> p.page_shift;
            if (entry != last)
                id = entry < before_s[b] ? p.page_table[static_cast<size_t>(b) * p.max_pages + entry]
                                         : taken(take[b] + entry - before_s[b]);
            last = entry;
            if (id >= 0 && id < p.num_pages)
                slot[e] = (static_cast<long long>(id) << p.page_shift) + (pos[e] & (p.page_size - 1));
            else
                report_sequence(p.ws, b);
        }
        if (wide && t0 + kSlotRows <= p.total_q) {
            if (p.slots) {
                reinterpret_cast<longlong2*>(p.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
                reinterpret_cast<longlong2*>(p.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
            }
            if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int e = 0; e < kSlotRows; ++e) {
                if (t0 + e >= p.total_q) break;
                if (p.slots) p.slots[t0 + e] = slot[e];
                if (p.positions) p.positions[t0 + e] = pos[e];
            }
        }
    }

    // who was last to read writes in place
    if (gridDim.x > 1) {
        if (tid == 0) {
            __threadfence();
            ticket = drawn;
        }
        __syncthreads();
        if (ticket != gridDim.x - 1) return;
        if (tid == 0) p.ws[kStepTicket] = 0;
    }
    for (int b = b0; b < b1; ++b) {
        p.q_start[b] = good ? q_pre[b] : 0;
        if (good)
            p.kv_len_out[b] = keep_s[b] + (q_pre[b + 1] - q_pre[b]);
        else if (p.kv_len_out != p.kv_len)
            p.kv_len_out[b] = p.kv_len[b];
    }
    if (tid == 0) {
        p.q_start[p.B] = rows;
        p.free_count_out[0] = F + R - N;
        if (!good) {
            // the sequence whose numbers do not fit, or at which the rows, the stack or its pages run out
            int b = first_bad;
            if (b == INT_MAX) {
                long long q = 0, took = 0, gave = F;
                for (b = 0; b < p.B - 1 && F >= 0 && F <= p.num_pages; ++b) {
                    const StepSeq s = step_sequence(p, b);
                    q += s.count;
                    took += max(s.after - s.before, 0);
                    gave += max(s.before - s.after, 0);
                    if (q > p.total_q || took > F + all.give || gave > p.num_pages) break;
                }
            }
            report_sequence(p.ws, b);
        }
    }
}

}  // namespace

cudaError_t launch_paged_step(const StepParams& p, cudaStream_t s) {
    const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
    const long long rows = p.slots || p.positions ? p.total_q : p.B;
    const unsigned ctas = static_cast<unsigned>(std::min<long long>((rows + kRowsEach - 1) / kRowsEach, 4 * device_sm_count()));
    const size_t smem = 4u * (5u * p.B + 3u);
    // few sequences and rows: a small block starts and scans sooner (64 sequences with a
    // token each 5.2 us, 5.6 with 512 threads; 256 of them 5.9 and 6.4; one 2.7 and 3.1)
    return p.B <= 256 && rows <= 1024
               ? paged_launch(paged_step_kernel<256>, dim3(std::max(ctas, 1u)), 256, smem, true, s, p, wide)
               : paged_launch(paged_step_kernel<512>, dim3(std::max(ctas, 1u)), 512, smem, true, s, p, wide);
}

}  // namespace fa
