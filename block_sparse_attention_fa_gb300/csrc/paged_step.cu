// paged_step.cu -- a step's page tables, offsets and slots from its sequences'
// lengths (fa_paged_step).
//
// With before_b and after_b the entries of sequence b's row of the page table
// before and behind the step (at least the shared ones), three exclusive sums
// over the sequences place everything:
//     Q of new_len, G of max(before - after, 0), T of max(after - before, 0).
// The g-th page given back (sequences and entries ascending) goes to place
// F + R - 1 - g of the stack of free pages (F pages before, R given in all),
// and the k-th page taken is the one at place F + R - 1 - k.  Row t of the step
// belongs to the sequence with Q_b <= t < Q_b + new_b.
//
// The lengths of 2048 sequences are 24 KB and a step moves few pages, so that
// what this costs is latency: one CTA of 1024 threads does it all, in shared
// memory, and the page numbers of a batch of prompts (6000 pages for 100000
// tokens) are a few rounds of it.  The slots of many rows (12 bytes each) are
// memory traffic: from kRowsHere rows on they are a second launch of as many
// CTAs as they fill.
//
// Nothing is written before every number has been checked, the pages that move
// among them; one that does not fit makes the step an empty one.
#include <algorithm>

#include "paged.cuh"

namespace fa {
namespace {

constexpr int kStepThreads = 1024;
constexpr int kRowsHere = 4 * kStepThreads;
constexpr int kSlotThreads = 256, kSlotRows = 4;       // rows of a thread, adjacent ones

// The last of the B sequences with pre[b] <= x (pre[0] = 0 <= x < pre[B]): the one whose share holds x.
__device__ __forceinline__ int share_of(const int* pre, int B, int x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

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

__device__ __forceinline__ bool is_page(const StepParams& p, int id) { return id >= 0 && id < p.num_pages; }

// The slot and the position of row t, of sequence b whose first row is q0 and
// first new position `keep`.
__device__ __forceinline__ void place_row(const StepParams& p, int t, int b, int q0, int keep, long long& slot, int& pos) {
    pos = keep + (t - q0);
    const int page = p.page_table[static_cast<size_t>(b) * p.max_pages + (pos >> p.page_shift)];
    slot = (static_cast<long long>(page) << p.page_shift) + (pos & (p.page_size - 1));
}

__global__ void __launch_bounds__(kStepThreads) paged_step_kernel(const StepParams p, bool rows_here) {
    extern __shared__ int step_smem[];
    int* const q_pre = step_smem;
    int* const take = q_pre + p.B + 1;
    int* const give = take + p.B + 1;
    __shared__ int warp_sums[kStepThreads / 32];
    __shared__ unsigned long long sums[3];
    __shared__ int first_bad, bad_seq;
    const int tid = threadIdx.x;
    if (tid < 3) sums[tid] = 0;
    if (tid == 0) {
        first_bad = INT_MAX;
        bad_seq = INT_MAX;
    }
    __syncthreads();
    pdl_wait_previous();
    pdl_launch_next();
    for (int b = tid; b < p.B; b += kStepThreads) {
        const StepSeq s = step_sequence(p, b);
        if (!s.fits) atomicMin(&first_bad, b);
        q_pre[b] = s.count;
        take[b] = max(s.after - s.before, 0);
        give[b] = max(s.before - s.after, 0);
        // (sums of integers: in any order the same)
        if (q_pre[b]) atomicAdd(&sums[0], static_cast<unsigned long long>(q_pre[b]));
        if (take[b]) atomicAdd(&sums[1], static_cast<unsigned long long>(take[b]));
        if (give[b]) atomicAdd(&sums[2], static_cast<unsigned long long>(give[b]));
    }
    const int F = p.free_count[0];
    __syncthreads();
    const bool counted = F >= 0 && F <= p.num_pages && sums[0] <= static_cast<unsigned long long>(p.total_q) &&
                         F + sums[2] <= static_cast<unsigned long long>(p.num_pages);
    const bool enough = sums[1] <= F + sums[2];
    bool good = first_bad == INT_MAX && counted && enough;
    const int N = good ? static_cast<int>(sums[1]) : 0, R = good ? static_cast<int>(sums[2]) : 0;
    if (good) {
        block_prefix<kStepThreads>(p.B, q_pre, warp_sums, [&](int b) { return q_pre[b]; });
        if (N) block_prefix<kStepThreads>(p.B, take, warp_sums, [&](int b) { return take[b]; });
        if (R) block_prefix<kStepThreads>(p.B, give, warp_sums, [&](int b) { return give[b]; });
        // the pages that move
        for (int g = tid; g < R; g += kStepThreads) {
            const int b = share_of(give, p.B, g);
            const StepSeq s = step_sequence(p, b);
            if (!is_page(p, p.page_table[static_cast<size_t>(b) * p.max_pages + s.after + g - give[b]])) atomicMin(&bad_seq, b);
        }
        for (int k = R + tid; k < N; k += kStepThreads)
            if (!is_page(p, p.free_pages[F + R - 1 - k])) atomicMin(&bad_seq, share_of(take, p.B, k));
        __syncthreads();
        good = bad_seq == INT_MAX;
    }
    if (!good) {
        if (tid == 0) {
            // the sequence whose numbers do not fit, or at which the rows, the stack or its pages run out
            int at = min(first_bad, bad_seq);
            if (at == INT_MAX) {
                const long long given = static_cast<long long>(F) + static_cast<long long>(sums[2]);
                long long rows = 0, took = 0, gave = F;
                for (at = 0; at < p.B - 1 && F >= 0 && F <= p.num_pages; ++at) {
                    const StepSeq s = step_sequence(p, at);
                    rows += s.count;
                    took += max(s.after - s.before, 0);
                    gave += max(s.before - s.after, 0);
                    if (rows > p.total_q || took > given || gave > p.num_pages) break;
                }
            }
            report_sequence(p.ws, at);
            p.free_count_out[0] = F;
        }
        for (int b = tid; b <= p.B; b += kStepThreads) {
            p.q_start[b] = 0;
            if (b < p.B) p.kv_len_out[b] = p.kv_len[b];
        }
        for (int t = tid; rows_here && t < p.total_q; t += kStepThreads) {
            if (p.slots) p.slots[t] = -1;
            if (p.positions) p.positions[t] = 0;
        }
        return;
    }
    for (int g = tid; g < R; g += kStepThreads) {
        const int b = share_of(give, p.B, g);
        const StepSeq s = step_sequence(p, b);
        p.free_pages[F + R - 1 - g] = p.page_table[static_cast<size_t>(b) * p.max_pages + s.after + g - give[b]];
    }
    __syncthreads();
    for (int k = tid; k < N; k += kStepThreads) {
        const int b = share_of(take, p.B, k);
        const StepSeq s = step_sequence(p, b);
        p.page_table[static_cast<size_t>(b) * p.max_pages + s.before + k - take[b]] = p.free_pages[F + R - 1 - k];
    }
    __syncthreads();
    const int rows = q_pre[p.B];
    for (int t = tid; rows_here && t < p.total_q; t += kStepThreads) {
        long long slot = -1;
        int pos = 0;
        if (t < rows) {
            const int b = share_of(q_pre, p.B, t);
            place_row(p, t, b, q_pre[b], p.keep_len[b], slot, pos);
        }
        if (p.slots) p.slots[t] = slot;
        if (p.positions) p.positions[t] = pos;
    }
    // (kv_len and free_count may be written in place: every thread is past their last reading)
    __syncthreads();
    for (int b = tid; b <= p.B; b += kStepThreads) {
        p.q_start[b] = q_pre[b];
        if (b < p.B) p.kv_len_out[b] = p.keep_len[b] + (q_pre[b + 1] - q_pre[b]);
    }
    if (tid == 0) p.free_count_out[0] = F + R - N;
}

// Slots and positions of many rows, from what the kernel above has written.
__global__ void __launch_bounds__(kSlotThreads) paged_slots_kernel(const StepParams p, bool wide) {
    extern __shared__ int step_smem[];
    pdl_wait_previous();
    pdl_launch_next();
    for (int b = threadIdx.x; b <= p.B; b += kSlotThreads) step_smem[b] = p.q_start[b];
    __syncthreads();
    const int* const q_pre = step_smem;
    const int rows = q_pre[p.B];
    const long long t0 = (static_cast<long long>(blockIdx.x) * kSlotThreads + threadIdx.x) * kSlotRows;
    if (t0 >= p.total_q) return;
    long long slot[kSlotRows];
    int pos[kSlotRows];
    int b = -1, keep = 0;
#pragma unroll
    for (int e = 0; e < kSlotRows; ++e) {
        const int t = static_cast<int>(min(t0 + e, static_cast<long long>(p.total_q) - 1));
        slot[e] = -1;
        pos[e] = 0;
        if (t >= rows) continue;
        if (b < 0 || t >= q_pre[b + 1]) {
            b = share_of(q_pre, p.B, t);
            keep = p.kv_len_out[b] - (q_pre[b + 1] - q_pre[b]);
        }
        place_row(p, t, b, q_pre[b], keep, slot[e], pos[e]);
    }
    if (wide && t0 + kSlotRows <= p.total_q) {
        if (p.slots) {
            reinterpret_cast<longlong2*>(p.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
            reinterpret_cast<longlong2*>(p.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
        }
        if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        return;
    }
#pragma unroll
    for (int e = 0; e < kSlotRows; ++e) {
        if (t0 + e >= p.total_q) break;
        if (p.slots) p.slots[t0 + e] = slot[e];
        if (p.positions) p.positions[t0 + e] = pos[e];
    }
}

}  // namespace

cudaError_t launch_paged_step(const StepParams& p, cudaStream_t s) {
    const bool wants = (p.slots || p.positions) && p.total_q > 0, here = p.total_q <= kRowsHere;
    cudaError_t e = paged_launch(paged_step_kernel, dim3(1), kStepThreads, 3u * 4u * (p.B + 1), true, s, p, here && wants);
    if (e != cudaSuccess || here || !wants) return e;
    const int per = kSlotThreads * kSlotRows;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) & 15) == 0;
    return paged_launch(paged_slots_kernel, dim3((p.total_q + per - 1LL) / per), kSlotThreads, 4u * (p.B + 1), true, s, p, wide);
}

}  // namespace fa
