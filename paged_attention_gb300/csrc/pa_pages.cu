// pa_pages.cu -- pages for the new tokens of a step and the maps of its rows;
// pages of tokens that go, back on the free stack.
//
//   need_b = ceil((len_b + q_b) / ps) - ceil(len_b / ps)
//   the j-th new page of sequence b is free[F - 1 - (sum of need before b) - j]
//
// Everything follows from two prefix sums over the sequences, so every CTA takes
// them itself (a few KB of lengths from L2) and then its share of the rows: one
// launch, and no CTA waits for another.  A row finds its sequence by a search in
// the prefix sums in shared memory.  Nothing that a CTA reads is written by
// another: the stack is read below its top only, and the table at pages that were
// there before.  Bound by latency (a chain of length, sums, page number, slot): both
// calls of a decode step of 64 sequences 5.3 us in a graph, of 190149 new rows of 256
// prompts 7.2, 12 from the host.
#include <algorithm>

#include "pa_step_common.cuh"

namespace pa {

namespace {

constexpr int kThreads = 512;            // and sequences of a round
constexpr int kWarps = kThreads / 32;
constexpr int kItems = 4;                // rows or pages of a thread, before there are more CTAs

// Inclusive sum over the CTA's threads, and the total.
template <typename T>
__device__ __forceinline__ T cta_inclusive(T v, T* warp_sum, T& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();                     // the last sum's readers are done
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    return v + before;
}

// The first i with sums[i] > x (sums ascend; the last exceeds x).
template <typename T>
__device__ __forceinline__ int first_above(const T* sums, T x) {
    int i = 0;
#pragma unroll
    for (int o = kThreads / 2; o > 0; o >>= 1)
        if (sums[i + o - 1] <= x) i += o;
    return i;
}

__device__ __forceinline__ int pages_of(const CacheGeom& g, int tokens) {
    return (int)(((int64_t)tokens + g.ps - 1) >> g.ps_shift);
}

__device__ __forceinline__ int free_pages_of(const CacheGeom& g, const int32_t* count, bool report,
                                             int32_t* err) {
    const int f = *count;
    if (f >= 0 && f <= g.num_pages) return f;
    if (report) flag_error(err, PA_DEV_BAD_LENGTHS);
    return f < 0 ? 0 : g.num_pages;
}

// What a row has to know of a sequence of the round.
struct SeqOf {
    int32_t len, held;       // tokens and pages it had; held < 0: its rows are padding
    int64_t first;           // where its new pages begin, counted from the top of the stack
};

__global__ void __launch_bounds__(kThreads)
take_kernel(const CacheGeom g, const int32_t* __restrict__ seq_lens,
            const int32_t* __restrict__ q_lens, int32_t* table,
            const int32_t* __restrict__ free_pages, const int32_t* __restrict__ free_count,
            int32_t* __restrict__ context_lens, int32_t* __restrict__ row_seq,
            int32_t* __restrict__ positions, int32_t* __restrict__ slots,
            int32_t* __restrict__ free_left, int32_t* err) {
    __shared__ int64_t s_sum[kWarps];
    __shared__ int32_t s_qsum[kWarps];
    __shared__ int32_t s_end[kThreads];  // rows up to and with each sequence
    __shared__ SeqOf s_seq[kThreads];
    grid_dependency_wait();
    const bool lead = blockIdx.x == 0;
    const int tid = threadIdx.x;
    const int F = free_pages_of(g, free_count, lead && tid == 0, err);
    int64_t need0 = 0;                   // pages that the sequences before the round need
    int64_t taken = 0;                   // pages that the thread's own sequences got
    int row0 = 0;
    for (int b0 = 0; b0 < g.B; b0 += kThreads) {
        const int b = b0 + tid;
        const bool there = b < g.B;
        const int len = there ? seq_lens[b] : 0, q = there ? q_lens[b] : 0;
        bool ok = there && len >= 0 && q >= 0 && q <= g.max_q_len && (int64_t)len + q <= g.max_ctx;
        int rows;
        const int end = row0 + cta_inclusive(there ? clamp_q(g, q) : 0, s_qsum, rows);
        ok = ok && end <= g.total_q;
        const int held = ok ? pages_of(g, len) : 0;
        const int need = ok ? pages_of(g, len + q) - held : 0;
        int64_t all;
        const int64_t upto = need0 + cta_inclusive((int64_t)need, s_sum, all);
        const bool granted = ok && (need == 0 || upto <= F);
        if (granted) taken += need;
        s_end[tid] = end;
        s_seq[tid] = {len, granted ? held : -1, upto - need};
        if (lead && there) {
            context_lens[b] = granted ? len + q : max(0, min(len, g.max_ctx));
            if (!ok) flag_error(err, PA_DEV_BAD_LENGTHS);
            if (ok && !granted) flag_error(err, PA_DEV_NO_PAGES);
        }
        __syncthreads();
        // (bad lengths add up to as much as 2^31 - 1 rows: one step further needs the 32nd bit)
        for (uint32_t i = blockIdx.x * kThreads + tid;
             i < (uint32_t)rows && row0 + i < (uint32_t)g.total_q; i += gridDim.x * kThreads) {
            const int r = (int)(row0 + i);
            const int s = first_above(s_end, r);
            const SeqOf x = s_seq[s];
            int seq = -1, pos = 0, slot = -1;
            if (x.held >= 0) {
                seq = b0 + s;
                // (the rows of a sequence end where the prefix sum does)
                const int begin = s > 0 ? s_end[s - 1] : row0;
                pos = x.len + (r - begin);
                const int pi = pos >> g.ps_shift;
                int32_t* entry = table + (int64_t)seq * g.mpps + pi;
                int page;
                if (pi < x.held) {
                    page = *entry;
                } else {
                    page = free_pages[F - 1 - (x.first + (pi - x.held))];
                    if ((pos & (g.ps - 1)) == 0) *entry = page;
                }
                if ((uint32_t)page < (uint32_t)g.num_pages)
                    slot = (int)(((int64_t)page << g.ps_shift) + (pos & (g.ps - 1)));
                else
                    flag_error(err, PA_DEV_BAD_PAGE);
            }
            row_seq[r] = seq;
            positions[r] = pos;
            slots[r] = slot;
        }
        row0 += rows;
        need0 += all;
        __syncthreads();                 // the round's rows are done with s_end and s_seq
    }
    for (uint32_t r = row0 + blockIdx.x * kThreads + tid; r < (uint32_t)g.total_q;
         r += gridDim.x * kThreads) {
        row_seq[r] = -1;
        positions[r] = 0;
        slots[r] = -1;
    }
    if (lead) {
        int64_t all;
        cta_inclusive(taken, s_sum, all);
        if (tid == 0) *free_left = F - (int)all;
    }
}

__global__ void __launch_bounds__(kThreads)
return_kernel(const CacheGeom g, const int32_t* __restrict__ seq_lens,
              const int32_t* __restrict__ keep_lens, const int32_t* __restrict__ table,
              int32_t* __restrict__ free_pages, const int32_t* __restrict__ free_count,
              int32_t* __restrict__ free_left, int32_t* err) {
    __shared__ int64_t s_sum[kWarps];
    __shared__ int32_t s_end[kThreads];  // pages up to and with each sequence of the round
    __shared__ int32_t s_first[kThreads];
    grid_dependency_wait();
    const bool lead = blockIdx.x == 0;
    const int tid = threadIdx.x;
    const int F = free_pages_of(g, free_count, lead && tid == 0, err);
    int64_t at = F;                      // where the round's pages go
    for (int b0 = 0; b0 < g.B; b0 += kThreads) {
        const int b = b0 + tid;
        int first = 0, n = 0;
        if (b < g.B) {
            const int len = seq_lens[b], keep = keep_lens[b];
            if (keep >= 0 && keep <= len && len <= g.max_ctx) {
                first = pages_of(g, keep);
                n = pages_of(g, len) - first;
            } else if (lead) {
                flag_error(err, PA_DEV_BAD_LENGTHS);
            }
        }
        int64_t all;
        // (a round's pages: at most 512 sequences of 2^26 pages)
        const int64_t end = cta_inclusive((int64_t)n, s_sum, all);
        s_end[tid] = (int32_t)min(end, (int64_t)0x7fffffff);
        s_first[tid] = first;
        __syncthreads();
        // what does not fit the stack is not moved
        const int64_t room = max((int64_t)0, (int64_t)g.num_pages - at);
        if (all > room && lead && tid == 0) flag_error(err, PA_DEV_BAD_LENGTHS);
        const int m = (int)min(all, room);
        for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < m;
             i += (int64_t)gridDim.x * kThreads) {
            const int s = first_above(s_end, (int32_t)i);
            const int pi = s_first[s] + ((int)i - (s > 0 ? s_end[s - 1] : 0));
            const int page = table[(int64_t)(b0 + s) * g.mpps + pi];
            const bool ok = (uint32_t)page < (uint32_t)g.num_pages;
            if (!ok) flag_error(err, PA_DEV_BAD_PAGE);
            free_pages[at + i] = ok ? page : -1;
        }
        at += all;
        __syncthreads();
    }
    if (lead && tid == 0) *free_left = (int)min(at, (int64_t)g.num_pages);
}

}  // namespace

cudaError_t launch_pages_take(const CacheGeom& g, const int32_t* seq_lens, const int32_t* q_lens,
                              int32_t* table, const int32_t* free_pages, const int32_t* free_count,
                              int32_t* context_lens, int32_t* row_seq, int32_t* positions,
                              int32_t* slots, int32_t* free_left, int32_t* err, int sms,
                              cudaStream_t stream) {
    const int64_t per = (int64_t)kThreads * kItems;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(sms, (g.total_q + per - 1) / per));
    return launch_dependent(take_kernel, dim3(grid), dim3(kThreads), 0, stream, g, seq_lens, q_lens,
                            table, free_pages, free_count, context_lens, row_seq, positions, slots,
                            free_left, err);
}

cudaError_t launch_pages_return(const CacheGeom& g, const int32_t* seq_lens,
                                const int32_t* keep_lens, const int32_t* table,
                                int32_t* free_pages, const int32_t* free_count, int32_t* free_left,
                                int32_t* err, int sms, cudaStream_t stream) {
    // (how many pages go back is known on the device only: at most the pool's)
    const int64_t per = (int64_t)kThreads * kItems;
    const int64_t most = std::min<int64_t>(g.num_pages, (int64_t)g.B * g.mpps);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(sms, (most + per - 1) / per));
    return launch_dependent(return_kernel, dim3(grid), dim3(kThreads), 0, stream, g, seq_lens,
                            keep_lens, table, free_pages, free_count, free_left, err);
}

}  // namespace pa
