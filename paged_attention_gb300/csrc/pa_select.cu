// pa_select.cu -- for every row and KV head, the pages with the highest bound on
// a logit.
//
//   score = 2^e_page max_h 2^e_h sum_d max(q8 hi, q8 lo)
//         = 2^e_page max_h 2^e_h [max(q8, 0), min(q8, 0)] . [hi, lo]
//
// so a group's scores are products of 8-bit matrices: 16 pages by 8 heads a
// product (mma m16n8k32, 32-bit whole sums: exact, in any order).  The contraction's
// order being free, a lane takes 16 bytes of a page's bounds as they lie.
//
// One cluster of CTAs a row and KV head, each with a part of the pages: scores
// stay in shared memory as order-preserving integers, the budget-th largest is
// found by a radix select, eight bits a pass, whose histograms the CTAs add up
// through distributed shared memory, and every CTA lists its part in order.  As many
// CTAs a cluster as it takes to fill the GPU.  Bound by HBM (2 D bytes a page and
// head) for many rows or long contexts, else by the latency of the passes.
#include <algorithm>

#include "pa_step_common.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxGroup = 64;    // q heads of a KV head
constexpr int kBins = 256;
static_assert(kBins == kThreads, "a thread a bin");

// D = A * B of 8-bit whole numbers, + D
__device__ __forceinline__ void mma_s8_16832(int* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ int ld_dsm_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Larger scores (never NaN) get larger keys, all above 0.
__device__ __forceinline__ uint32_t key_of(float score) {
    const uint32_t u = __float_as_uint(score + 0.f);   // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Codes of a query row's words (two elements each) with 2^-e as factor.
__device__ __forceinline__ uint32_t q_codes(uint32_t w0, uint32_t w1, float inv) {
    uint32_t out = 0;
    const float x[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u),
                        __uint_as_float(w1 << 16), __uint_as_float(w1 & 0xffff0000u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = x[i] == x[i] ? fminf(fmaxf(rintf(x[i] * inv), -127.f), 127.f) : 0.f;
        out |= (uint32_t)((int)y & 255) << (8 * i);
    }
    return out;
}

template <int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ SelectParams P) {
    constexpr int J = 2 * D / 64;                // 64-byte runs of a page's bounds
    constexpr int kQRow = 2 * D + 64;            // 8 lanes' 16 bytes (two rows) meet no bank twice
    extern __shared__ uint32_t s_key[];          // of the CTA's pages
    __shared__ __align__(16) uint8_t s_q[kMaxGroup * kQRow];
    __shared__ float s_factor[kMaxGroup];
    __shared__ uint32_t s_hist[4][kBins];        // of each pass
    __shared__ int s_count[2];                   // keys above, and at, the threshold
    __shared__ uint32_t s_warp[kWarps];
    __shared__ int2 s_part[kWarps];
    __shared__ uint32_t s_digit, s_left;
    const CacheGeom& g = P.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = P.cluster, rank = blockIdx.x % C, unit = blockIdx.x / C;
    const int t = unit / g.Hkv, hk = unit % g.Hkv;
    grid_dependency_wait();

    // (the cluster's CTAs leave together: they all look at the same row)
    const int b = P.row_seq[t], pos = P.positions[t];
    if (b < 0) return;
    if (b >= g.B || pos < 0 || pos >= g.max_ctx) {
        if (rank == 0 && hk == 0 && tid == 0) flag_error(P.err, PA_DEV_BAD_LENGTHS);
        return;
    }
    const int first = g.window > 0 ? max(0, pos - g.window + 1) >> g.ps_shift : 0;
    const int n = (pos >> g.ps_shift) + 1 - first;
    int32_t* out = P.selected + (int64_t)unit * P.budget;
    if (n <= P.budget) {
        for (int i = rank * kThreads + tid; i < P.budget; i += C * kThreads)
            out[i] = i < n ? first + i : -1;
        return;
    }

    // ---- the group's queries in 8 bits, positive and negative parts
    const int tiles = (g.G + 7) / 8;
    for (int h = warp; h < 8 * tiles; h += kWarps) {
        uint32_t w[D / 64];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) w[i] = 0u;
        if (h < g.G) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                P.q + ((int64_t)t * g.Hq + (int64_t)hk * g.G + h) * D);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                // (D = 64: a lane has a word, its neighbour the rest of its four codes)
                w[i] = src[lane * (D / 64) + i];
                const uint32_t x = w[i] & 0x7fffu, y = (w[i] >> 16) & 0x7fffu;
                top = max(top, max(x > 0x7f80u ? 0u : x, y > 0x7f80u ? 0u : y));   // NaN: none
            }
        }
        const uint32_t m = __reduce_max_sync(0xffffffffu, top);
        // least e with m <= 127 * 2^e = 1.984375 * 2^(e + 6)
        const int e = max(-50, min(50, (int)(m >> 7) - 133 + ((m & 127u) == 127u ? 1 : 0)));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t w0, w1;
        if constexpr (D == 128) {
            w0 = w[0];
            w1 = w[1];
        } else {
            w0 = __shfl_sync(0xffffffffu, w[0], 2 * (lane & 15));
            w1 = __shfl_sync(0xffffffffu, w[0], 2 * (lane & 15) + 1);
        }
        const uint32_t code = q_codes(w0, w1, inv);
        if (D == 128 || lane < 16) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(s_q + h * kQRow);
            dst[lane] = __vmaxs4(code, 0u);
            dst[D / 4 + lane] = __vmins4(code, 0u);
        }
        if (lane == 0) s_factor[h] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
    for (int i = tid; i < 4 * kBins; i += kThreads) (&s_hist[0][0])[i] = 0u;
    __syncthreads();

    // ---- scores of the CTA's pages [lo, lo + m)
    const int part = (n + C - 1) / C, lo = min(n, rank * part), m = min(part, n - lo);
    const int32_t* row = P.table + (int64_t)b * g.mpps + first + lo;
    const int gr = lane >> 2, t4 = lane & 3;
    bool none = false;
    for (int i0 = 16 * warp; i0 < m; i0 += 16 * kWarps) {
        int64_t at[2];
        float sc[2];
        bool ok[2];
        uint4 a[2][J];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + gr + 8 * r;
            const int page = row[min(i, m - 1)];
            ok[r] = (uint32_t)page < (uint32_t)g.num_pages;
            none |= !ok[r] && i < m;
            at[r] = (int64_t)(ok[r] ? page : 0) * g.Hkv + hk;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sc[r] = P.scale[at[r]];
            const uint4* src = reinterpret_cast<const uint4*>(P.bounds + at[r] * 2 * D) + t4;
#pragma unroll
            for (int j = 0; j < J; ++j) a[r][j] = __ldg(src + 4 * j);
        }
        float best[2] = {-INFINITY, -INFINITY};
        for (int nt = 0; nt < tiles; ++nt) {
            int d[4] = {0, 0, 0, 0};
            const uint8_t* qr = s_q + (8 * nt + gr) * kQRow + 16 * t4;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint4 q = *reinterpret_cast<const uint4*>(qr + 64 * j);
                mma_s8_16832(d, a[0][j].x, a[1][j].x, a[0][j].y, a[1][j].y, q.x, q.y);
                mma_s8_16832(d, a[0][j].z, a[1][j].z, a[0][j].w, a[1][j].w, q.z, q.w);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int h = 8 * nt + 2 * t4 + (x & 1);
                if (h < g.G) best[x >> 1] = fmaxf(best[x >> 1], (float)d[x] * s_factor[h]);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
            const int i = i0 + gr + 8 * r;
            if (t4 == 0 && i < m) {
                const bool kept = lo + i < P.num_first || lo + i >= n - P.num_recent;
                s_key[i] = kept ? 0xffffffffu : ok[r] ? key_of(best[r] * sc[r]) : 0u;
            }
        }
    }
    if (none) flag_error(P.err, PA_DEV_BAD_PAGE);
    __syncthreads();

    // ---- the budget-th largest key of the cluster's
    uint32_t prefix = 0, left = (uint32_t)P.budget;   // rank from the top among equal prefixes
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int i0 = 32 * warp; i0 < m; i0 += kThreads) {
            const int i = i0 + lane;
            const uint32_t x = i < m ? s_key[i] : 0u;
            const bool in = i < m && (pass == 0 || x >> (shift + 8) == prefix);
            const uint32_t digit = in ? (x >> shift) & 255u : 256u;
            // (scores crowd into few bins: one addition for all lanes of a bin)
            const uint32_t same = __match_any_sync(0xffffffffu, digit);
            if (in && __ffs(same) - 1 == lane) atomicAdd(&s_hist[pass][digit], __popc(same));
        }
        uint32_t mine;
        __syncwarp();
        if (C > 1) {
            cluster_sync_all();
            mine = 0;
            const uint32_t addr = smem_u32(&s_hist[pass][tid]);
            for (int c = 0; c < C; ++c) mine += (uint32_t)ld_dsm_s32(mapa_shared(addr, c));
        } else {
            __syncthreads();
            mine = s_hist[pass][tid];
        }
        // keys in this bin and above: bins in descending order along the threads' mirror
        uint32_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_down_sync(0xffffffffu, sum, o);
            if (lane + o < 32) sum += y;
        }
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w > warp) sum += s_warp[w];
        if (sum >= left && sum - mine < left) {       // one thread: the bins are ordered
            s_digit = (uint32_t)tid;
            s_left = left - (sum - mine);
        }
        __syncthreads();
        prefix = prefix << 8 | s_digit;
        left = s_left;
    }
    const uint32_t limit = prefix;                     // `left` of the keys equal to it are kept

    // ---- how many of its keys each CTA lists, and each of its warps
    const int seg = (m + kThreads - 1) / kThreads * 32;        // of a warp
    const int w0 = min(m, warp * seg), w1 = min(m, w0 + seg);
    int above = 0, equal = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t x = i < w1 ? s_key[i] : 0u;
        above += __popc(__ballot_sync(0xffffffffu, i < w1 && x > limit));
        equal += __popc(__ballot_sync(0xffffffffu, i < w1 && x == limit));
    }
    if (lane == 0) s_part[warp] = make_int2(above, equal);
    __syncthreads();
    int before_above = 0, before_equal = 0, all_above = 0, all_equal = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            before_above += s_part[w].x;
            before_equal += s_part[w].y;
        }
        all_above += s_part[w].x;
        all_equal += s_part[w].y;
    }
    if (C > 1) {
        if (tid == 0) {
            s_count[0] = all_above;
            s_count[1] = all_equal;
        }
        __syncwarp();
        cluster_sync_all();
        for (int c = 0; c < rank; ++c) {
            before_above += ld_dsm_s32(mapa_shared(smem_u32(&s_count[0]), c));
            before_equal += ld_dsm_s32(mapa_shared(smem_u32(&s_count[1]), c));
        }
    }
    // ---- list them: a key's place is the number of listed ones before it
    const int take = (int)left;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t x = i < w1 ? s_key[i] : 0u;
        const uint32_t up = __ballot_sync(0xffffffffu, i < w1 && x > limit);
        const uint32_t eq = __ballot_sync(0xffffffffu, i < w1 && x == limit);
        const uint32_t below = (1u << lane) - 1u;
        const int eq_rank = before_equal + __popc(eq & below);
        const int place = before_above + __popc(up & below) + min(take, eq_rank);
        if ((up >> lane & 1u) || ((eq >> lane & 1u) && eq_rank < take)) out[place] = first + lo + i;
        before_above += __popc(up);
        before_equal += __popc(eq);
    }
    __syncwarp();
    if (C > 1) cluster_sync_all();                     // nobody leaves while it is read
}

template <int D>
cudaError_t launch(const SelectParams& P, int smem, int most, cudaStream_t stream) {
    const cudaError_t e = allow_smem<select_kernel<D>>(most);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(P.g.total_q * P.g.Hkv * P.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)P.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<D>, P);
}

}  // namespace

// Pages of a context that a cluster's shared memory has room for.
static_assert(PA_MAX_SELECT_PAGES <= kMaxCluster * 32768, "keys of a CTA");

cudaError_t launch_select(const SelectParams& P0, int sms, cudaStream_t stream) {
    SelectParams P = P0;
    const int pages = (int)(((int64_t)P.g.max_ctx + P.g.ps - 1) >> P.g.ps_shift);
    // CTAs of a cluster: until the GPU has two an SM, none with under 64 pages; a part's keys
    // must fit
    int c = 1;
    const int64_t units = (int64_t)P.g.total_q * P.g.Hkv;
    while (c < kMaxCluster && ((units * c < 2 * sms && pages >= 128 * c) || pages > 32768 * c)) c *= 2;
    P.cluster = c;
    const int smem = ((pages + c - 1) / c) * 4;
    return P.g.D == 128 ? launch<128>(P, smem, 32768 * 4, stream)
                        : launch<64>(P, smem, 32768 * 4, stream);
}

}  // namespace pa
