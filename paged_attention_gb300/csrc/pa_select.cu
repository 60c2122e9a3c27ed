// pa_select.cu -- for every row and KV head, the pages with the highest bound on
// a logit.
//
//   score = 2^e_page max_h 2^e_h sum_d (q8 > 0 ? q8 hi : q8 lo)
//         = 2^e_page max_h 2^e_h [max(q8, 0), min(q8, 0)] . [hi, lo]
//
// so a group's scores are products of whole-number matrices: 16 pages by 8 heads a
// product.  They are taken in f16 (mma m16n8k16, fp32 sums): products of 8-bit integers
// are slow here (with them the scores of 64 rows took 2 us more than their loads alone).  A code
// c becomes the f16 1152 + c by one permutation of bytes a pair; 64 codes a sum stay
// below 2^24, so every sum is exact, and 1152 times the sum of q8 is taken off it.  The
// contraction's order being free, a lane takes 16 bytes of a page's bounds as they lie.
//
// One cluster of CTAs a row and KV head, each scoring a part of the pages; the scores go,
// as order-preserving integers, to the first CTA's shared memory, which finds the
// budget-th largest by a radix select over the bits in which they differ, eleven a pass,
// until a pass decides all, and lists the pages in order.  As many CTAs a cluster as it
// takes to fill the GPU.  Bound by the latency of its steps (row, page numbers, bounds,
// two or three passes), by HBM (2 D bytes a page and head) for many rows of long contexts.
// 64 rows of up to 459 pages, 8 heads: 10.4 us; one row of 8192 pages 17, 5.5 of them the
// scores on 64 SMs (clusters of 12 CTAs, which are not portable: 16.2).  Slower here: fewer
// registers and more CTAs an SM (12.3 to 14.2 and 21 to 23), clusters of 16 (22: one of
// eight waits for the others), pages pruned by groups' largest scores (11.2 and 19).
#include <algorithm>

#include "pa_cache_mma.cuh"
#include "pa_step_common.cuh"

namespace pa {

namespace {

constexpr int kMaxCluster = 8;
constexpr float kBias = 1152.f;  // of a code's f16
constexpr int kMaxGroup = 64;    // q heads of a KV head
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kTile = 32;        // pages of a warp at a time: two products' rows

constexpr uint32_t kKept = 0xffffffffu;      // key of a page that is kept whatever its score

// A query row in shared memory: 2 D f16, and padding (so that rows begin on other banks)
constexpr int q_row_bytes(int D) { return 4 * D + 16; }

// Larger scores get larger keys, all above 0; NaN (a scale that no bounds were written
// for) the smallest.
__device__ __forceinline__ uint32_t key_of(float score) {
    if (score != score) return 0u;
    const uint32_t u = __float_as_uint(score + 0.f);   // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The two halves of a barrier over the cluster: this CTA has begun; all have.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// The codes of four elements (two words) of a query row, with 2^-e as factor.
__device__ __forceinline__ void q_codes(uint32_t w0, uint32_t w1, float inv, float* c) {
    const float x[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u),
                        __uint_as_float(w1 << 16), __uint_as_float(w1 & 0xffff0000u)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = x[i] == x[i] ? fminf(fmaxf(rintf(x[i] * inv), -127.f), 127.f) : 0.f;
}

// Four codes as f16 pairs, kBias above their values.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;          // 128 above
    lo = prmt(u, 0x64646464u, 0x4140u);          // 0x6400 is 1024
    hi = prmt(u, 0x64646464u, 0x4342u);
}

__device__ __forceinline__ void st_dsm_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int D, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads)
select_kernel(const __grid_constant__ SelectParams P) {
    constexpr int kWarps = kThreads / 32;
    constexpr int kMine = kBins / kThreads;      // bins of a thread
    static_assert(kMine % 4 == 0, "read four at a time");
    constexpr int J = 2 * D / 64;                // 64-byte runs of a page's bounds
    constexpr int RT = kTile / 8;                // page rows of a lane
    constexpr int kQRow = q_row_bytes(D);
    extern __shared__ __align__(16) uint8_t smem[];      // queries; the cluster's keys
    __shared__ float s_factor[kMaxGroup];
    __shared__ float s_bias[kMaxGroup][J];       // what the bias of the codes adds to a run's sum
    __shared__ __align__(16) uint32_t s_hist[2][kBins];    // of one pass and the next
    __shared__ uint32_t s_warp[kWarps];
    __shared__ uint2 s_range[kWarps];
    __shared__ int2 s_part[kWarps];
    __shared__ int3 s_found;
    const CacheGeom& g = P.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, t4 = lane & 3;
    const int C = P.cluster, rank = blockIdx.x % C, unit = blockIdx.x / C;
    const int t = unit / g.Hkv, hk = unit % g.Hkv;
    const int tiles = (g.G + 7) / 8;
    uint32_t* s_key = reinterpret_cast<uint32_t*>(smem + 8 * tiles * kQRow);
    for (int i = tid; i < 2 * kBins / 4; i += kThreads)
        reinterpret_cast<uint4*>(&s_hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    grid_dependency_wait();

    // a warp's head: lane l has the words l * D / 64 .. of its query row (0: no such head)
    uint32_t q_words[D / 64];
    auto load_q = [&](int h) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) q_words[i] = 0u;
        if (h < g.G) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                P.q + ((int64_t)t * g.Hq + (int64_t)hk * g.G + h) * D);
#pragma unroll
            for (int i = 0; i < D / 64; ++i) q_words[i] = src[lane * (D / 64) + i];
        }
    };
    load_q(warp);
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
        // (a budget near 2^31: one step further needs the 32nd bit)
        for (uint32_t i = rank * kThreads + tid; i < (uint32_t)P.budget; i += C * kThreads)
            out[i] = i < (uint32_t)n ? first + (int)i : -1;
        return;
    }

    if (C > 1) cluster_arrive();
    // ---- the CTA's pages [lo, lo + m); a warp has kTile at a time, whose bounds are under
    // way while the queries are made ready
    const int part = (n + C - 1) / C, lo = min(n, rank * part), m = min(part, n - lo);
    const int32_t* row = P.table + (int64_t)b * g.mpps + first + lo;
    bool none = false;
    uint4 a[RT][J];
    float sc[RT];
    auto load_tile = [&](int i0, int page) {
        none |= i0 + lane < m && (uint32_t)page >= (uint32_t)g.num_pages;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int p = __shfl_sync(0xffffffffu, page, gr + 8 * r);
            const bool ok = (uint32_t)p < (uint32_t)g.num_pages;
            const int64_t at = (int64_t)(ok ? p : 0) * g.Hkv + hk;
            const uint4* src = reinterpret_cast<const uint4*>(P.bounds + at * 2 * D) + t4;
#pragma unroll
            for (int j = 0; j < J; ++j) a[r][j] = __ldg(src + 4 * j);
            sc[r] = ok ? P.scale[at] : -1.f;     // (no page has a negative scale)
        }
    };
    auto page_of = [&](int i0) -> int { return i0 < m ? row[min(i0 + lane, m - 1)] : 0; };
    int i0 = kTile * warp;
    const int page0 = page_of(i0);
    int page1 = page_of(i0 + kTile * kWarps);
    if (i0 < m) load_tile(i0, page0);

    // ---- the group's queries in 8 bits, as f16: positive, then negative parts
    for (int h = warp; h < 8 * tiles; h += kWarps) {
        if (h != warp) load_q(h);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const uint32_t x = q_words[i] & 0x7fffu, y = (q_words[i] >> 16) & 0x7fffu;
            top = max(top, max(x > 0x7f80u ? 0u : x, y > 0x7f80u ? 0u : y));   // NaN: none
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, top);
        // least e with most <= 127 * 2^e = 1.984375 * 2^(e + 6)
        const int e = max(-50, min(50, (int)(most >> 7) - 133 + ((most & 127u) == 127u ? 1 : 0)));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t w0, w1;
        if constexpr (D == 128) {
            w0 = q_words[0];
            w1 = q_words[1];
        } else {
            // (a lane has a word, its neighbour the rest of its four codes)
            w0 = __shfl_sync(0xffffffffu, q_words[0], 2 * (lane & 15));
            w1 = __shfl_sync(0xffffffffu, q_words[0], 2 * (lane & 15) + 1);
        }
        float c[4];
        q_codes(w0, w1, inv, c);
        float up = 0.f, down = 0.f;              // sums over a run: 16 lanes' codes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            up += fmaxf(c[i], 0.f);
            down += fminf(c[i], 0.f);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
            up += __shfl_xor_sync(0xffffffffu, up, o);
            down += __shfl_xor_sync(0xffffffffu, down, o);
        }
        if (D == 128 || lane < 16) {
            uint2* dst = reinterpret_cast<uint2*>(smem + h * kQRow);
            dst[lane] = make_uint2(pack_f16x2(fmaxf(c[0], 0.f), fmaxf(c[1], 0.f)),
                                   pack_f16x2(fmaxf(c[2], 0.f), fmaxf(c[3], 0.f)));
            dst[D / 4 + lane] = make_uint2(pack_f16x2(fminf(c[0], 0.f), fminf(c[1], 0.f)),
                                           pack_f16x2(fminf(c[2], 0.f), fminf(c[3], 0.f)));
            if (lane % 16 == 0) {
                s_bias[h][lane / 16] = kBias * up;
                s_bias[h][J / 2 + lane / 16] = kBias * down;
            }
        }
        if (lane == 0) s_factor[h] = __uint_as_float((uint32_t)(127 + e) << 23);
    }
    // (a cluster's first CTA must have begun before the others write to it)
    __syncthreads();
    if (C > 1) cluster_wait();

    // ---- scores
    const uint32_t keys = C > 1 ? mapa_shared(smem_u32(s_key), 0) : smem_u32(s_key);
#pragma unroll 1
    for (; i0 < m; i0 += kTile * kWarps) {
        float best[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) best[r] = -INFINITY;
        for (int nt = 0; nt < tiles; ++nt) {
            float sum[RT / 2][4];
#pragma unroll
            for (int r = 0; r < RT / 2; ++r) sum[r][0] = sum[r][1] = sum[r][2] = sum[r][3] = 0.f;
            const uint8_t* qr = smem + (8 * nt + gr) * kQRow + 32 * t4;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint4 q0 = *reinterpret_cast<const uint4*>(qr + 128 * j);
                const uint4 q1 = *reinterpret_cast<const uint4*>(qr + 128 * j + 16);
                const float b0 = s_bias[8 * nt + 2 * t4][j], b1 = s_bias[8 * nt + 2 * t4 + 1][j];
#pragma unroll
                for (int r = 0; r < RT / 2; ++r) {
                    const uint4 x = a[2 * r][j], y = a[2 * r + 1][j];
                    float d[4];
                    uint32_t f[4];
                    codes_to_f16(x.x, f[0], f[2]);
                    codes_to_f16(y.x, f[1], f[3]);
                    mma_f16_first(d, f, q0.x, q0.y);
                    codes_to_f16(x.y, f[0], f[2]);
                    codes_to_f16(y.y, f[1], f[3]);
                    mma_f16_16816(d, f, q0.z, q0.w);
                    codes_to_f16(x.z, f[0], f[2]);
                    codes_to_f16(y.z, f[1], f[3]);
                    mma_f16_16816(d, f, q1.x, q1.y);
                    codes_to_f16(x.w, f[0], f[2]);
                    codes_to_f16(y.w, f[1], f[3]);
                    mma_f16_16816(d, f, q1.z, q1.w);
                    sum[r][0] += d[0] - b0;
                    sum[r][1] += d[1] - b1;
                    sum[r][2] += d[2] - b0;
                    sum[r][3] += d[3] - b1;
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int h = 8 * nt + 2 * t4 + x;
                const float f = s_factor[h];
                if (h < g.G)
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        best[r] = fmaxf(best[r], sum[r / 2][2 * (r & 1) + x] * f);
            }
        }
        uint32_t key[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
            best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
            const int i = lo + i0 + gr + 8 * r;
            const bool kept = i < P.num_first || i >= n - P.num_recent;
            key[r] = kept ? kKept : sc[r] < 0.f ? 0u : key_of(best[r] * sc[r]);
        }
        // lane (gr, t4) writes the key of its row t4
        static_assert(RT == 4, "a row a lane");
        const uint32_t mine = t4 == 0 ? key[0] : t4 == 1 ? key[1] : t4 == 2 ? key[2] : key[3];
        const int i = i0 + gr + 8 * t4;
        if (i < m) st_dsm_u32(keys + 4u * (uint32_t)(lo + i), mine);
        const int next = i0 + kTile * kWarps;
        if (next < m) {
            load_tile(next, page1);
            page1 = page_of(next + kTile * kWarps);
        }
    }
    if (none) flag_error(P.err, PA_DEV_BAD_PAGE);
    __syncwarp();
    if (C > 1) {
        cluster_sync_all();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    // ---- between which two keys the bits differ
    uint32_t least = 0xffffffffu, most = 0u;
    for (int i = tid; i < n; i += kThreads) {
        const uint32_t x = s_key[i];
        if (x != kKept) {
            least = min(least, x);
            most = max(most, x);
        }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s_range[warp] = make_uint2(least, most);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        least = min(least, s_range[w].x);
        most = max(most, s_range[w].y);
    }
    // ---- the keys to list: those from `from` up, and `take` of those equal to `equal`
    // (the kept ones, above all others, are the first num_first + num_recent)
    auto four_keys = [&](int i, uint32_t* x) {   // (behind the last: anything)
        const uint4 v = *reinterpret_cast<const uint4*>(s_key + i);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    };
    int take = P.budget - P.num_first - P.num_recent;
    uint32_t from = kKept, equal = 0u;
    if (take > 0) {
        int shift = 32 - __clz(least ^ most);    // bits that differ (0: all keys are equal)
        uint32_t prefix = shift < 32 ? most >> shift : 0u;
        for (int pass = 0; shift > 0; ++pass) {
            const int width = min(kBinBits, shift);
            uint32_t* hist = s_hist[pass & 1];
            if (pass > 0)                        // (the last one's is read; a third pass has it)
                for (int i = tid; i < kBins / 4; i += kThreads)
                    reinterpret_cast<uint4*>(s_hist[pass & 1 ^ 1])[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int i = tid; i < n; i += kThreads) {
                const uint32_t x = s_key[i];
                if (x != kKept && (shift == 32 || x >> shift == prefix))
                    atomicAdd(&hist[(x >> (shift - width)) & ((1u << width) - 1u)], 1u);
            }
            __syncthreads();
            // a thread has kMine bins: in which one is the take-th from the top?
            uint32_t h[kMine], sum = 0;
#pragma unroll
            for (int d = 0; d < kMine; d += 4) {
                const uint4 v = reinterpret_cast<const uint4*>(hist + tid * kMine)[d / 4];
                h[d] = v.x;
                h[d + 1] = v.y;
                h[d + 2] = v.z;
                h[d + 3] = v.w;
                sum += v.x + v.y + v.z + v.w;
            }
            uint32_t upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_down_sync(0xffffffffu, upto, o);
                if (lane + o < 32) upto += y;
            }
            if (lane == 0) s_warp[warp] = upto;
            __syncthreads();
            uint32_t above = upto - sum;
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                if (w > warp) above += s_warp[w];
            if (above < (uint32_t)take && above + sum >= (uint32_t)take) {   // one thread
#pragma unroll
                for (int d = kMine - 1; d >= 0; --d) {
                    if (above < (uint32_t)take && above + h[d] >= (uint32_t)take)
                        s_found = make_int3(tid * kMine + d, (int)h[d], (int)above);
                    above += h[d];
                }
            }
            __syncthreads();
            const int3 found = s_found;
            take -= found.z;
            prefix = prefix << width | (uint32_t)found.x;
            shift -= width;
            if (found.y == take) {               // the whole bin
                from = prefix << shift;
                take = 0;
                break;
            }
        }
        if (take > 0) {
            equal = shift > 0 ? 0u : prefix;     // (no bits differ: prefix is the one key)
            from = equal + 1;
        }
    }

    // ---- list them: a key's place is the number of listed ones before it.  A lane has four
    // keys at a time; counts of keys from `from` up, and 2^16 times those of equal ones
    const int seg = (n + 4 * kThreads - 1) / (4 * kThreads) * 128;   // keys of a warp
    const int w0 = min(n, warp * seg), w1 = min(n, w0 + seg);
    auto count = [&](const uint32_t* x, int i) -> uint32_t {
        uint32_t c = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < w1) c += x[j] >= from ? 1u : x[j] == equal ? 0x10000u : 0u;
        return c;
    };
    int above = 0, same = 0;
    for (int i = w0 + 4 * lane; i < w0 + seg; i += 128) {
        uint32_t x[4], c = 0;
        if (i < w1) {
            four_keys(i, x);
            c = count(x, i);
        }
        c = __reduce_add_sync(0xffffffffu, c);
        above += (int)(c & 0xffffu);
        same += (int)(c >> 16);
    }
    if (lane == 0) s_part[warp] = make_int2(above, same);
    __syncthreads();
    above = same = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) {
            above += s_part[w].x;
            same += s_part[w].y;
        }
    for (int i = w0 + 4 * lane; i < w0 + seg; i += 128) {
        uint32_t x[4] = {0u, 0u, 0u, 0u}, c = 0;
        if (i < w1) {
            four_keys(i, x);
            c = count(x, i);
        }
        uint32_t upto = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        int up = above + (int)((upto - c) & 0xffffu), eq = same + (int)((upto - c) >> 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < w1) {
                if (x[j] >= from) {
                    out[up + min(take, eq)] = first + i + j;
                    ++up;
                } else if (x[j] == equal) {
                    if (eq < take) out[up + eq] = first + i + j;
                    ++eq;
                }
            }
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        above += (int)(all & 0xffffu);
        same += (int)(all >> 16);
    }
}

template <int D, int kThreads>
cudaError_t launch(const SelectParams& P, int smem, cudaStream_t stream) {
    const cudaError_t e = allow_smem<select_kernel<D, kThreads>>(
        kMaxGroup * q_row_bytes(D) + PA_MAX_SELECT_PAGES * 4);
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
    return cudaLaunchKernelEx(&cfg, select_kernel<D, kThreads>, P);
}

}  // namespace

cudaError_t launch_select(const SelectParams& P0, int sms, cudaStream_t stream) {
    SelectParams P = P0;
    const int pages = (int)(((int64_t)P.g.max_ctx + P.g.ps - 1) >> P.g.ps_shift);
    // CTAs of a cluster: until the GPU has two an SM, none with under 64 pages
    int c = 1;
    const int64_t units = (int64_t)P.g.total_q * P.g.Hkv;
    while (c < kMaxCluster && units * c < 2 * sms && pages >= 128 * c) c *= 2;
    P.cluster = c;
    // (keys are read four at a time)
    const int smem = (P.g.G + 7) / 8 * 8 * q_row_bytes(P.g.D) + (pages + 3) / 4 * 16;
    // (more threads where a CTA scores or selects from many)
    if (pages > 1024)
        return P.g.D == 128 ? launch<128, 512>(P, smem, stream) : launch<64, 512>(P, smem, stream);
    return P.g.D == 128 ? launch<128, 256>(P, smem, stream) : launch<64, 256>(P, smem, stream);
}

}  // namespace pa
