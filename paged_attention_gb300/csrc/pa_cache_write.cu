// pa_cache_write.cu -- new K/V rows into a paged cache (bf16 copied, or
// quantised to the PA_MX4 form), and rows of a PA_MX4 cache back into bf16 pages.
//
// Quantisation of a block x of 32: e = max(-127, floor(log2 max|x|) - 2), codes
// = round(x / 2^e) to E2M1.  x / 2^e is a product with a power of two, so the
// only rounding is the hardware conversion's (nearest, ties to even).
#include "pa_cache_common.cuh"

namespace pa {

namespace {

constexpr int kWriteThreads = 256;
constexpr int kWriteCtas = 5;    // of an SM
constexpr int kMaxTokens = 32;   // tokens of one CTA: one per lane of its first warp

// Where a CTA's tokens live: the rows of their first head (-1: a token to skip),
// in the cache and, for reading back, in the other pages; and where their key
// weights of the first head are.
struct TokenPlace {
    int64_t row, dst_row, weight;
};

// A thread has one position in a token -- K or V, head, 16 bytes of bf16 -- and
// takes it of many tokens: narrow tokens share the CTA's threads, wide ones take
// several CTAs (blockIdx.y).
struct Position {
    int first, step;             // the thread's tokens: first, first + step, ...
    int kv, hc, h, c;            // K or V; position in it; head; position in the row
};
template <int C>
__device__ __forceinline__ Position my_position(const CacheGeom& g) {
    const int half = g.Hkv * C, per_token = 2 * half;
    Position p;
    int r;
    if (per_token <= kWriteThreads) {
        p.step = kWriteThreads / per_token;
        p.first = threadIdx.x / per_token;
        r = threadIdx.x % per_token;
        if (p.first >= p.step) p.first = kMaxTokens;       // left over: no tokens
    } else {
        p.step = 1;
        r = blockIdx.y * kWriteThreads + threadIdx.x;
        p.first = r < per_token ? 0 : kMaxTokens;
    }
    p.kv = r >= half;
    p.hc = r - (p.kv ? half : 0);
    p.h = p.hc / C;
    p.c = p.hc % C;
    return p;
}

// The first warp finds the places of the CTA's tokens [t0, t0 + n).
__device__ __forceinline__ void find_places(const CacheGeom& g, const int32_t* table,
                                            const int32_t* ctx, const int32_t* ql, int t0, int n,
                                            const int32_t* dst_table, int dst_mpps, int dst_pages,
                                            TokenPlace* place, int32_t* err) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int start = 0;
        const int b = seq_of_row(g, ql, t0 + min(lane, n - 1), lane, start);
        TokenPlace p = {-1, -1, 0};
        if (b >= 0 && lane < n) {
            const int q = ql[b], c = ctx[b];
            if (good_lens(g, q, c)) {
                const int pos = c - q + (t0 + lane - start);
                const int pi = pos >> g.ps_shift, slot = pos & (g.ps - 1);
                const int page = table[(int64_t)b * g.mpps + pi];
                bool bad = page < 0 || page >= g.num_pages;
                if (dst_table != nullptr && !bad) {
                    const int dst = dst_table[(int64_t)b * dst_mpps + pi];
                    bad = dst < 0 || dst >= dst_pages;
                    if (!bad) p.dst_row = row_of(g, dst, slot, 0);
                }
                if (!bad) {
                    p.row = row_of(g, page, slot, 0);
                    p.weight = (int64_t)page * g.Hkv * g.ps + slot;
                }
                if (bad) flag_error(err, PA_DEV_BAD_PAGE);
            }
        }
        if (lane < n) place[lane] = p;
        if (blockIdx.x == 0 && blockIdx.y == 0) check_lens(g, ctx, ql, lane, err);
    }
    __syncthreads();
}

// Quantise the 8 elements a lane holds of a block spread over 4 lanes.
__device__ __forceinline__ uint32_t quantise8(uint4 x, uint32_t& e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t two = max_bf16x2(max_bf16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                              max_bf16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    two = max_bf16x2(two, __shfl_xor_sync(0xffffffffu, two, 1));
    two = max_bf16x2(two, __shfl_xor_sync(0xffffffffu, two, 2));
    e = block_scale(two);
    return codes8(w, e);
}

// A thread quantises 8 elements (16 source bytes) of a row at a time.  Bound by
// HBM on long prompts and by latency on a decode step.
template <int D, bool MX4>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas)
append_kernel(const CacheGeom g, const __nv_bfloat16* __restrict__ k_new,
              const __nv_bfloat16* __restrict__ v_new, int64_t k_stride, int64_t v_stride,
              const int32_t* __restrict__ table, const int32_t* __restrict__ ctx,
              const int32_t* __restrict__ ql, void* k_cache, uint8_t* k_scale, void* v_cache,
              uint8_t* v_scale, float* weights, int32_t* err, int tokens) {
    grid_dependency_wait();
    constexpr int C = D / 8;   // threads of a row
    __shared__ TokenPlace place[kMaxTokens];
    const int t0 = blockIdx.x * tokens, n = min(tokens, g.total_q - t0);
    find_places(g, table, ctx, ql, t0, n, nullptr, 0, 0, place, err);
    const Position p = my_position<C>(g);
    const int64_t stride = p.kv ? v_stride : k_stride;
    const __nv_bfloat16* src = (p.kv ? v_new : k_new) + (int64_t)t0 * stride + p.hc * 8;
    void* cache = p.kv ? v_cache : k_cache;
    uint8_t* scale = p.kv ? v_scale : k_scale;
    const int64_t head = (int64_t)p.h * g.head_rows;
    // every lane of a warp takes part in the shuffles: the trip count is
    // uniform; U tokens' loads are under way at a time
    constexpr int U = 4;
    for (int i = 0; i < n; i += U * p.step) {
        uint4 x[U];
        int64_t row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = i + u * p.step + p.first;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            row[u] = t < n ? place[t].row : -1;
            if (row[u] >= 0) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + t * stride));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t codes = 0, e = 0;
            if constexpr (MX4) codes = quantise8(x[u], e);
            if (row[u] < 0) continue;
            const int64_t to = row[u] + head;
            if constexpr (MX4) {
                reinterpret_cast<uint32_t*>(cache)[to * C + p.c] = codes;
                if (p.c % 4 == 0) scale[to * (D / 32) + p.c / 4] = (uint8_t)e;
            } else {
                reinterpret_cast<uint4*>(cache)[to * C + p.c] = x[u];
            }
            if (weights != nullptr && p.kv == 0 && p.c == 0)
                weights[place[i + u * p.step + p.first].weight + (int64_t)p.h * g.ps] = 0.f;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kWriteThreads, kWriteCtas)
expand_kernel(const CacheGeom g, const uint32_t* __restrict__ k_cache,
              const uint8_t* __restrict__ k_scale, const uint32_t* __restrict__ v_cache,
              const uint8_t* __restrict__ v_scale, const int32_t* __restrict__ table,
              const int32_t* __restrict__ ctx, const int32_t* __restrict__ ql,
              const int32_t* __restrict__ dst_table, int dst_mpps, int dst_pages, void* k_out,
              void* v_out, int32_t* err, int tokens) {
    grid_dependency_wait();
    constexpr int C = D / 8;
    __shared__ TokenPlace place[kMaxTokens];
    const int t0 = blockIdx.x * tokens, n = min(tokens, g.total_q - t0);
    find_places(g, table, ctx, ql, t0, n, dst_table, dst_mpps, dst_pages, place, err);
    const Position p = my_position<C>(g);
    const uint32_t* code = p.kv ? v_cache : k_cache;
    const uint8_t* scale = p.kv ? v_scale : k_scale;
    uint4* out = reinterpret_cast<uint4*>(p.kv ? v_out : k_out);
    const int64_t head = (int64_t)p.h * g.head_rows;
    constexpr int U = 4;       // tokens of a thread under way at a time
    for (int i = p.first; i < n; i += U * p.step) {
        uint32_t w[U], e[U];
        int64_t row[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = i + u * p.step;
            w[u] = e[u] = 0;
            row[u] = t < n ? place[t].row : -1;
            if (row[u] >= 0) {
                w[u] = code[(row[u] + head) * C + p.c];
                e[u] = scale[(row[u] + head) * (D / 32) + p.c / 4];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (row[u] < 0) continue;
            // 2^(e - 127) in bf16
            const uint32_t f = e[u] == 0 ? 0x0040u : e[u] == 255 ? 0x7fc0u : e[u] << 7;
            uint32_t v[4];
            e2m1x8_to_f16(w[u], v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
                v[j] = mul_bf16x2(pack_bf16x2(x.x, x.y), f | (f << 16));
            }
            out[(place[i + u * p.step].dst_row + head) * C + p.c] =
                make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

// Tokens of a CTA: as few as fill its threads once, so that a decode step takes
// one pass, and on long prompts as many as make whole waves of CTAs, so that all
// of them look their pages up at once and none is left over (20000 tokens of 8
// heads written and read back: 48 us in one wave, 50 in two or three, 56 in four;
// 4 tokens of a thread under way and 5 CTAs an SM 48 us, 2 and 6 50, 6 and 4 49).
dim3 write_grid(const CacheGeom& g, int sms, int& tokens) {
    const int per_token = 2 * g.Hkv * (g.D / 8);
    const int least = per_token >= kWriteThreads ? 1 : kWriteThreads / per_token;
    const int wide = (per_token + kWriteThreads - 1) / kWriteThreads;
    const int64_t resident = max(1, sms * kWriteCtas / wide);
    const int64_t waves =
        max((int64_t)1, (g.total_q + resident * kMaxTokens - 1) / (resident * kMaxTokens));
    const int even = (int)((g.total_q + resident * waves - 1) / (resident * waves));
    tokens = min(max(least, even), kMaxTokens);
    return dim3((g.total_q + tokens - 1) / tokens, wide);
}

}  // namespace

cudaError_t launch_append(const CacheGeom& g, bool mx4, const void* k_new, const void* v_new,
                          int64_t k_stride, int64_t v_stride, const int32_t* table,
                          const int32_t* ctx, const int32_t* ql, void* k_cache, void* k_scale,
                          void* v_cache, void* v_scale, float* weights, int32_t* err, int sms,
                          cudaStream_t stream) {
    int tokens;
    const dim3 grid = write_grid(g, sms, tokens);
    auto kern = g.D == 128 ? (mx4 ? append_kernel<128, true> : append_kernel<128, false>)
                           : (mx4 ? append_kernel<64, true> : append_kernel<64, false>);
    return launch_dependent(kern, grid, dim3(kWriteThreads), 0, stream, g,
                            (const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, k_stride,
                            v_stride, table, ctx, ql, k_cache, (uint8_t*)k_scale, v_cache,
                            (uint8_t*)v_scale, weights, err, tokens);
}

cudaError_t launch_expand(const CacheGeom& g, const void* k_cache, const void* k_scale,
                          const void* v_cache, const void* v_scale, const int32_t* table,
                          const int32_t* ctx, const int32_t* ql, const int32_t* dst_table,
                          int dst_mpps, int dst_pages, void* k_out, void* v_out, int32_t* err,
                          int sms, cudaStream_t stream) {
    int tokens;
    const dim3 grid = write_grid(g, sms, tokens);
    auto kern = g.D == 128 ? expand_kernel<128> : expand_kernel<64>;
    return launch_dependent(kern, grid, dim3(kWriteThreads), 0, stream, g,
                            (const uint32_t*)k_cache, (const uint8_t*)k_scale,
                            (const uint32_t*)v_cache, (const uint8_t*)v_scale, table, ctx, ql,
                            dst_table, dst_mpps, dst_pages, k_out, v_out, err, tokens);
}

}  // namespace pa
