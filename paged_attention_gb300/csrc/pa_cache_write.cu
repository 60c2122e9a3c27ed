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
constexpr int kMaxTokens = 32;   // tokens of one CTA: one per lane of its first warp

// Where a CTA's tokens live: the rows of their first head (-1: a token to skip),
// in the cache and, for reading back, in the other pages; and where their key
// weights of the first head are.
struct TokenPlace {
    int64_t row, dst_row, weight;
};

// The thread's items run through token (of the CTA) and position within a token:
// kWriteThreads further each time, without a division.
struct Cursor {
    int t, r;
    __device__ __forceinline__ void step(int per_token) {
        r += kWriteThreads;
        while (r >= per_token) {
            r -= per_token;
            ++t;
        }
    }
};
__device__ __forceinline__ Cursor first_item(int per_token) {
    Cursor c = {0, (int)threadIdx.x - kWriteThreads};
    c.step(per_token);
    return c;
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
        if (blockIdx.x == 0) check_lens(g, ctx, ql, lane, err);
    }
    __syncthreads();
}

// Quantise the 8 elements a lane holds of a block spread over 4 lanes.
__device__ __forceinline__ uint32_t quantise8(uint4 x, uint32_t& e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    // magnitudes of bf16 order like their bits
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t ex = top >> 7;   // biased exponent of the largest magnitude
    e = ex == 255 ? 255u : ex > 2 ? ex - 2 : 0u;
    if (ex == 255) return 0u;
    const float inv = __uint_as_float((254u - e) << 23);   // 2^(127 - e), never subnormal
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(w[i] << 16) * inv;
        const float hi = __uint_as_float(w[i] & 0xffff0000u) * inv;
        codes |= f32x2_to_e2m1x2(lo, hi) << (8 * i);
    }
    return codes;
}

// One item: 8 elements (16 source bytes) of one row of K or V.  Bound by HBM
// on long prompts and by latency on a decode step.
template <int D, bool MX4>
__global__ void __launch_bounds__(kWriteThreads)
append_kernel(const CacheGeom g, const __nv_bfloat16* __restrict__ k_new,
              const __nv_bfloat16* __restrict__ v_new, int64_t k_stride, int64_t v_stride,
              const int32_t* __restrict__ table, const int32_t* __restrict__ ctx,
              const int32_t* __restrict__ ql, void* k_cache, uint8_t* k_scale, void* v_cache,
              uint8_t* v_scale, float* weights, int32_t* err, int tokens) {
    constexpr int C = D / 8;   // items of a row
    __shared__ TokenPlace place[kMaxTokens];
    const int t0 = blockIdx.x * tokens, n = min(tokens, g.total_q - t0);
    find_places(g, table, ctx, ql, t0, n, nullptr, 0, 0, place, err);
    const int half = g.Hkv * C, per_token = 2 * half;
    // every lane of a warp takes part in the shuffles: the trip count is
    // uniform; U items' loads are under way at a time
    constexpr int U = 4;
    const int rounds = (n * per_token + kWriteThreads - 1) / kWriteThreads;
    Cursor at = first_item(per_token);
    for (int i = 0; i < rounds; i += U) {
        uint4 x[U];
        Cursor ahead = at;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (ahead.t < n && place[ahead.t].row >= 0) {
                const int kv = ahead.r >= half;
                const __nv_bfloat16* src = kv ? v_new + (int64_t)(t0 + ahead.t) * v_stride
                                              : k_new + (int64_t)(t0 + ahead.t) * k_stride;
                x[u] = __ldcs(reinterpret_cast<const uint4*>(src) + (ahead.r - (kv ? half : 0)));
            }
            ahead.step(per_token);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= rounds) break;
            const Cursor me = at;
            at.step(per_token);
            const int kv = me.r >= half, hc = me.r - (kv ? half : 0), h = hc / C, c = hc % C;
            uint32_t codes = 0, scales = 0;
            if constexpr (MX4) {
                uint32_t e;
                codes = quantise8(x[u], e);
                // the row's scale bytes, collected in its first lane
                const int lane = threadIdx.x & 31, base = lane & ~(C - 1);
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    scales |= __shfl_sync(0xffffffffu, e, base + 4 * j) << (8 * j);
            }
            if (me.t >= n || place[me.t].row < 0) continue;
            const int64_t row = place[me.t].row + (int64_t)h * g.head_rows;
            void* cache = kv ? v_cache : k_cache;
            if constexpr (MX4) {
                reinterpret_cast<uint32_t*>(cache)[row * C + c] = codes;
                if (c == 0) {
                    uint8_t* sc = kv ? v_scale : k_scale;
                    if constexpr (D == 128)
                        reinterpret_cast<uint32_t*>(sc)[row] = scales;
                    else
                        reinterpret_cast<uint16_t*>(sc)[row] = (uint16_t)scales;
                }
            } else {
                reinterpret_cast<uint4*>(cache)[row * C + c] = x[u];
            }
            if (weights != nullptr && kv == 0 && c == 0)
                weights[place[me.t].weight + (int64_t)h * g.ps] = 0.f;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kWriteThreads)
expand_kernel(const CacheGeom g, const uint32_t* __restrict__ k_cache,
              const uint8_t* __restrict__ k_scale, const uint32_t* __restrict__ v_cache,
              const uint8_t* __restrict__ v_scale, const int32_t* __restrict__ table,
              const int32_t* __restrict__ ctx, const int32_t* __restrict__ ql,
              const int32_t* __restrict__ dst_table, int dst_mpps, int dst_pages, void* k_out,
              void* v_out, int32_t* err, int tokens) {
    constexpr int C = D / 8;
    __shared__ TokenPlace place[kMaxTokens];
    const int t0 = blockIdx.x * tokens, n = min(tokens, g.total_q - t0);
    find_places(g, table, ctx, ql, t0, n, dst_table, dst_mpps, dst_pages, place, err);
    const int half = g.Hkv * C, per_token = 2 * half;
    constexpr int U = 4;   // items of a thread under way at a time
    Cursor at = first_item(per_token);
    while (at.t < n) {
        uint32_t w[U], e[U];
        Cursor ahead = at;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            w[u] = e[u] = 0;
            if (ahead.t < n && place[ahead.t].row >= 0) {
                const int kv = ahead.r >= half, hc = ahead.r - (kv ? half : 0);
                const int64_t row = place[ahead.t].row + (int64_t)(hc / C) * g.head_rows;
                w[u] = (kv ? v_cache : k_cache)[row * C + hc % C];
                e[u] = (kv ? v_scale : k_scale)[row * (D / 32) + hc % C / 4];
            }
            ahead.step(per_token);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Cursor me = at;
            at.step(per_token);
            if (me.t >= n || place[me.t].row < 0) continue;
            const int kv = me.r >= half, hc = me.r - (kv ? half : 0);
            const float f = e8m0_to_f32(e[u]);
            uint32_t v[4];
            e2m1x8_to_f16(w[u], v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
                v[j] = pack_bf16x2(x.x * f, x.y * f);
            }
            const int64_t out = place[me.t].dst_row + (int64_t)(hc / C) * g.head_rows;
            reinterpret_cast<uint4*>(kv ? v_out : k_out)[out * C + hc % C] =
                make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}

// Tokens of a CTA: as few as fill its threads once, so that a decode step takes
// one pass, and more on long prompts, so that a CTA spends less of its life
// finding its tokens' pages; but still 32 CTAs an SM, to keep the last of them
// short (18000 tokens of 8 heads written and read back: 75 us with 8 an SM, 65
// with 16, 61 with 32, 64 with 64).
int tokens_per_cta(const CacheGeom& g, int sms) {
    const int per_token = 2 * g.Hkv * (g.D / 8);
    int n = per_token >= kWriteThreads ? 1 : kWriteThreads / per_token;
    while (n < kMaxTokens && (int64_t)n * sms * 32 < g.total_q) n *= 2;
    return n < kMaxTokens ? n : kMaxTokens;
}

}  // namespace

cudaError_t launch_append(const CacheGeom& g, bool mx4, const void* k_new, const void* v_new,
                          int64_t k_stride, int64_t v_stride, const int32_t* table,
                          const int32_t* ctx, const int32_t* ql, void* k_cache, void* k_scale,
                          void* v_cache, void* v_scale, float* weights, int32_t* err, int sms,
                          cudaStream_t stream) {
    const int tokens = tokens_per_cta(g, sms);
    const int grid = (g.total_q + tokens - 1) / tokens;
    auto kern = g.D == 128 ? (mx4 ? append_kernel<128, true> : append_kernel<128, false>)
                           : (mx4 ? append_kernel<64, true> : append_kernel<64, false>);
    kern<<<grid, kWriteThreads, 0, stream>>>(
        g, (const __nv_bfloat16*)k_new, (const __nv_bfloat16*)v_new, k_stride, v_stride, table,
        ctx, ql, k_cache, (uint8_t*)k_scale, v_cache, (uint8_t*)v_scale, weights, err, tokens);
    return cudaGetLastError();
}

cudaError_t launch_expand(const CacheGeom& g, const void* k_cache, const void* k_scale,
                          const void* v_cache, const void* v_scale, const int32_t* table,
                          const int32_t* ctx, const int32_t* ql, const int32_t* dst_table,
                          int dst_mpps, int dst_pages, void* k_out, void* v_out, int32_t* err,
                          int sms, cudaStream_t stream) {
    const int tokens = tokens_per_cta(g, sms);
    const int grid = (g.total_q + tokens - 1) / tokens;
    auto kern = g.D == 128 ? expand_kernel<128> : expand_kernel<64>;
    kern<<<grid, kWriteThreads, 0, stream>>>(
        g, (const uint32_t*)k_cache, (const uint8_t*)k_scale, (const uint32_t*)v_cache,
        (const uint8_t*)v_scale, table, ctx, ql, dst_table, dst_mpps, dst_pages, k_out, v_out, err,
        tokens);
    return cudaGetLastError();
}

}  // namespace pa
