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

// Where a CTA's tokens live: page and slot, page -1 for a token to skip.
struct TokenPlace {
    int page, slot, dst_page;
};

// The first warp finds the places of the CTA's tokens [t0, t0 + n).
__device__ __forceinline__ void find_places(const CacheGeom& g, const int32_t* table,
                                            const int32_t* ctx, const int32_t* ql, int t0, int n,
                                            const int32_t* dst_table, int dst_mpps, int dst_pages,
                                            TokenPlace* place, int32_t* err) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int start = 0;
        const int b = seq_of_row(g, ql, t0 + min(lane, n - 1), lane, start);
        TokenPlace p = {-1, 0, -1};
        if (b >= 0 && lane < n) {
            const int q = ql[b], c = ctx[b];
            if (good_lens(g, q, c)) {
                const int pos = c - q + (t0 + lane - start);
                const int pi = pos >> g.ps_shift;
                p.slot = pos & (g.ps - 1);
                p.page = table[(int64_t)b * g.mpps + pi];
                if (p.page < 0 || p.page >= g.num_pages) p.page = -1;
                bool bad = p.page < 0;
                if (dst_table != nullptr && !bad) {
                    p.dst_page = dst_table[(int64_t)b * dst_mpps + pi];
                    if (p.dst_page < 0 || p.dst_page >= dst_pages) p.page = -1;
                    bad = p.page < 0;
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
    const int per_token = 2 * g.Hkv * C;
    // every lane of a warp takes part in the shuffles: the trip count is uniform
    const int items = n * per_token;
    for (int i0 = 0; i0 < items; i0 += kWriteThreads) {
        const int i = i0 + threadIdx.x;
        const bool in = i < items;
        const int t = in ? i / per_token : 0;
        const int r = in ? i - t * per_token : 0;
        const int kv = r / (g.Hkv * C), h = (r / C) % g.Hkv, c = r % C;
        const TokenPlace p = place[t];
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (in && p.page >= 0) {
            const __nv_bfloat16* src = kv ? v_new + (int64_t)(t0 + t) * v_stride
                                          : k_new + (int64_t)(t0 + t) * k_stride;
            x = *reinterpret_cast<const uint4*>(src + h * D + c * 8);
        }
        uint32_t codes = 0, scales = 0;
        if constexpr (MX4) {
            uint32_t e;
            codes = quantise8(x, e);
            // the row's scale bytes, collected in its first lane
            const int lane = threadIdx.x & 31, base = lane & ~(C - 1);
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
                scales |= __shfl_sync(0xffffffffu, e, base + 4 * j) << (8 * j);
        }
        if (!in || p.page < 0) continue;
        const int64_t row = row_of(g, p.page, p.slot, h);
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
            reinterpret_cast<uint4*>(cache)[row * C + c] = x;
        }
        if (weights != nullptr && kv == 0 && c == 0)
            weights[((int64_t)p.page * g.Hkv + h) * g.ps + p.slot] = 0.f;
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
    const int per_token = 2 * g.Hkv * C;
    const int items = n * per_token;
    for (int i = threadIdx.x; i < items; i += kWriteThreads) {
        const int t = i / per_token, r = i - t * per_token;
        const int kv = r / (g.Hkv * C), h = (r / C) % g.Hkv, c = r % C;
        const TokenPlace p = place[t];
        if (p.page < 0) continue;
        const int64_t row = row_of(g, p.page, p.slot, h);
        const uint32_t w = (kv ? v_cache : k_cache)[row * C + c];
        const float s = e8m0_to_f32((kv ? v_scale : k_scale)[row * (D / 32) + c / 4]);
        uint32_t v[4];
        e2m1x8_to_f16(w, v[0], v[1], v[2], v[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
            v[j] = pack_bf16x2(f.x * s, f.y * s);
        }
        const int64_t out = row_of(g, p.dst_page, p.slot, h);
        reinterpret_cast<uint4*>(kv ? v_out : k_out)[out * C + c] =
            make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// Tokens of a CTA: as few as fill its threads once while that leaves no more
// CTAs than the GPU runs at a time, else up to four times that, so that a CTA
// spends less of its life finding its tokens' pages.
int tokens_per_cta(const CacheGeom& g, int sms) {
    const int per_token = 2 * g.Hkv * (g.D / 8);
    const int once = per_token >= kWriteThreads ? 1 : kWriteThreads / per_token;
    int n = once;
    while (n < 4 * once && n < kMaxTokens && (int64_t)n * sms * 8 < g.total_q) n *= 2;
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
