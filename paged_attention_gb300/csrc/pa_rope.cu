// pa_rope.cu -- rotary positions on a step's queries and keys, on the keys' (and
// values') way into the paged cache.
//
//   (x, y) -> s (x cos a - y sin a, y cos a + x sin a),   a = position * inv_freq
//
// The angle is held in turns, as a fraction of 2^64: position * step wraps where
// the angle does, so a position of a million is as exact as one of ten, without
// 64-bit floating point (of which the GPU has little).  Its upper 32 bits go to
// sincospif.
//
// A CTA takes some tokens: cos and sin of their pairs once into shared memory,
// then rows (a head's 2 D bytes) of q, k and v alike, each by D / 16 neighbouring
// lanes.  A lane has two pieces of 16 bytes, the pairs' both halves, so a row is
// read and written once, in whole sectors.  Bound by HBM on long prompts (15237
// rows of 32 + 8 + 8 heads: 58.5 us for 56.3 of HBM time), by latency on a decode step
// (64 rows: 2.6 us in a graph, 9 from the host).
#include <algorithm>

#include "pa_step_common.cuh"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;                 // of an SM
// Tokens of a CTA: few, so that the CTAs of an SM are at their angles at different times
// (15237 rows: 58.5 us with 4, 61 with 8, 65 with 16, 74 with 32).
constexpr int kMaxTokens = 4;

// Two bf16 pairs (x0 y0, ...) turned; cs: (cos, sin) of each pair.
__device__ __forceinline__ void turn(float x, float y, float2 cs, float& u, float& w) {
    u = fmaf(x, cs.x, -(y * cs.y));
    w = fmaf(y, cs.x, x * cs.y);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The scale bytes of a row's blocks (32 elements, four pieces), of which this lane
// has the pieces c0 and c1 and its L neighbours the others.
template <int D>
__device__ __forceinline__ void row_scales(const uint4& a, const uint4& b, int c0, int c1,
                                           uint32_t& e0, uint32_t& e1) {
    constexpr int L = D / 16;
    auto top = [](const uint4& x) {
        return max_bf16x2(max_bf16x2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                          max_bf16x2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    };
    const uint32_t ta = top(a), tb = top(b);
#pragma unroll
    for (int blk = 0; blk < D / 32; ++blk) {
        uint32_t m = max_bf16x2(c0 / 4 == blk ? ta : 0u, c1 / 4 == blk ? tb : 0u);
#pragma unroll
        for (int o = 1; o < L; o <<= 1) m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t e = block_scale(m);
        if (c0 / 4 == blk) e0 = e;
        if (c1 / 4 == blk) e1 = e;
    }
}

template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads, kCtas)
rope_kernel(const __grid_constant__ RopeParams P) {
    constexpr int L = D / 16;            // lanes of a row
    constexpr int RP = kThreads / L;     // rows of a pass
    constexpr int U = MX4 ? 2 : 3;       // rows of a thread under way at a time
    __shared__ float2 s_cs[kMaxTokens * (D / 2)];
    __shared__ int2 s_at[kMaxTokens];    // position, slot (-1: a row to skip)
    const CacheGeom& g = P.g;
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * P.tokens, n = min(P.tokens, g.total_q - t0);
    const int half = P.rotary / 2;
    grid_dependency_wait();

    if (tid < n) {
        const int pos = P.positions[t0 + tid];
        int slot = P.slots[t0 + tid];
        if (slot >= 0 && (slot >> g.ps_shift) >= g.num_pages) {
            flag_error(P.err, PA_DEV_BAD_PAGE);
            slot = -1;
        }
        if (slot < -1) {
            flag_error(P.err, PA_DEV_BAD_PAGE);
            slot = -1;
        }
        if (slot >= 0 && pos < 0) {
            flag_error(P.err, PA_DEV_BAD_LENGTHS);
            slot = -1;
        }
        s_at[tid] = make_int2(pos, slot);
    }
    for (int i = tid; i < n * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const uint64_t turns = (uint64_t)(uint32_t)P.positions[t0 + t] * P.steps[f];
        // half turns in [-1, 1)
        const float x = (float)(int32_t)(turns >> 32) * 4.656612873077393e-10f;
        float sn, cs;
        sincospif(x, &sn, &cs);
        s_cs[t * (D / 2) + f] = make_float2(cs * P.scale, sn * P.scale);
    }
    __syncthreads();

    const int nq = P.q != nullptr ? g.Hq : 0;
    const int rows = nq + 2 * g.Hkv;     // of a token
    const int j = tid % L;
    const bool turns = 16 * j < P.rotary;
    // the lane's two pieces of a row
    int c0 = 2 * j, c1 = 2 * j + 1;
    if (!P.interleaved && turns) {
        c0 = j;
        c1 = j + P.rotary / 16;
    }
    int t = 0, r = tid / L;
    while (r >= rows) {
        r -= rows;
        ++t;
    }
    const int passes = (n * rows + RP - 1) / RP;   // the same for every lane: they shuffle
    for (int p0 = 0; p0 < passes; p0 += U) {
        uint4 a[U], b[U];
        int tt[U], rr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tt[u] = t;
            rr[u] = r;
            a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
            if (t < n && s_at[t].y >= 0) {
                const __nv_bfloat16* src =
                    r < nq ? P.q + (int64_t)(t0 + t) * P.q_stride + (int64_t)r * D
                    : r < nq + g.Hkv
                        ? P.k + (int64_t)(t0 + t) * P.k_stride + (int64_t)(r - nq) * D
                        : P.v + (int64_t)(t0 + t) * P.v_stride + (int64_t)(r - nq - g.Hkv) * D;
                a[u] = reinterpret_cast<const uint4*>(src)[c0];
                b[u] = reinterpret_cast<const uint4*>(src)[c1];
            } else {
                tt[u] = n;
            }
            r += RP;
            while (r >= rows) {
                r -= rows;
                ++t;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool live = tt[u] < n;
            if (live && turns && rr[u] < nq + g.Hkv) {
                const float2* cs = s_cs + tt[u] * (D / 2) + 8 * j;
                uint32_t x[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
                uint32_t y[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
                if (P.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float m, w;
                        turn(lo_f(x[i]), hi_f(x[i]), cs[i], m, w);
                        x[i] = pack_bf16x2(m, w);
                        turn(lo_f(y[i]), hi_f(y[i]), cs[4 + i], m, w);
                        y[i] = pack_bf16x2(m, w);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float m0, w0, m1, w1;
                        turn(lo_f(x[i]), lo_f(y[i]), cs[2 * i], m0, w0);
                        turn(hi_f(x[i]), hi_f(y[i]), cs[2 * i + 1], m1, w1);
                        x[i] = pack_bf16x2(m0, m1);
                        y[i] = pack_bf16x2(w0, w1);
                    }
                }
                a[u] = make_uint4(x[0], x[1], x[2], x[3]);
                b[u] = make_uint4(y[0], y[1], y[2], y[3]);
            }
            uint32_t e0 = 0, e1 = 0;
            if constexpr (MX4) row_scales<D>(a[u], b[u], c0, c1, e0, e1);
            if (!live) continue;
            if (rr[u] < nq) {
                uint4* dst = reinterpret_cast<uint4*>(
                    P.q_out + ((int64_t)(t0 + tt[u]) * g.Hq + rr[u]) * D);
                dst[c0] = a[u];
                dst[c1] = b[u];
                continue;
            }
            const bool is_v = rr[u] >= nq + g.Hkv;
            const int h = rr[u] - nq - (is_v ? g.Hkv : 0), slot = s_at[tt[u]].y;
            const int64_t to = row_of(g, slot >> g.ps_shift, slot & (g.ps - 1), h);
            void* cache = is_v ? P.v_cache : P.k_cache;
            if constexpr (MX4) {
                uint8_t* scale = is_v ? P.v_scale : P.k_scale;
                const uint32_t x[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
                const uint32_t y[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
                uint32_t* codes = reinterpret_cast<uint32_t*>(cache) + to * (D / 8);
                codes[c0] = codes8(x, e0);
                codes[c1] = codes8(y, e1);
                if (c0 % 4 == 0) scale[to * (D / 32) + c0 / 4] = (uint8_t)e0;
                if (c1 % 4 == 0) scale[to * (D / 32) + c1 / 4] = (uint8_t)e1;
            } else {
                uint4* dst = reinterpret_cast<uint4*>(cache) + to * (D / 8);
                dst[c0] = a[u];
                dst[c1] = b[u];
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& P0, bool mx4, int sms, cudaStream_t stream) {
    RopeParams P = P0;
    // as many tokens a CTA as make whole waves of them
    const int64_t resident = (int64_t)sms * kCtas;
    const int64_t waves = (P.g.total_q + resident * kMaxTokens - 1) / (resident * kMaxTokens);
    P.tokens = (int)std::min<int64_t>(
        kMaxTokens, (P.g.total_q + resident * waves - 1) / (resident * waves));
    auto kern = P.g.D == 128 ? (mx4 ? rope_kernel<128, true> : rope_kernel<128, false>)
                             : (mx4 ? rope_kernel<64, true> : rope_kernel<64, false>);
    return launch_dependent(kern, dim3((P.g.total_q + P.tokens - 1) / P.tokens), dim3(kThreads), 0,
                            stream, P);
}

}  // namespace pa
