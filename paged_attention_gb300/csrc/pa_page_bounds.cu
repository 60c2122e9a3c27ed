// pa_page_bounds.cu -- per page and KV head, each channel's largest and smallest
// key, rounded outward to 8 bits of a power of two.
//
// A row of the call is its page's last where the next row's slot lies in another
// page; it stands for the page.  A CTA looks through some rows for one head and takes
// the pages it finds one after the other, all its warps on a page: every row of it is
// read once, 16 bytes a lane, all of a page of 64 under way at a time; maxima and
// minima are taken of bf16 pairs, exactly.  Bound by HBM (2 D bytes a key) where pages
// are whole, by latency on a decode step, which reads one page a sequence and head.
// 69575 keys of 8 heads: 27 us for 21.8 of HBM time; 64 sequences' last pages 2.8 us in a
// graph, 5 from the host.
#include <algorithm>

#include "pa_cache_common.cuh"

namespace pa {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// x * 2^-e rounded up (or down) to a code; NaN as told
__device__ __forceinline__ int code_of(float x, float inv, bool up) {
    if (x != x) return up ? 127 : -127;
    float y = x * inv;
    if (y == 0.f && x != 0.f) y = x > 0.f ? 1e-30f : -1e-30f;   // (what is too small for fp32)
    return (int)fminf(fmaxf(up ? ceilf(y) : floorf(y), -127.f), 127.f);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8)
bounds_kernel(const CacheGeom g, const __nv_bfloat16* __restrict__ k,
              const int32_t* __restrict__ slots, int8_t* __restrict__ bounds,
              float* __restrict__ scale, int32_t* err, int rows) {
    constexpr int C = D / 8;             // 16-byte pieces of a row
    constexpr int RPI = 32 / C;          // rows of a warp's load
    constexpr int U = 8;                 // loads of a lane under way
    __shared__ uint4 s_part[2][kWarps][2][C];        // a warp's largest and smallest
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hk = blockIdx.y;
    grid_dependency_wait();
    const int r0 = blockIdx.x * rows, r1 = min(r0 + rows, g.total_q);
    int turn = 0;                        // (one half of s_part is read, the next page fills the other)
    for (int c = r0; c < r1; c += 32) {
        const int r = c + lane;
        const int slot = r < r1 ? slots[r] : -1;
        const int next = r + 1 < g.total_q && r < r1 ? slots[r + 1] : -1;
        // (a next slot that is negative shifts to a negative page: another one)
        bool last = slot >= 0 && (slot >> g.ps_shift) != (next >> g.ps_shift);
        const bool none = slot < -1 || (slot >= 0 && (slot >> g.ps_shift) >= g.num_pages);
        if (none && hk == 0 && warp == 0) flag_error(err, PA_DEV_BAD_PAGE);
        last = last && !none;
        for (uint32_t found = __ballot_sync(0xffffffffu, last); found != 0; found &= found - 1) {
            const int at = __shfl_sync(0xffffffffu, slot, __ffs(found) - 1);
            const int page = at >> g.ps_shift, used = (at & (g.ps - 1)) + 1;
            const uint4* src = reinterpret_cast<const uint4*>(k) + row_of(g, page, 0, hk) * C;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = 0xff80ff80u;     // -inf
                lo[i] = 0x7f807f80u;
            }
            const int k0 = warp * RPI + lane / C;
            for (int s = 0; s < used; s += U * kWarps * RPI) {
                uint4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // (behind the last key: that key again)
                    const int key = min(s + u * kWarps * RPI + k0, used - 1);
                    if (s + u * kWarps * RPI < used)
                        x[u] = __ldcs(src + (int64_t)key * g.tok_rows * C + lane % C);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (s + u * kWarps * RPI < used) {
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            hi[i] = max_bf16x2(hi[i], w[i]);
                            lo[i] = min_bf16x2(lo[i], w[i]);
                        }
                    }
            }
#pragma unroll
            for (int o = C; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hi[i] = max_bf16x2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
                    lo[i] = min_bf16x2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
                }
            if (lane < C) {
                s_part[turn][warp][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                s_part[turn][warp][1][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            __syncthreads();
            const int now = turn;
            turn ^= 1;
            if (warp != 0) continue;     // on to the next page
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const uint4 h = s_part[now][w][0][lane % C], l = s_part[now][w][1][lane % C];
                hi[0] = max_bf16x2(hi[0], h.x);
                hi[1] = max_bf16x2(hi[1], h.y);
                hi[2] = max_bf16x2(hi[2], h.z);
                hi[3] = max_bf16x2(hi[3], h.w);
                lo[0] = min_bf16x2(lo[0], l.x);
                lo[1] = min_bf16x2(lo[1], l.y);
                lo[2] = min_bf16x2(lo[2], l.z);
                lo[3] = min_bf16x2(lo[3], l.w);
            }
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top = max_bf16x2(top, max_bf16x2(hi[i] & 0x7fff7fffu, lo[i] & 0x7fff7fffu));
            // (bits of magnitudes order like the magnitudes, NaN above infinity)
            const uint32_t m = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
            // least e with m <= 127 * 2^e = 1.984375 * 2^(e + 6)
            int e = (int)(m >> 7) - 133 + ((m & 127u) == 127u ? 1 : 0);
            e = m >= 0x7f80u ? 50 : max(-50, min(50, e));
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
            // lanes of the first half of the warp write the largest, of the second the smallest
            if (lane % 16 < C) {
                const bool up = lane < 16;
                uint32_t word[2] = {0u, 0u};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = up ? hi[i] : lo[i];
                    const int x = code_of(__uint_as_float(w << 16), inv, up);
                    const int y = code_of(__uint_as_float(w & 0xffff0000u), inv, up);
                    word[i / 2] |= ((uint32_t)(x & 255) | (uint32_t)(y & 255) << 8)
                                   << (16 * (i & 1));
                }
                const int64_t row = (int64_t)page * g.Hkv + hk;
                reinterpret_cast<uint2*>(bounds + row * 2 * D + (up ? 0 : D))[lane % C] =
                    make_uint2(word[0], word[1]);
                if (lane == 0) scale[row] = __uint_as_float((uint32_t)(127 + e) << 23);
            }
        }
    }
}

}  // namespace

cudaError_t launch_page_bounds(const CacheGeom& g, const void* k, const int32_t* slots,
                               int8_t* bounds, float* scale, int32_t* err,
                               cudaStream_t stream) {
    // rows of a CTA: a sequence's new ones, which lie in a page or two, up to four pages
    // (8 prompts of 4096 .. 16384 tokens, pages of 64: 27 us with two or four, 29 with one,
    // 39 with eight)
    const int rows = std::max(1, std::min(g.max_q_len, 4 * g.ps));
    const dim3 grid((g.total_q + rows - 1) / rows, g.Hkv);
    auto kern = g.D == 128 ? bounds_kernel<128> : bounds_kernel<64>;
    return launch_dependent(kern, grid, dim3(kThreads), 0, stream, g, (const __nv_bfloat16*)k,
                            slots, bounds, scale, err, rows);
}

}  // namespace pa
