// pa_cache_common.cuh -- shared by the cache operators (pa_cache.h): launch
// parameters, the geometry of paged rows, finding sequences from q_lens on the
// device, and the E2M1 / E8M0 conversions of the PA_MX4 cache.
#pragma once

#include <atomic>

#include "pa_cache.h"
#include "pa_internal.cuh"

namespace pa {

// What every cache kernel needs to know of the problem.
struct CacheGeom {
    int32_t B, Hq, Hkv, G, D;
    int32_t ps, ps_shift;        // page size and its log2
    int32_t num_pages, mpps;     // pages in the pool, row stride of block_table
    int32_t total_q, max_q_len, max_ctx;
    int32_t window;
    int32_t tok_rows, head_rows; // rows between tokens / heads of a page (NHD: Hkv, 1; HND: 1, ps)
    float sm_scale;
};

// Row index (of Hkv * ps per page) of (page, slot, head).
__device__ __forceinline__ int64_t row_of(const CacheGeom& g, int page, int slot, int head) {
    return (int64_t)page * g.ps * g.Hkv + (int64_t)slot * g.tok_rows + (int64_t)head * g.head_rows;
}

// Every kernel of the cache operators is launched as a dependent of the kernel
// before it on the stream (launch_dependent) and waits for that kernel, and for
// what it wrote, before it does anything else: launches of a serving step's row
// of short kernels then overlap (three short sequences decoded: 8.4 -> 6.9 us a
// call).  None lets the next one start before it ends: CTAs that wait take room
// from those that run (evict 32 prompts: 129 us, with an early start 145; decode
// 64 sequences: 105 and 111).

__device__ __forceinline__ void flag_error(int32_t* err, int code) {
    if (err != nullptr) atomicOr(err, code);
}

// Lengths of sequence b that attention accepts.
__device__ __forceinline__ bool good_lens(const CacheGeom& g, int q, int c) {
    return q >= 0 && c >= q && c <= g.max_ctx && q <= g.max_q_len;
}
// What a sequence adds to the offsets of the rows after it, whatever its length says.
__device__ __forceinline__ int clamp_q(const CacheGeom& g, int q) {
    return max(0, min(q, g.max_q_len));
}

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// The sequence whose new tokens hold row `t` (per lane; the warp calls it
// together): its index, or -1, and in `start` its first row.
__device__ __forceinline__ int seq_of_row(const CacheGeom& g, const int32_t* ql, int t, int lane,
                                          int& start) {
    int found = -1, run = 0;
    for (int c0 = 0; c0 < g.B; c0 += 32) {
        const int v = c0 + lane < g.B ? clamp_q(g, ql[c0 + lane]) : 0;
        const int inc = warp_inclusive(v, lane) + run;
        const int end = __shfl_sync(0xffffffffu, inc, 31);
        // the first i whose inclusive sum exceeds t
        int i = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int x = __shfl_sync(0xffffffffu, inc, i + o - 1);
            if (x <= t) i += o;
        }
        const int q = __shfl_sync(0xffffffffu, v, i), e = __shfl_sync(0xffffffffu, inc, i);
        if (found < 0 && t >= run && t < end) {
            found = c0 + i;
            start = e - q;
        }
        run = end;
        if (__all_sync(0xffffffffu, found >= 0)) break;
    }
    return found;
}

// One warp checks what no single row's owner can see: every sequence's
// lengths, and that the q_lens add up to the rows there are.
__device__ __forceinline__ void check_lens(const CacheGeom& g, const int32_t* ctx,
                                           const int32_t* ql, int lane, int32_t* err) {
    int64_t sum = 0;
    bool bad = false;
    for (int b = lane; b < g.B; b += 32) {
        const int q = ql[b];
        bad |= !good_lens(g, q, ctx[b]);
        sum += clamp_q(g, q);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (__any_sync(0xffffffffu, bad || sum != g.total_q) && lane == 0)
        flag_error(err, PA_DEV_BAD_LENGTHS);
}

// Lets a kernel take up to `bytes` (the same in every call) of dynamic shared
// memory on the current device; asked of the runtime once per kernel and device.
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};          // a bit per device
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
    const cudaError_t f =
        cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (f == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return f;
}

// ------------------------------------------------------------- E2M1 / E8M0

// The eight E2M1 codes of a word as four f16x2 (exact): byte j -> elements 2j, 2j + 1.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& h0, uint32_t& h1, uint32_t& h2,
                                              uint32_t& h3) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
        : "r"(w));
}

// Two floats -> one byte of E2M1 codes, round to nearest even, saturating
// (lo in the low four bits).
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
    uint32_t d;
    asm("{\n\t.reg .b8 b, z;\n\t"
        "mov.b32 {z, z, z, z}, 0;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
        "mov.b32 %0, {b, z, z, z};\n\t}"
        : "=r"(d)
        : "f"(hi), "f"(lo));
    return d;
}

// 2^(e - 127) as fp32; e = 255 is NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t e) {
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23);
}

}  // namespace pa
