// pa_cache_host.cuh -- argument checks that the entry points of pa_cache.h and pa_step.h share.
#pragma once

#include "pa_cache_common.cuh"

namespace pa {

// SMs of the current device, -1 if it cannot be asked.
int sm_count();
// The fields every operator relies on (`queries`: rows need a max_q_len).
pa_status geometry(const pa_problem* problem, bool queries, CacheGeom& g);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// A cache and, for PA_MX4, its scales.
inline bool cache_ok(const pa_problem& p, const void* cache, const void* scale) {
    if (!cache || !aligned(cache, 16)) return false;
    return p.kv_dtype != PA_MX4 || (scale && aligned(scale, 16));
}
// Whether a kernel can count a call's work on one line: a unit of up to `tiles` tiles and its
// fixed cost in 32 bits, and all units, times the CTAs of a grid (2^10 at most), in 64.
inline bool line_fits(int64_t units, int64_t tiles, int unit_cost) {
    const int64_t each = tiles + unit_cost;
    return each <= 0x7fffffff && (units <= 0 || each <= ((int64_t)1 << 52) / units);
}
inline bool ints_ok(const void* p) { return p && aligned(p, 4); }
inline bool lens_ok(const int32_t* table, const int32_t* ctx, const int32_t* ql) {
    return ints_ok(table) && ints_ok(ctx) && ints_ok(ql);
}
inline pa_status status_of(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

}  // namespace pa
