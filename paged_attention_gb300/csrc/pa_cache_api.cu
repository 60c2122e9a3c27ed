// pa_cache_api.cu -- the entry points of pa_cache.h: argument checks and launches.
#include <cmath>
#include <mutex>

#include "pa_cache_common.cuh"

namespace pa {

cudaError_t launch_append(const CacheGeom& g, bool mx4, const void* k_new, const void* v_new,
                          int64_t k_stride, int64_t v_stride, const int32_t* table,
                          const int32_t* ctx, const int32_t* ql, void* k_cache, void* k_scale,
                          void* v_cache, void* v_scale, float* weights, int32_t* err, int sms,
                          cudaStream_t stream);
cudaError_t launch_expand(const CacheGeom& g, const void* k_cache, const void* k_scale,
                          const void* v_cache, const void* v_scale, const int32_t* table,
                          const int32_t* ctx, const int32_t* ql, const int32_t* dst_table,
                          int dst_mpps, int dst_pages, void* k_out, void* v_out, int32_t* err,
                          int sms, cudaStream_t stream);
int mx4_row_tiles(int D, int rows);
int mx4_ctas_per_sm(int D, int nt);
cudaError_t launch_decode_mx4(const CacheGeom& g, int nt, const void* q, const void* k,
                              const void* ks, const void* v, const void* vs, const int32_t* table,
                              const int32_t* ctx, const int32_t* ql, int32_t* header,
                              int32_t* done, float* part_o, float* part_lse, void* out, float* lse,
                              int unit_cost, int grid, cudaStream_t stream);
cudaError_t launch_key_weights(const CacheGeom& g, bool mx4, const void* q, const void* k,
                               const void* ks, const int32_t* table, const int32_t* ctx,
                               const int32_t* ql, const float* lse, float* weights, int32_t* err,
                               int sms, cudaStream_t stream);
cudaError_t launch_evict(const CacheGeom& g, bool mx4, int budget, int num_first, int num_recent,
                         void* k, void* ks, void* v, void* vs, float* weights,
                         const int32_t* table, const int32_t* dst_table, int dst_mpps,
                         const int32_t* ctx, int32_t* kept, int32_t* new_ctx, int32_t* err, int sms,
                         cudaStream_t stream);

namespace {

constexpr int kMaxGrid = 1024;          // CTAs of pa_decode_mx4
constexpr int kMaxHeads = 1 << 15;      // KV heads
// A unit's fixed cost (its first loads, its warps' merge), in 64-key tiles.  64
// sequences of 128 .. 32768 tokens, 8 rows: 154 us with 0, 112 with 4, 105 with 8,
// 109 with 12; 128 of 1024 .. 16384 tokens, 24 rows: 533, 512, 497 and 492.
constexpr int mx4_unit_cost(int rows) { return rows > 16 ? 12 : 8; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

int sm_count() {
    constexpr int kMaxDevices = 64;
    static std::mutex mu;
    static int count[kMaxDevices] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    std::lock_guard<std::mutex> lk(mu);
    if (count[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return -1;
        count[dev] = n;
    }
    return count[dev];
}

// The fields every cache operator relies on.
pa_status geometry(const pa_problem* pp, bool queries, CacheGeom& g) {
    if (!pp) return PA_ERR_INVALID_ARG;
    const pa_problem& p = *pp;
    if (p.num_seqs < 1 || p.num_q_heads < 1 || p.num_kv_heads < 1 ||
        p.num_q_heads % p.num_kv_heads != 0 || p.num_pages < 1 || p.max_pages_per_seq < 1 ||
        p.total_q_tokens < 0 || p.max_q_len < 0 || p.max_context_len < 0 ||
        p.max_context_len < p.max_q_len || p.num_ctas < 0 || !std::isfinite(p.sm_scale) ||
        p.sm_scale < 0.f || p.window < 0)
        return PA_ERR_INVALID_ARG;
    if (p.mask_q_tiles != 0 || p.mask_kv_tiles != 0) return PA_ERR_INVALID_ARG;
    if (p.layout != PA_NHD && p.layout != PA_HND) return PA_ERR_INVALID_ARG;
    if (p.kv_dtype != PA_BF16 && p.kv_dtype != PA_FP8_E4M3 && p.kv_dtype != PA_MX4)
        return PA_ERR_INVALID_ARG;
    if (p.q_dtype != PA_BF16 || p.kv_dtype == PA_FP8_E4M3) return PA_ERR_UNSUPPORTED;
    if (p.head_dim != 64 && p.head_dim != 128) return PA_ERR_UNSUPPORTED;
    int shift = 4;
    while (shift < 9 && (1 << shift) != p.page_size) ++shift;
    if (shift == 9) return PA_ERR_UNSUPPORTED;
    if (p.num_kv_heads > kMaxHeads) return PA_ERR_UNSUPPORTED;
    if ((int64_t)p.max_pages_per_seq * p.page_size < p.max_context_len) return PA_ERR_INVALID_ARG;
    if ((int64_t)p.max_context_len > (1 << 30)) return PA_ERR_UNSUPPORTED;
    if (queries && p.total_q_tokens > 0 && p.max_q_len == 0) return PA_ERR_INVALID_ARG;
    if ((int64_t)p.num_seqs * p.max_q_len > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    if ((int64_t)p.num_seqs * p.num_kv_heads > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    const int G = p.num_q_heads / p.num_kv_heads;
    if ((int64_t)G * p.max_q_len > (1 << 30)) return PA_ERR_UNSUPPORTED;
    g.B = p.num_seqs;
    g.Hq = p.num_q_heads;
    g.Hkv = p.num_kv_heads;
    g.G = G;
    g.D = p.head_dim;
    g.ps = p.page_size;
    g.ps_shift = shift;
    g.num_pages = p.num_pages;
    g.mpps = p.max_pages_per_seq;
    g.total_q = p.total_q_tokens;
    g.max_q_len = p.max_q_len;
    g.max_ctx = p.max_context_len;
    g.window = p.window;
    g.tok_rows = p.layout == PA_NHD ? p.num_kv_heads : 1;
    g.head_rows = p.layout == PA_NHD ? 1 : p.page_size;
    g.sm_scale = p.sm_scale;
    return PA_OK;
}

// A cache and, for PA_MX4, its scales.
bool cache_ok(const pa_problem& p, const void* cache, const void* scale) {
    if (!cache || !aligned(cache, 16)) return false;
    return p.kv_dtype != PA_MX4 || (scale && aligned(scale, 16));
}
bool lens_ok(const int32_t* table, const int32_t* ctx, const int32_t* ql) {
    return table && ctx && ql && aligned(table, 4) && aligned(ctx, 4) && aligned(ql, 4);
}
pa_status status_of(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// Workspace of pa_decode_mx4: header (error word) and the counters of as many
// CTAs as a call may have, then two partial slots per CTA, each `rows` rows of D +
// 1 floats.  The partials begin at the same place whatever the grid: no call
// writes them where another finds its counters.
struct Mx4Layout {
    int grid, nt, unit_cost;
    int64_t off_done, off_part, rows, total;
};
pa_status mx4_layout(const pa_problem* pp, CacheGeom& g, Mx4Layout& L) {
    pa_status st = geometry(pp, true, g);
    if (st != PA_OK) return st;
    if (pp->kv_dtype != PA_MX4) return PA_ERR_UNSUPPORTED;
    L.nt = mx4_row_tiles(g.D, g.G * (g.max_q_len > 0 ? g.max_q_len : 1));
    if (L.nt < 0) return PA_ERR_UNSUPPORTED;
    if (pp->num_ctas > kMaxGrid) return PA_ERR_UNSUPPORTED;
    L.grid = pp->num_ctas;
    if (L.grid == 0) {
        L.grid = sm_count();
        if (L.grid <= 0) return PA_ERR_CUDA;
        L.grid *= mx4_ctas_per_sm(g.D, L.nt);
        if (L.grid > kMaxGrid) L.grid = kMaxGrid;
    }
    L.unit_cost = pp->unit_cost > 0 ? pp->unit_cost : pp->unit_cost < 0 ? 0 : mx4_unit_cost(8 * L.nt);
    L.rows = 8 * L.nt;
    L.off_done = kHeaderWords * 4;
    L.off_part = align256(L.off_done + (int64_t)kMaxGrid * 4);
    L.total = align256(L.off_part + 2 * (int64_t)L.grid * L.rows * (g.D + 1) * 4);
    return PA_OK;
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_kv_append(const pa_problem* problem, const void* k_new, const void* v_new,
                       int64_t k_stride, int64_t v_stride, const int32_t* block_table,
                       const int32_t* context_lens, const int32_t* q_lens, void* k_cache,
                       void* k_scale, void* v_cache, void* v_scale, float* key_weights,
                       int32_t* device_error, void* stream) {
    CacheGeom g;
    pa_status st = geometry(problem, true, g);
    if (st != PA_OK) return st;
    if (g.total_q == 0) return PA_OK;   // no new token
    const int64_t row = (int64_t)g.Hkv * g.D;
    if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16) || k_stride < row ||
        v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0 ||
        !lens_ok(block_table, context_lens, q_lens) || !cache_ok(*problem, k_cache, k_scale) ||
        !cache_ok(*problem, v_cache, v_scale) || !aligned(key_weights, 4) ||
        !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_append(g, problem->kv_dtype == PA_MX4, k_new, v_new, k_stride,
                                   v_stride, block_table, context_lens, q_lens, k_cache, k_scale,
                                   v_cache, v_scale, key_weights, device_error, sms,
                                   (cudaStream_t)stream));
}

pa_status pa_kv_expand(const pa_problem* problem, const void* k_cache, const void* k_scale,
                       const void* v_cache, const void* v_scale, const int32_t* block_table,
                       const int32_t* context_lens, const int32_t* q_lens,
                       const int32_t* dst_block_table, int32_t dst_max_pages_per_seq,
                       int32_t dst_num_pages, void* k_out, void* v_out, int32_t* device_error,
                       void* stream) {
    CacheGeom g;
    pa_status st = geometry(problem, true, g);
    if (st != PA_OK) return st;
    if (problem->kv_dtype != PA_MX4) return PA_ERR_UNSUPPORTED;
    if (dst_max_pages_per_seq < 1 || dst_num_pages < 1 ||
        (int64_t)dst_max_pages_per_seq * g.ps < g.max_ctx)
        return PA_ERR_INVALID_ARG;
    if (g.total_q == 0) return PA_OK;   // nothing to read back
    if (!lens_ok(block_table, context_lens, q_lens) || !cache_ok(*problem, k_cache, k_scale) ||
        !cache_ok(*problem, v_cache, v_scale) || !dst_block_table || !aligned(dst_block_table, 4) ||
        !k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16) ||
        !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_expand(g, k_cache, k_scale, v_cache, v_scale, block_table,
                                   context_lens, q_lens, dst_block_table, dst_max_pages_per_seq,
                                   dst_num_pages, k_out, v_out, device_error, sms,
                                   (cudaStream_t)stream));
}

size_t pa_mx4_workspace_size(const pa_problem* problem) {
    CacheGeom g;
    Mx4Layout L;
    return mx4_layout(problem, g, L) == PA_OK ? (size_t)L.total : 0;
}

pa_status pa_decode_mx4(const pa_problem* problem, const void* q, const void* k_cache,
                        const void* k_scale, const void* v_cache, const void* v_scale,
                        const int32_t* block_table, const int32_t* context_lens,
                        const int32_t* q_lens, void* ws, size_t ws_bytes, void* out, float* lse,
                        void* stream) {
    CacheGeom g;
    Mx4Layout L;
    pa_status st = mx4_layout(problem, g, L);
    if (st != PA_OK) return st;
    if (!ws || !aligned(ws, 256)) return PA_ERR_INVALID_ARG;
    if (ws_bytes < (size_t)L.total) return PA_ERR_WORKSPACE;
    const bool rows = g.total_q > 0;
    if (rows && (!q || !aligned(q, 16) || !cache_ok(*problem, k_cache, k_scale) ||
                 !cache_ok(*problem, v_cache, v_scale) ||
                 !lens_ok(block_table, context_lens, q_lens) || !out || !aligned(out, 16) ||
                 !aligned(lse, 4)))
        return PA_ERR_INVALID_ARG;
    if (!rows) return PA_OK;   // no query row: nothing to compute
    char* base = static_cast<char*>(ws);
    float* part_o = reinterpret_cast<float*>(base + L.off_part);
    return status_of(launch_decode_mx4(
        g, L.nt, q, k_cache, k_scale, v_cache, v_scale, block_table, context_lens, q_lens,
        reinterpret_cast<int32_t*>(base), reinterpret_cast<int32_t*>(base + L.off_done), part_o,
        part_o + 2 * (int64_t)L.grid * L.rows * g.D, out, lse, L.unit_cost, L.grid, (cudaStream_t)stream));
}

pa_status pa_key_weights(const pa_problem* problem, const void* q, const void* k_cache,
                         const void* k_scale, const int32_t* block_table,
                         const int32_t* context_lens, const int32_t* q_lens, const float* lse,
                         float* key_weights, int32_t* device_error, void* stream) {
    CacheGeom g;
    pa_status st = geometry(problem, true, g);
    if (st != PA_OK) return st;
    if (g.total_q == 0) return PA_OK;   // no query
    if (!q || !aligned(q, 16) || !cache_ok(*problem, k_cache, k_scale) ||
        !lens_ok(block_table, context_lens, q_lens) || !lse || !aligned(lse, 4) || !key_weights ||
        !aligned(key_weights, 4) || !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_key_weights(g, problem->kv_dtype == PA_MX4, q, k_cache, k_scale,
                                        block_table, context_lens, q_lens, lse, key_weights,
                                        device_error, sms, (cudaStream_t)stream));
}

pa_status pa_kv_evict(const pa_problem* problem, int32_t budget, int32_t num_first,
                      int32_t num_recent, void* k_cache, void* k_scale, void* v_cache,
                      void* v_scale, float* key_weights, const int32_t* block_table,
                      const int32_t* dst_block_table, int32_t dst_max_pages_per_seq,
                      const int32_t* context_lens, int32_t* kept, int32_t* new_context_lens,
                      int32_t* device_error, void* stream) {
    CacheGeom g;
    pa_status st = geometry(problem, false, g);
    if (st != PA_OK) return st;
    if (budget < 1 || num_first < 0 || num_recent < 0 ||
        (int64_t)num_first + num_recent > budget || dst_max_pages_per_seq < 1 ||
        (g.max_ctx > budget && (int64_t)dst_max_pages_per_seq * g.ps < budget))
        return PA_ERR_INVALID_ARG;
    const char* c0 = reinterpret_cast<const char*>(context_lens);
    const char* n0 = reinterpret_cast<const char*>(new_context_lens);
    const int64_t len_bytes = (int64_t)g.B * 4;
    if (!cache_ok(*problem, k_cache, k_scale) || !cache_ok(*problem, v_cache, v_scale) ||
        !key_weights || !aligned(key_weights, 4) || !block_table || !aligned(block_table, 4) ||
        !dst_block_table || !aligned(dst_block_table, 4) || dst_block_table == block_table ||
        !context_lens || !aligned(context_lens, 4) || !kept || !aligned(kept, 4) ||
        !new_context_lens || !aligned(new_context_lens, 4) ||
        (n0 < c0 + len_bytes && c0 < n0 + len_bytes) || !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_evict(g, problem->kv_dtype == PA_MX4, budget, num_first, num_recent,
                                  k_cache, k_scale, v_cache, v_scale, key_weights, block_table,
                                  dst_block_table, dst_max_pages_per_seq, context_lens, kept,
                                  new_context_lens, device_error, sms, (cudaStream_t)stream));
}

}  // extern "C"
