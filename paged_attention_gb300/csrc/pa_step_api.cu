// pa_step_api.cu -- the entry points of pa_step.h: argument checks and launches, and
// the frequencies of rotary positions, which are worked out on the host.
#include <algorithm>
#include <cmath>

#include "pa_cache_host.cuh"
#include "pa_step_common.cuh"

namespace pa {

namespace {

constexpr int kMaxGridSel = 1024;        // CTAs of pa_decode_selected
// A unit's fixed cost (its first loads, its warps' merge), in 64-key tiles, which are half
// the bytes with head_dim 64.  64 rows of up to 32 pages of 64: 61 us with 1 to 8, 62 with
// 12; head_dim 64 46.8 with 1, 40.2 with 3, 38.0 with 6; 64 sequences of 4 rows (16 query rows a
// unit) 75.2 with 3, 72.7 with 6, 75.5 with 12; of 64 q heads (32) 109 with 4, 89 with 8 and 10;
// 128 sequences of 3 rows (24) 211 with 3, 207 with 6, 206 with 10 and 12.
constexpr int sel_unit_cost(int D, int rows) {
    return (rows > 16 ? 10 : rows > 8 ? 6 : 3) * 128 / D;
}

// Memory that a call reads, or writes.
struct Span {
    const void* at;
    int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}
// Whether one of the first `outputs` spans overlaps any other.
template <int N>
bool overlap(const Span (&s)[N], int outputs) {
    for (int i = 0; i < outputs; ++i)
        for (int j = i + 1; j < N; ++j)
            if (overlap(s[i], s[j])) return true;
    return false;
}

// (no more than addresses have room for)
int64_t table_bytes(const CacheGeom& g) {
    return std::min((int64_t)g.B * g.mpps, (int64_t)1 << 56) * 4;
}

// Pages are pages whatever they hold: E4M3 caches have them too.
pa_status page_geometry(const pa_problem* pp, CacheGeom& g) {
    if (!pp) return PA_ERR_INVALID_ARG;
    pa_problem p = *pp;
    if (p.kv_dtype == PA_FP8_E4M3) p.kv_dtype = PA_BF16;
    if (p.q_dtype == PA_FP8_E4M3) p.q_dtype = PA_BF16;
    return geometry(&p, false, g);
}
bool slots_fit(const CacheGeom& g) { return (int64_t)g.num_pages * g.ps <= 0x7fffffff; }
// Rows that 32 bits count with room for a grid's step beyond.
bool rows_fit(const CacheGeom& g) { return g.total_q <= 1 << 30; }

// Workspace of pa_decode_selected: header (error word) and the counters, one a query
// row, of as many CTAs as a call may have, then two partial slots per CTA, each `rows` rows of D +
// 1 floats; where several rows of a sequence may be one unit, the units and their
// joined lists.
struct SelLayout {
    int grid, nt, unit_cost;
    int together;        // rows of a sequence in a unit, at most
    int64_t off_done, off_part, rows, off_lead, off_entries, off_list, total;
};
pa_status sel_layout(const pa_problem* pp, int budget, CacheGeom& g, SelLayout& L) {
    const pa_status st = geometry(pp, false, g);
    if (st != PA_OK) return st;
    if (budget < 1) return PA_ERR_INVALID_ARG;
    if (pp->kv_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (g.G > (g.D == 128 ? 32 : 64)) return PA_ERR_UNSUPPORTED;
    L.together = selected_rows(g.G, g.max_q_len);
    L.nt = selected_row_tiles(g.D, g.G * L.together);
    if (L.nt < 0 || pp->num_ctas > kMaxGridSel) return PA_ERR_UNSUPPORTED;
    if (!rows_fit(g) || (int64_t)g.total_q * g.Hkv > 0x7fffffff) return PA_ERR_UNSUPPORTED;
    L.grid = pp->num_ctas;
    if (L.grid == 0) {
        L.grid = sm_count();
        if (L.grid <= 0) return PA_ERR_CUDA;
        L.grid *= selected_ctas_per_sm();
        if (L.grid > kMaxGridSel) L.grid = kMaxGridSel;
    }
    L.unit_cost = pp->unit_cost > 0   ? pp->unit_cost
                  : pp->unit_cost < 0 ? 0
                                      : sel_unit_cost(g.D, 8 * L.nt);
    // (a unit's list has no page twice, nor more than its rows' lists together)
    const int64_t pages = std::min(((int64_t)g.max_ctx + g.ps - 1) >> g.ps_shift,
                                   (int64_t)L.together * budget);
    if (!line_fits((int64_t)g.total_q * g.Hkv,
                   ((pages << g.ps_shift) + kDecodeTile - 1) / kDecodeTile, L.unit_cost))
        return PA_ERR_UNSUPPORTED;
    L.rows = 8 * L.nt;
    L.off_done = kHeaderWords * 4;
    L.off_part = align256(L.off_done + (int64_t)kMaxGridSel * kSelDoneRows * 4);
    L.off_lead = align256(L.off_part + 2 * (int64_t)L.grid * L.rows * (g.D + 1) * 4);
    L.off_entries = L.off_list = L.total = L.off_lead;
    if (L.together > 1) {
        const int64_t units = (int64_t)g.total_q * g.Hkv;
        // (a size that 64 bits hold: below 2^60)
        if (units > 0 && budget > ((int64_t)1 << 56) / units) return PA_ERR_UNSUPPORTED;
        L.off_entries = align256(L.off_lead + (int64_t)g.total_q * (1 + kMostJoinParts) * 4);
        L.off_list = align256(L.off_entries + units * 4);
        L.total = align256(L.off_list + units * budget * 8);
    }
    return PA_OK;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

pa_status pa_pages_take(const pa_problem* problem, const int32_t* seq_lens, const int32_t* q_lens,
                        int32_t* block_table, const int32_t* free_pages,
                        const int32_t* free_count, int32_t* context_lens, int32_t* row_seq,
                        int32_t* positions, int32_t* slots, int32_t* free_left,
                        int32_t* device_error, void* stream) {
    CacheGeom g;
    pa_status st = page_geometry(problem, g);
    if (st != PA_OK) return st;
    if (!slots_fit(g) || !rows_fit(g)) return PA_ERR_UNSUPPORTED;
    const bool rows = g.total_q > 0;
    if (!ints_ok(seq_lens) || !ints_ok(q_lens) || !ints_ok(block_table) || !ints_ok(free_pages) ||
        !ints_ok(free_count) || !ints_ok(context_lens) || !ints_ok(free_left) ||
        (rows && (!ints_ok(row_seq) || !ints_ok(positions) || !ints_ok(slots))) ||
        !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    // every CTA reads what others would overwrite, rounds of sequences after it has written rows
    const int64_t n = (int64_t)g.B * 4, t = (int64_t)g.total_q * 4;
    const Span spans[] = {{context_lens, n},
                          {free_left, 4},
                          {row_seq, t},
                          {positions, t},
                          {slots, t},
                          {block_table, table_bytes(g)},
                          {seq_lens, n},
                          {q_lens, n},
                          {free_pages, (int64_t)g.num_pages * 4},
                          {free_count, 4}};
    if (overlap(spans, 6)) return PA_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_pages_take(g, seq_lens, q_lens, block_table, free_pages, free_count,
                                       context_lens, row_seq, positions, slots, free_left,
                                       device_error, sms, (cudaStream_t)stream));
}

pa_status pa_pages_return(const pa_problem* problem, const int32_t* seq_lens,
                          const int32_t* keep_lens, const int32_t* block_table,
                          int32_t* free_pages, const int32_t* free_count, int32_t* free_left,
                          int32_t* device_error, void* stream) {
    CacheGeom g;
    pa_status st = page_geometry(problem, g);
    if (st != PA_OK) return st;
    if (!ints_ok(seq_lens) || !ints_ok(keep_lens) || !ints_ok(block_table) ||
        !ints_ok(free_pages) || !ints_ok(free_count) || !ints_ok(free_left) ||
        !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)g.B * 4;
    const Span spans[] = {{free_pages, (int64_t)g.num_pages * 4},
                          {free_left, 4},
                          {block_table, table_bytes(g)},
                          {seq_lens, n},
                          {keep_lens, n},
                          {free_count, 4}};
    if (overlap(spans, 2)) return PA_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_pages_return(g, seq_lens, keep_lens, block_table, free_pages,
                                         free_count, free_left, device_error, sms,
                                         (cudaStream_t)stream));
}

pa_status pa_rope_inv_freq(const pa_rope_scaling* s, double* inv_freq, double* cos_sin_scale) {
    if (!s || !inv_freq || !cos_sin_scale) return PA_ERR_INVALID_ARG;
    const int d = s->rotary_dim;
    if (d < 2 || d > 128 || d % 2 != 0 || !(s->base > 1.0) || !std::isfinite(s->base) ||
        s->kind < PA_ROPE_NONE || s->kind > PA_ROPE_BANDS)
        return PA_ERR_INVALID_ARG;
    const bool ends = s->kind == PA_ROPE_YARN || s->kind == PA_ROPE_BANDS;
    if (s->kind != PA_ROPE_NONE && !(s->factor >= 1.0 && std::isfinite(s->factor)))
        return PA_ERR_INVALID_ARG;
    if (s->kind == PA_ROPE_NTK && d == 2) return PA_ERR_INVALID_ARG;
    if (ends && !(s->original_context >= 1.0 && std::isfinite(s->original_context) &&
                  s->low_turns > 0.0 && s->high_turns > s->low_turns &&
                  std::isfinite(s->high_turns)))
        return PA_ERR_INVALID_ARG;
    double base = s->base;
    if (s->kind == PA_ROPE_NTK) base *= std::pow(s->factor, (double)d / (d - 2));
    // YARN: the pair indices that make `turns` turns over the original context
    auto index_of = [&](double turns) {
        return d * std::log(s->original_context / (turns * kTwoPi)) / (2 * std::log(base));
    };
    double lo = 0, hi = 1;
    if (s->kind == PA_ROPE_YARN) {
        lo = std::fmax(0.0, std::floor(index_of(s->high_turns)));
        hi = std::fmin(d - 1.0, std::ceil(index_of(s->low_turns)));
        // (where no pair makes more than low_turns, or all make more than high_turns, the ends
        // as they were cut would meet or cross: all pairs are divided, or none)
        if (hi <= 0.0) {
            lo = -1.0;
            hi = 0.0;
        } else if (hi <= lo) {
            hi = lo + 0.001;
        }
    }
    for (int i = 0; i < d / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / d);
        double scaled = 1.0;                 // how much of the pair is divided by the factor
        if (s->kind == PA_ROPE_NONE || s->kind == PA_ROPE_NTK) scaled = 0.0;
        if (s->kind == PA_ROPE_YARN) scaled = std::fmin(1.0, std::fmax(0.0, (i - lo) / (hi - lo)));
        if (s->kind == PA_ROPE_BANDS) {
            const double turns = s->original_context * f / kTwoPi;
            const double kept = (turns - s->low_turns) / (s->high_turns - s->low_turns);
            scaled = 1.0 - std::fmin(1.0, std::fmax(0.0, kept));
        }
        inv_freq[i] = scaled == 0.0 ? f : f / s->factor * scaled + f * (1.0 - scaled);
    }
    *cos_sin_scale = s->kind == PA_ROPE_YARN ? 0.1 * std::log(s->factor) + 1.0 : 1.0;
    return PA_OK;
}

pa_status pa_rope_steps(const double* inv_freq, int32_t count, uint64_t* steps) {
    if (!inv_freq || !steps || count < 1) return PA_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i)
        if (!std::isfinite(inv_freq[i])) return PA_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const double turns = inv_freq[i] / kTwoPi;
        const double frac = turns - std::floor(turns);   // in [0, 1]
        const double x = std::ldexp(frac, 64);
        steps[i] = x >= 18446744073709551616.0 ? 0u : (uint64_t)x;
    }
    return PA_OK;
}

pa_status pa_rope_append(const pa_problem* problem, const pa_rope* rope, const uint64_t* steps,
                         const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const int32_t* positions,
                         const int32_t* slots, void* q_out, void* k_cache, void* k_scale,
                         void* v_cache, void* v_scale, int32_t* device_error, void* stream) {
    RopeParams P;
    pa_status st = geometry(problem, false, P.g);
    if (st != PA_OK) return st;
    const CacheGeom& g = P.g;
    if (!rope || !std::isfinite(rope->cos_sin_scale) || rope->rotary_dim < 16 ||
        rope->rotary_dim > g.D || rope->rotary_dim % 16 != 0 ||
        (rope->interleaved != 0 && rope->interleaved != 1))
        return PA_ERR_INVALID_ARG;
    if (!slots_fit(g) || !rows_fit(g)) return PA_ERR_UNSUPPORTED;
    if (g.total_q == 0) return PA_OK;   // no new token
    const int64_t kv = (int64_t)g.Hkv * g.D, qd = (int64_t)g.Hq * g.D;
    if (!steps || !aligned(steps, 8) || !k_new || !v_new || !aligned(k_new, 16) ||
        !aligned(v_new, 16) || k_stride < kv || v_stride < kv || k_stride % 8 != 0 ||
        v_stride % 8 != 0 || !ints_ok(positions) || !ints_ok(slots) ||
        !cache_ok(*problem, k_cache, k_scale) || !cache_ok(*problem, v_cache, v_scale) ||
        !aligned(device_error, 4) || (q == nullptr) != (q_out == nullptr) || !aligned(q, 16) ||
        !aligned(q_out, 16) || (q != nullptr && (q_stride < qd || q_stride % 8 != 0)) ||
        (q != nullptr && q == q_out && q_stride != qd && g.total_q > 1))
        return PA_ERR_INVALID_ARG;
    if (q != nullptr) {
        // q is read row by row while others are written; in place a lane reads what it writes
        auto rows = [&](const void* x, int64_t stride, int64_t width) -> Span {
            return {x, ((g.total_q - 1) * stride + width) * 2};
        };
        const Span out = {q_out, g.total_q * qd * 2};
        if ((q != q_out && overlap(out, rows(q, q_stride, qd))) ||
            overlap(out, rows(k_new, k_stride, kv)) || overlap(out, rows(v_new, v_stride, kv)))
            return PA_ERR_INVALID_ARG;
    }
    P.rotary = rope->rotary_dim;
    P.interleaved = rope->interleaved;
    P.scale = rope->cos_sin_scale;
    P.steps = steps;
    P.q = (const __nv_bfloat16*)q;
    P.k = (const __nv_bfloat16*)k_new;
    P.v = (const __nv_bfloat16*)v_new;
    P.q_stride = q_stride;
    P.k_stride = k_stride;
    P.v_stride = v_stride;
    P.positions = positions;
    P.slots = slots;
    P.q_out = (__nv_bfloat16*)q_out;
    P.k_cache = k_cache;
    P.k_scale = (uint8_t*)k_scale;
    P.v_cache = v_cache;
    P.v_scale = (uint8_t*)v_scale;
    P.err = device_error;
    P.tokens = 0;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_rope(P, problem->kv_dtype == PA_MX4, sms, (cudaStream_t)stream));
}

pa_status pa_page_bounds(const pa_problem* problem, const void* k_cache, const int32_t* slots,
                         int8_t* bounds, float* bound_scale, int32_t* device_error,
                         void* stream) {
    CacheGeom g;
    pa_status st = geometry(problem, false, g);
    if (st != PA_OK) return st;
    if (problem->kv_dtype != PA_BF16 || !slots_fit(g) || !rows_fit(g)) return PA_ERR_UNSUPPORTED;
    if (g.total_q == 0) return PA_OK;   // no page got a new token
    if (!k_cache || !aligned(k_cache, 16) || !ints_ok(slots) || !bounds || !aligned(bounds, 16) ||
        !bound_scale || !aligned(bound_scale, 4) || !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    return status_of(launch_page_bounds(g, k_cache, slots, bounds, bound_scale, device_error,
                                        (cudaStream_t)stream));
}

pa_status pa_select_pages(const pa_problem* problem, int32_t budget, int32_t num_first,
                          int32_t num_recent, const void* q, const int8_t* bounds,
                          const float* bound_scale, const int32_t* block_table,
                          const int32_t* row_seq, const int32_t* positions, int32_t* selected,
                          int32_t* device_error, void* stream) {
    SelectParams P;
    pa_status st = page_geometry(problem, P.g);
    if (st != PA_OK) return st;
    const CacheGeom& g = P.g;
    if (budget < 1 || num_first < 0 || num_recent < 0 ||
        (int64_t)num_first + num_recent > budget)
        return PA_ERR_INVALID_ARG;
    if (g.G > 64 || ((int64_t)g.max_ctx + g.ps - 1) / g.ps > PA_MAX_SELECT_PAGES ||
        (int64_t)g.total_q * g.Hkv > 0x7fffffff / 8)
        return PA_ERR_UNSUPPORTED;
    if (g.total_q == 0) return PA_OK;   // no query
    if (!q || !aligned(q, 16) || !bounds || !aligned(bounds, 16) || !bound_scale ||
        !aligned(bound_scale, 4) || !ints_ok(block_table) || !ints_ok(row_seq) ||
        !ints_ok(positions) || !ints_ok(selected) || !aligned(device_error, 4))
        return PA_ERR_INVALID_ARG;
    P.budget = budget;
    P.num_first = num_first;
    P.num_recent = num_recent;
    P.q = (const __nv_bfloat16*)q;
    P.bounds = bounds;
    P.scale = bound_scale;
    P.table = block_table;
    P.row_seq = row_seq;
    P.positions = positions;
    P.selected = selected;
    P.err = device_error;
    P.cluster = 1;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(launch_select(P, sms, (cudaStream_t)stream));
}

size_t pa_selected_workspace_size(const pa_problem* problem, int32_t budget) {
    CacheGeom g;
    SelLayout L;
    return sel_layout(problem, budget, g, L) == PA_OK ? (size_t)L.total : 0;
}

pa_status pa_decode_selected(const pa_problem* problem, int32_t budget, const void* q,
                             const void* k_cache, const void* v_cache, const int32_t* block_table,
                             const int32_t* row_seq, const int32_t* positions,
                             const int32_t* selected, void* ws, size_t ws_bytes, void* out,
                             float* lse, void* stream) {
    SelectedParams P;
    SelLayout L;
    pa_status st = sel_layout(problem, budget, P.g, L);
    if (st != PA_OK) return st;
    const CacheGeom& g = P.g;
    if (!ws || !aligned(ws, 256)) return PA_ERR_INVALID_ARG;
    if (ws_bytes < (size_t)L.total) return PA_ERR_WORKSPACE;
    if (g.total_q == 0) return PA_OK;   // no query row: nothing to compute
    if (!q || !aligned(q, 16) || !k_cache || !aligned(k_cache, 16) || !v_cache ||
        !aligned(v_cache, 16) || !ints_ok(block_table) || !ints_ok(row_seq) ||
        !ints_ok(positions) || !ints_ok(selected) || !out || !aligned(out, 16) ||
        !aligned(lse, 4))
        return PA_ERR_INVALID_ARG;
    char* base = static_cast<char*>(ws);
    P.budget = budget;
    P.q = (const __nv_bfloat16*)q;
    P.k = (const __nv_bfloat16*)k_cache;
    P.v = (const __nv_bfloat16*)v_cache;
    P.table = block_table;
    P.row_seq = row_seq;
    P.positions = positions;
    P.selected = selected;
    P.header = reinterpret_cast<int32_t*>(base);
    P.done = reinterpret_cast<int32_t*>(base + L.off_done);
    P.part_o = reinterpret_cast<float*>(base + L.off_part);
    P.part_lse = P.part_o + 2 * (int64_t)L.grid * L.rows * g.D;
    P.out = (__nv_bfloat16*)out;
    P.lse = lse;
    P.unit_cost = L.unit_cost;
    P.once = g.max_q_len <= L.together;
    P.row_lead = reinterpret_cast<int32_t*>(base + L.off_lead);
    P.row_tiles = P.row_lead + g.total_q;
    P.unit_entries = reinterpret_cast<int32_t*>(base + L.off_entries);
    P.list = reinterpret_cast<int2*>(base + L.off_list);
    P.join_parts = P.join_team = 1;
    const int sms = sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    return status_of(
        launch_decode_selected(P, L.together, L.nt, L.grid, sms, (cudaStream_t)stream));
}

}  // extern "C"
