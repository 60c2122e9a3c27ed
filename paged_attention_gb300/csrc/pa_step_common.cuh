// pa_step_common.cuh -- launch parameters of the operators of pa_step.h.
#pragma once

#include "pa_cache_common.cuh"
#include "pa_step.h"

namespace pa {

struct RopeParams {
    CacheGeom g;
    int32_t rotary, interleaved;
    float scale;
    const uint64_t* steps;
    const __nv_bfloat16* q;              // null: keys and values only
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t* positions;
    const int32_t* slots;
    __nv_bfloat16* q_out;
    void* k_cache;
    uint8_t* k_scale;
    void* v_cache;
    uint8_t* v_scale;
    int32_t* err;
    int32_t tokens;                      // of a CTA
};

struct SelectParams {
    CacheGeom g;
    int32_t budget, num_first, num_recent;
    const __nv_bfloat16* q;
    const int8_t* bounds;
    const float* scale;
    const int32_t* table;
    const int32_t* row_seq;
    const int32_t* positions;
    int32_t* selected;
    int32_t* err;
    int32_t cluster;             // CTAs of a row and KV head
};

struct SelectedParams {
    CacheGeom g;
    int32_t budget;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const int32_t* table;
    const int32_t* row_seq;
    const int32_t* positions;
    const int32_t* selected;
    int32_t* header;     // error word at H_ERROR
    int32_t* done;       // completion counters of the rows of the unit a CTA begins
    float* part_o;       // [2 * grid][rows][D]
    float* part_lse;     // [2 * grid][rows]
    __nv_bfloat16* out;
    float* lse;
    int32_t unit_cost;   // fixed cost of a unit, in tiles (line_fits)
    int32_t once;        // the rows of a sequence are one unit at most
    // rows of a sequence joined to units: per row, how many it leads (0: none) and its
    // units' tiles (by each of the CTAs that joined them); per row and KV head, the entries of
    // the joined list; and the lists
    int32_t* row_lead;
    int32_t* row_tiles;
    int32_t* unit_entries;
    int2* list;          // page number, index in the sequence and rows
    int32_t join_parts;  // CTAs of a row that join its heads' lists, at most kMostJoinParts
    int32_t join_team;   // warps of a head
};

constexpr int kMostJoinParts = 8;
constexpr int kSelDoneRows = 64;     // query rows of a unit of pa_decode_selected, at most

cudaError_t launch_pages_take(const CacheGeom& g, const int32_t* seq_lens, const int32_t* q_lens,
                              int32_t* table, const int32_t* free_pages, const int32_t* free_count,
                              int32_t* context_lens, int32_t* row_seq, int32_t* positions,
                              int32_t* slots, int32_t* free_left, int32_t* err, int sms,
                              cudaStream_t stream);
cudaError_t launch_pages_return(const CacheGeom& g, const int32_t* seq_lens,
                                const int32_t* keep_lens, const int32_t* table,
                                int32_t* free_pages, const int32_t* free_count, int32_t* free_left,
                                int32_t* err, int sms, cudaStream_t stream);
cudaError_t launch_rope(const RopeParams& P, bool mx4, int sms, cudaStream_t stream);
cudaError_t launch_page_bounds(const CacheGeom& g, const void* k, const int32_t* slots,
                               int8_t* bounds, float* scale, int32_t* err,
                               cudaStream_t stream);
cudaError_t launch_select(const SelectParams& P, int sms, cudaStream_t stream);
int selected_rows(int heads, int max_q_len);
int selected_row_tiles(int D, int rows);
int selected_ctas_per_sm();
cudaError_t launch_decode_selected(const SelectedParams& P, int rows, int nt, int grid, int sms,
                                   cudaStream_t stream);

}  // namespace pa
