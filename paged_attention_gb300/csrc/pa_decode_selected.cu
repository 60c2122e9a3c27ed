// pa_decode_selected.cu -- attention of single query rows over the cache pages
// listed for them (bf16 K/V).
//
//   S^T = K Q^T,  P = exp2(S^T - m),  O^T += V^T P,  per row and KV head
//
// Persistent CTAs, two per SM, take equal shares of the flat line of (row, KV
// head, 64-token tile of the listed pages); the warps of a CTA cut each unit's
// tokens between them in 16-token steps, every warp with its own running (max, sum,
// O), its own ring of cp.async stages that runs ahead over unit boundaries, and no
// barrier until the unit ends.  Then the warps' states merge through shared memory;
// a unit that spans CTAs leaves normalised parts in the workspace, and the last warp
// to leave a part of a query row joins that row's.
//
// What bounds it: 4 D bytes a listed key and head from HBM.  A page is 16 tokens or
// a multiple, so a step lies in one page, and one look at its list entry tells which
// of its keys are there: keys that no row sees, or whose page is none, are not loaded
// but written as zeros, and their scores are -inf.  Products are transposed (mma
// m16n8k16 with 16 keys, or 16 columns of V, as rows): R query rows cost ceil(R / 8)
// of them.
//
// Rows of one sequence that stand together (drafts, a chunk's tokens) list mostly the
// same pages.  Where the problem allows several rows a sequence, up to kMostRows of
// them are one unit: a first kernel joins their lists into one of pages, each with
// the set of rows that listed it, and looks the pages up; the second reads every page
// once and hides its keys from the rows that did not list it.  What is hidden from a
// row must not reach it as 0 * NaN either: a step that not all rows see in full looks
// whether V is finite, and multiplies row by row where it is not.
//
// Measured (head_dim 128, 8 KV heads): 64 rows of up to 32 pages of 64, 32 q heads, 60 us
// for 54.5 of HBM time; 128 sequences of 3 rows, 64 q heads, 40 pages, 205 to 210 us for 194
// (each row by itself: 540), and where half of every row's list is its own 335 us for the 301
// that the pages together take.  With 32 query rows a unit the products and the softmax set
// the pace: 64 sequences of 4 rows, 64 q heads, 90 us for 56.
#include <algorithm>
#include <type_traits>

#include "pa_cache_mma.cuh"
#include "pa_step_common.cuh"

namespace pa {

template <int D, int NT>
struct SelCfg {
    static constexpr int kCtas = 2;                        // of an SM
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kStep = 16;                       // tokens of a warp's step
    static constexpr int kRow = 2 * D;                     // bytes of a K or V row
    static constexpr int kStage = 2 * kStep * kRow;
    static constexpr int kRows = 8 * NT;                   // q heads a unit has room for
    static constexpr int kQRow = 2 * D + 16;               // (ldmatrix: rows on other banks)
    // eight rows: every warp has their queries in registers, and merges of four alternate
    // between two buffers, so that a unit costs one barrier or two.  More: merges of sixteen in
    // the ring's stage that is free just then
    static constexpr bool kQInRegs = NT == 1;
    static constexpr int kMergeRows = NT == 1 ? 4 : 16;    // rows merged at a time
    static constexpr int kBuffers = NT == 1 ? 2 : 1;
    static constexpr int kOffQ = kWarps * kStages * kStage;
    static constexpr int kOffMl = kOffQ + (kQInRegs ? 0 : kRows * kQRow);     // max and sum
    static constexpr int kOffFree = kOffMl + kBuffers * kWarps * kMergeRows * 8;   // free stages
    static constexpr int kOffMerge = kOffFree + 16;
    static constexpr int kMergeWarp = kMergeRows * D * 4;
    static constexpr int kSmem = kOffMerge + (NT == 1 ? kBuffers * kWarps * kMergeWarp : 0);
    static_assert(NT == 1 || kMergeWarp <= kStage, "a warp's rows in a stage");
    static_assert((kSmem + 1024) * kCtas <= 233472, "shared memory");
    static_assert(kOffQ % 16 == 0 && kOffMerge % 16 == 0, "alignment");
};

namespace {

// No CTA takes less than this of the flat line: joining a unit's parts costs more
// than the tiles it would spread (one sequence of 131071 tokens, 256 pages of 16, 8
// heads: 13.1 us with 2, 12.7 with 3, 12.2 with 4, 12.1 with 6; four rows of it 28.9 with 4,
// 30.2 with 12).
constexpr int kMinShareSel = 4;

constexpr int kDoneRows = kSelDoneRows;       // counters of a CTA: one a query row
constexpr int kMostRows = 6;                  // of a unit: what an entry has bits for
constexpr int kRowBits = 26;                  // a page index is below 2^26 (a context below 2^30)

constexpr float kUnseen = -3.402823466e38f;   // running max of a row that has seen no key
constexpr float kRise = 8.f;                  // (log2) how far a score may pass it before it moves

// A unit (row or rows of a sequence, KV head) as a CTA meets it.
struct SelUnit {
    int row, hk;
    int seq, pos;          // of the (first) row
    int rows;              // how many
    int n;                 // tiles
    int entries;           // of its list
    int64_t list;          // where that begins
    int64_t start;         // position of its fixed cost on the flat line
};

template <int N>
using Const = std::integral_constant<int, N>;

// x / y, in 32 bits where they fit (64 bits take ten times as long)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    return (((uint64_t)x | (uint64_t)y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

__device__ __forceinline__ bool good_row(const CacheGeom& g, int seq, int pos) {
    return seq >= 0 && seq < g.B && pos >= 0 && pos < g.max_ctx;
}
// Entries of the list of a row at pos.
__device__ __forceinline__ int list_entries(const SelectedParams& P, int pos) {
    const CacheGeom& g = P.g;
    const int first = g.window > 0 ? max(0, pos - g.window + 1) >> g.ps_shift : 0;
    return min(P.budget, (pos >> g.ps_shift) + 1 - first);
}
__device__ __forceinline__ int tiles_of(const CacheGeom& g, int entries) {
    return (int)((((int64_t)entries << g.ps_shift) + kDecodeTile - 1) / kDecodeTile);
}

// What the rows' units are: from the row maps, or as the first kernel left them.
template <bool JOINED>
__device__ __forceinline__ int64_t row_cost(const SelectedParams& P, int t) {
    if constexpr (JOINED) {
        int64_t n = 0;
        for (int c = 0; c < P.join_parts; ++c) n += P.row_tiles[t * P.join_parts + c];
        return n > 0 ? n + (int64_t)P.g.Hkv * P.unit_cost : 0;
    } else {
        const int seq = P.row_seq[t], pos = P.positions[t];
        if (!good_row(P.g, seq, pos)) return 0;
        return (int64_t)P.g.Hkv * (tiles_of(P.g, list_entries(P, pos)) + P.unit_cost);
    }
}
// The rest of u, whose row and head are set; its row leads a unit.
template <bool JOINED>
__device__ __forceinline__ void load_unit(const SelectedParams& P, SelUnit& u) {
    const CacheGeom& g = P.g;
    const int64_t at = (int64_t)u.row * g.Hkv;
    if constexpr (JOINED) {
        u.entries = P.unit_entries[at + u.hk];
        u.list = (at + (int64_t)u.hk * u.rows) * P.budget;
    } else {
        u.list = (at + u.hk) * P.budget;
    }
    u.n = tiles_of(g, u.entries);
}
template <bool JOINED>
__device__ __forceinline__ void load_row(const SelectedParams& P, SelUnit& u) {
    u.seq = P.row_seq[u.row];
    u.pos = P.positions[u.row];
    u.rows = JOINED ? P.row_lead[u.row] : 1;
    if constexpr (!JOINED) u.entries = list_entries(P, u.pos);
}

// The unit after u (every lane the same); false past the share's end.  (That is looked
// at first: rows of padding behind the last sequence's are not stepped through.  64 rows
// and 192 of padding 61 us, else 84; and 960 of padding 69, else 208.)
template <bool JOINED>
__device__ __forceinline__ bool next_unit(const SelectedParams& P, SelUnit& u, int64_t hi) {
    u.start += P.unit_cost + u.n;
    if (u.start >= hi) return false;
    if (++u.hk >= P.g.Hkv) {
        u.hk = 0;
        do {
            if (++u.row >= P.g.total_q) return false;
        } while (JOINED ? P.row_tiles[u.row * P.join_parts] == 0 : row_cost<JOINED>(P, u.row) == 0);
        load_row<JOINED>(P, u);
    }
    load_unit<JOINED>(P, u);
    return true;
}

// What warp w of W of the CTA with the share [lo, hi) of the flat line runs of unit u:
// tokens [a, z) of its list.  A tile belongs to the CTA whose share it is in, but no CTA
// takes less than two tiles of a unit, and a short unit is not split.
struct SelShare {
    int t0, t1;     // tiles of the unit in the CTA's share
    int a, z;
};
__device__ __forceinline__ SelShare share_of(const CacheGeom& g, const SelUnit& u, int cost,
                                             int64_t lo, int64_t hi, int w, int W) {
    SelShare s = {0, 0, 0, 0};
    const int64_t p0 = u.start + cost;
    const int64_t x = u.n < 4 ? p0 + u.n - 1 : p0 + 1;           // whose CTA has the first tile
    const int64_t y = u.n < 4 ? x : p0 + u.n - 2;                // and the last
    if (x >= hi || y < lo) return s;
    s.t0 = x >= lo ? 0 : (int)(lo - p0);
    s.t1 = y < hi ? u.n : (int)(hi - p0);
    const int tok0 = s.t0 * kDecodeTile, end = min(u.entries << g.ps_shift, s.t1 * kDecodeTile);
    const int steps = (end - tok0) / 16;
    s.a = tok0 + 16 * (steps * w / W);
    s.z = tok0 + 16 * (steps * (w + 1) / W);
    return s;
}

__device__ __forceinline__ void cp_async16_row(uint32_t dst, const void* src, int bytes,
                                               uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}

// ---- joins the lists of rows of one sequence (the CTAs (t, c) of row t; only a unit's first
// row's go on).  P.join_team warps a KV head, some pages at a time: the set of rows of every
// page, and a bit for the pages that have any, in shared memory; the bits before a page tell
// its place.  Where rows are few their heads are shared out among P.join_parts CTAs (one
// sequence of 131071 tokens, 4 rows, attention and all: a CTA with a warp a head 50 us, 29 so).
constexpr int kJoinWarps = 8;
constexpr int kJoinPages = 4096;             // a warp

__global__ void __launch_bounds__(32 * kJoinWarps)
join_lists_kernel(const __grid_constant__ SelectedParams P, int most) {
    __shared__ __align__(16) uint32_t s_rows[kJoinWarps * kJoinPages / 4];    // a byte a page
    __shared__ __align__(16) uint32_t s_any[kJoinWarps * kJoinPages / 32];    // a bit
    __shared__ __align__(16) int s_before[kJoinWarps * kJoinPages / 32];
    __shared__ int s_sum[kJoinWarps], s_tiles[kJoinWarps];
    const CacheGeom& g = P.g;
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    int32_t* err = P.header + H_ERROR;
    // (read together: what follows is a chain of loads)
    const int ahead = min(t + lane, g.total_q - 1);
    const int seq = P.row_seq[t], seq_ahead = P.row_seq[ahead], pos_ahead = P.positions[ahead];
    int m = 0;                         // rows of the unit that t leads
    if (seq >= 0 && seq < g.B) {
        // rows of the sequence before t, 128 looked at together
        int before = 0;
        bool here = true;
        while (here) {
            uint32_t other[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = t - 1 - before - 32 * j - lane;
                other[j] = __ballot_sync(0xffffffffu, r < 0 || P.row_seq[max(r, 0)] != seq);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (here) {
                    before += other[j] != 0 ? __ffs(other[j]) - 1 : 32;
                    here = other[j] == 0;
                }
        }
        if (before % most == 0) {
            const uint32_t other =
                __ballot_sync(0xffffffffu, t + lane >= g.total_q || seq_ahead != seq);
            m = min(most, other != 0 ? __ffs(other) - 1 : 32);
        }
    }
    // lane i < m has row i's position and its list's length; a row with a position that
    // cannot be has none
    int pos = -1;
    if (lane < m && pos_ahead >= 0 && pos_ahead < g.max_ctx) pos = pos_ahead;
    const int mine = pos >= 0 ? list_entries(P, pos) : 0;
    const uint32_t good = __ballot_sync(0xffffffffu, pos >= 0);
    if (threadIdx.x == 0 && (seq >= g.B || __popc(good) != m))
        flag_error(err, PA_DEV_BAD_LENGTHS);
    const int parts = P.join_parts, c = blockIdx.y;
    if (good == 0) {
        if (threadIdx.x == 0) {
            P.row_lead[t] = 0;
            P.row_tiles[t * parts + c] = 0;
        }
        return;                        // (the same for every thread)
    }
    const int last = __reduce_max_sync(0xffffffffu, pos) >> g.ps_shift;   // page index
    const int each = __reduce_max_sync(0xffffffffu, mine);                // the longest list
    // the CTA has the heads c, c + parts, ..., its teams one each at a time
    const int S = P.join_team, teams = kJoinWarps / S, team = warp / S;
    const int me = threadIdx.x - 32 * S * team, size = 32 * S;            // of the team
    uint32_t* rows_of = s_rows + team * S * (kJoinPages / 4);
    uint32_t* any = s_any + team * S * (kJoinPages / 32);
    int* before_word = s_before + team * S * (kJoinPages / 32);
    const int64_t chunk = (int64_t)S * kJoinPages;
    auto team_sync = [&]() {           // (all teams take the same steps)
        if (S > 1)
            __syncthreads();
        else
            __syncwarp();
    };
    int tiles = 0;
    for (int h0 = c; h0 < g.Hkv; h0 += parts * teams) {
        const int hk = h0 + parts * team;
        const bool there = hk < g.Hkv;
        int2* to = P.list + ((int64_t)t * g.Hkv + (int64_t)hk * m) * P.budget;
        // The rows' lists end to end, kAhead entries a lane under way: f(entries, their rows),
        // -1 for none.
        const int32_t* sel = P.selected + ((int64_t)t * g.Hkv + hk) * P.budget;
        const int64_t next_row = (int64_t)g.Hkv * P.budget;
        const int all = there ? m * each : 0;
        auto entries = [&](auto f) {
            constexpr int kAhead = 4;
            for (int k0 = 0; k0 < all; k0 += size * kAhead) {
                int e[kAhead], of[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int k = k0 + j * size + me;
                    int r = 0;
#pragma unroll
                    for (int x = 1; x < kMostRows; ++x) r += x < m && k >= x * each;
                    const int i = k - r * each;
                    const int many = __shfl_sync(0xffffffffu, mine, r);
                    of[j] = r;
                    e[j] = i < many ? sel[r * next_row + i] : -1;
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int top = __shfl_sync(0xffffffffu, pos, of[j]) >> g.ps_shift;
                    if (e[j] < -1 || e[j] > top) {
                        flag_error(err, PA_DEV_BAD_LENGTHS);
                        e[j] = -1;
                    }
                }
                f(e, of);
            }
        };
        int n = 0;
        for (int64_t p0 = 0; p0 <= last; p0 += chunk) {
            const int first = (int)p0, span = (int)min(chunk, last + 1 - p0);
            for (int i = me; i < (span + 15) / 16; i += size)
                reinterpret_cast<uint4*>(rows_of)[i] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4*>(any)[me] = make_uint4(0u, 0u, 0u, 0u);
            team_sync();
            entries([&](const auto& e, const auto& of) {
#pragma unroll
                for (int j = 0; j < (int)(sizeof(e) / sizeof(int)); ++j) {
                    const int at = e[j] - first;
                    if (e[j] < first || at >= span) continue;
                    atomicOr(&rows_of[at >> 2], 1u << (8 * (at & 3) + of[j]));
                    atomicOr(&any[at >> 5], 1u << (at & 31));
                }
            });
            team_sync();
            // how many pages there are before each word of `any`
            static_assert(kJoinPages / 32 == 4 * 32, "four words a lane");
            const uint4 w = reinterpret_cast<const uint4*>(any)[me];
            const int c0 = __popc(w.x), c1 = c0 + __popc(w.y), c2 = c1 + __popc(w.z);
            const int here = c2 + __popc(w.w), upto = warp_inclusive(here, lane);
            if (lane == 31) s_sum[warp] = upto;
            team_sync();
            int from = n + upto - here;
            for (int x = team * S; x < (team + 1) * S; ++x) {
                const int y = s_sum[x];
                if (x < warp) from += y;
                n += y;
            }
            reinterpret_cast<int4*>(before_word)[me] = make_int4(from, from + c0, from + c1,
                                                                 from + c2);
            team_sync();
            // the first row that listed a page writes it
            entries([&](const auto& e, const auto& of) {
                constexpr int K = (int)(sizeof(e) / sizeof(int));
                uint32_t rows[K];
                int page[K];
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const int at = e[j] - first;
                    rows[j] = 0u;
                    if (e[j] >= first && at < span) {
                        const uint32_t x = rows_of[at >> 2] >> (8 * (at & 3)) & 255u;
                        if ((x & (0u - x)) == 1u << of[j]) rows[j] = x;
                    }
                    page[j] = rows[j] != 0 ? P.table[(int64_t)seq * g.mpps + e[j]] : 0;
                }
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    if (rows[j] == 0) continue;
                    const int at = e[j] - first;
                    const int k =
                        before_word[at >> 5] + __popc(any[at >> 5] & ((1u << (at & 31)) - 1u));
                    const bool ok = (uint32_t)page[j] < (uint32_t)g.num_pages;
                    if (!ok) flag_error(err, PA_DEV_BAD_PAGE);
                    to[k] = make_int2(ok ? page[j] : -1,
                                      (int)((uint32_t)e[j] | rows[j] << kRowBits));
                }
            });
            team_sync();
        }
        if (there && me == 0) {
            if (n == 0) {              // the rows' results are written all the same
                to[0] = make_int2(-1, 0);
                n = 1;
            }
            P.unit_entries[(int64_t)t * g.Hkv + hk] = n;
            tiles += tiles_of(g, n);
        }
    }
    if (me == 0) s_tiles[team] = tiles;
    __syncthreads();
    if (threadIdx.x == 0) {
        int sum = 0;
        for (int x = 0; x < teams; ++x) sum += s_tiles[x];
        P.row_lead[t] = m;
        P.row_tiles[t * parts + c] = sum;
    }
}

// Byte offset of 16-byte piece c of row r of a step's K or V rows: ldmatrix takes
// eight rows' piece c, on eight bank groups.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    return (uint32_t)(r * 2 * D + ((c ^ (r & 7)) << 4));
}

// JOINED: units of several rows, whose lists are joined; else of one.
template <int D, int NT, bool JOINED>
__global__ void __launch_bounds__(SelCfg<D, NT>::kThreads, SelCfg<D, NT>::kCtas)
decode_selected_kernel(const __grid_constant__ SelectedParams P) {
    using Cfg = SelCfg<D, NT>;
    constexpr int W = Cfg::kWarps, ST = Cfg::kStages, ROW = Cfg::kRow;
    constexpr int KK = D / 16;      // contraction steps of the scores
    constexpr int OT = D / 16;      // 16-column tiles of O
    constexpr int MR = Cfg::kMergeRows;
    extern __shared__ __align__(128) uint8_t smem[];
    const CacheGeom& g = P.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gr = lane >> 2, t4 = lane & 3;   // operand row, column pair
    const int cost = P.unit_cost;
    grid_dependency_wait();

    // ---- this CTA's share of the flat line: a lane has a run of rows
    auto before = [&](int64_t v) -> int64_t {            // sum over the lanes up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    const int run = (g.total_q + 31) / 32, run0 = min(lane * run, g.total_q);
    int64_t mine = 0;
#pragma unroll 4
    for (int t = run0; t < min(run0 + run, g.total_q); ++t) mine += row_cost<JOINED>(P, t);
    if (!JOINED && blockIdx.x == 0 && warp == 0) {
        for (int t = lane; t < g.total_q; t += 32)
            if (P.row_seq[t] >= 0 && !good_row(g, P.row_seq[t], P.positions[t]))
                flag_error(P.header + H_ERROR, PA_DEV_BAD_LENGTHS);
    }
    const int64_t upto = before(mine);
    const int64_t C = __shfl_sync(0xffffffffu, upto, 31);
    const int64_t N = min((int64_t)gridDim.x, (C + kMinShareSel - 1) / kMinShareSel);
    const int cta = blockIdx.x;
    if (cta >= N) return;
    const int64_t lo = quotient(C * cta, N), hi = quotient(C * (cta + 1), N);
    SelUnit u;
    {
        const int src = __ffs(__ballot_sync(0xffffffffu, upto > lo)) - 1;
        u.start = __shfl_sync(0xffffffffu, upto - mine, src);
        // the row among that lane's, then the head among the row's.  (Neither is missed but where
        // another call writes to the workspace at the same time.)
        auto missed = [&](bool past) {
            if (past) flag_error(P.header + H_ERROR, PA_DEV_BAD_WORKSPACE);
            return past;
        };
        for (int t0 = src * run;; t0 += 32) {
            if (missed(t0 >= g.total_q)) return;
            const int64_t c = t0 + lane < g.total_q ? row_cost<JOINED>(P, t0 + lane) : 0;
            const int64_t to = u.start + before(c);
            const uint32_t past = __ballot_sync(0xffffffffu, to > lo);
            if (past != 0) {
                u.row = t0 + __ffs(past) - 1;
                u.start = __shfl_sync(0xffffffffu, to - c, __ffs(past) - 1);
                break;
            }
            u.start = __shfl_sync(0xffffffffu, to, 31);
        }
        load_row<JOINED>(P, u);
        if constexpr (JOINED) {
            for (int h0 = 0;; h0 += 32) {
                if (missed(h0 >= g.Hkv)) return;
                const int64_t c =
                    h0 + lane < g.Hkv
                        ? tiles_of(g, P.unit_entries[(int64_t)u.row * g.Hkv + h0 + lane]) + cost
                        : 0;
                const int64_t to = u.start + before(c);
                const uint32_t past = __ballot_sync(0xffffffffu, to > lo);
                if (past != 0) {
                    u.hk = h0 + __ffs(past) - 1;
                    u.start = __shfl_sync(0xffffffffu, to - c, __ffs(past) - 1);
                    break;
                }
                u.start = __shfl_sync(0xffffffffu, to, 31);
            }
        } else {
            const int c = tiles_of(g, u.entries) + cost;
            u.hk = (int)quotient(lo - u.start, c);
            u.start += (int64_t)u.hk * c;
        }
        load_unit<JOINED>(P, u);
    }
    auto share = [&](const SelUnit& x) { return share_of(g, x, cost, lo, hi, warp, W); };

    const uint32_t ring = smem_u32(smem) + warp * ST * Cfg::kStage;
    const uint32_t qbase = smem_u32(smem + Cfg::kOffQ);

    // ---- the load side runs ST - 1 steps ahead, over unit boundaries
    constexpr int CH = ROW / 16, RPI = 32 / CH;   // pieces of a row, rows an instruction
    constexpr int INS = 16 / RPI;                 // instructions for a step's K (or V)
    // Where no other unit reads the same pages they leave L2 first (64 rows of 32 pages of 64:
    // 59.7 us, without 62.1 and with a prefetch of 128 bytes 63.1; 384 rows of 40: 221, 241, 242).
    uint64_t policy;
    if (P.once)
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    else
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    const int page_rows = g.ps * g.Hkv;
    const int r_lane = lane / CH, c_lane = lane % CH;
    // A list's entry i + lane: as it lies there (read well ahead), and as a page number
    // (-1: nothing is there) with its index in the sequence (and its rows' bits).
    auto read_entry = [&](const SelUnit& x, int i) -> int2 {
        const bool there = i + lane < x.entries;
        if constexpr (JOINED)
            return there ? P.list[x.list + i + lane] : make_int2(-1, 0);
        else
            return make_int2(-1, there ? P.selected[x.list + i + lane] : -1);
    };
    auto look_up = [&](const SelUnit& x, int2 e) -> int2 {
        if constexpr (JOINED) return e;
        const int s = e.y;
        e.y = 0;
        if (s < 0 || s > x.pos >> g.ps_shift) {
            if (s != -1) flag_error(P.header + H_ERROR, PA_DEV_BAD_LENGTHS);
            return e;
        }
        const int page = P.table[(int64_t)x.seq * g.mpps + s];
        if ((uint32_t)page < (uint32_t)g.num_pages)
            e = make_int2(page, s);
        else
            flag_error(P.header + H_ERROR, PA_DEV_BAD_PAGE);
        return e;
    };
    // Positions of a unit's rows (lane i has row i's; -1: none), and their extremes.
    auto row_pos = [&](const SelUnit& x) -> int {
        if constexpr (!JOINED) return x.pos;
        const int p = lane < x.rows ? P.positions[x.row + lane] : -1;
        return p < g.max_ctx ? max(p, -1) : -1;
    };
    auto extremes = [&](int p, int& least, int& most, uint32_t& rows) {
        least = most = p;
        rows = 1u;
        if constexpr (JOINED) {
            most = __reduce_max_sync(0xffffffffu, p);
            least = __reduce_min_sync(0xffffffffu, p >= 0 ? p : 0x7fffffff);
            rows = __ballot_sync(0xffffffffu, p >= 0);
        }
    };
    SelUnit ln = u;                          // the unit after the one being loaded
    SelUnit lu = u;                          // the one being loaded
    bool more = true;
    int l_tok, l_end, l_least, l_most;
    uint32_t l_rows;
    {
        const SelShare x = share(u);
        l_tok = x.a;
        l_end = x.z;
    }
    int win_lo = l_tok >> g.ps_shift;        // 32 entries, the 32 after them, the next unit's
    int2 win = read_entry(u, win_lo), nxt = read_entry(u, win_lo + 32), lnw = make_int2(-1, 0);
    bool ln_ok = next_unit<JOINED>(P, ln, hi);
    if (ln_ok) lnw = read_entry(ln, share(ln).a >> g.ps_shift);
    extremes(row_pos(u), l_least, l_most, l_rows);
    win = look_up(u, win);
    // per stage: its first key that is there, one past the last, the rows that listed its
    // page, whether all rows see all of it; where its first key is
    uint32_t meta = 0;
    int meta_at = 0;
    auto issue = [&](int stage) {
        while (more && l_tok >= l_end) {
            more = ln_ok;
            if (!more) break;
            lu = ln;
            const SelShare x = share(ln);
            l_tok = x.a;
            l_end = x.z;
            extremes(row_pos(ln), l_least, l_most, l_rows);
            win_lo = l_tok >> g.ps_shift;
            win = look_up(ln, lnw);
            nxt = read_entry(ln, win_lo + 32);
            ln_ok = next_unit<JOINED>(P, ln, hi);
            if (ln_ok) lnw = read_entry(ln, share(ln).a >> g.ps_shift);
        }
        if (more) {
            const int tok = l_tok;
            l_tok += 16;
            const int p0 = tok >> g.ps_shift;
            if (p0 - win_lo >= 32) {
                win_lo += 32;
                win = look_up(lu, nxt);
                nxt = read_entry(lu, win_lo + 32);
            }
            const int page = __shfl_sync(0xffffffffu, win.x, p0 - win_lo);
            const uint32_t entry = (uint32_t)__shfl_sync(0xffffffffu, win.y, p0 - win_lo);
            const int slot = tok & (g.ps - 1);
            const int at = (int)((entry & ((1u << kRowBits) - 1u)) << g.ps_shift) + slot;
            // keys a .. z - 1 of the step are there, and some row sees them
            int a = 0, z = 0;
            if (page >= 0) {
                a = g.window > 0 ? max(0, min(16, l_least - g.window + 1 - at)) : 0;
                z = max(a, min(16, l_most + 1 - at));
            }
            if (lane == stage) {
                meta = (uint32_t)(a | z << 5);
                if constexpr (JOINED) {
                    const uint32_t rows = entry >> kRowBits;
                    const bool all = rows == l_rows && a == 0 && z == 16 && at + 15 <= l_least &&
                                     (g.window == 0 || at > l_most - g.window);
                    meta |= rows << 10 | (all ? 1u << 16 : 0u);
                    meta_at = at;
                }
            }
            const int64_t row0 = (int64_t)max(page, 0) * page_rows + (int64_t)slot * g.tok_rows +
                                 (int64_t)lu.hk * g.head_rows;
            const uint32_t dst = ring + stage * Cfg::kStage;
            const int64_t off = (row0 + (int64_t)r_lane * g.tok_rows) * D + c_lane * 8;
            const __nv_bfloat16* k = P.k + off;
            const __nv_bfloat16* v = P.v + off;
            const int64_t step = (int64_t)RPI * g.tok_rows * D;
            if (a == 0 && z == 16) {
#pragma unroll
                for (int i = 0; i < INS; ++i) {
                    const uint32_t to = dst + piece_at<D>(i * RPI + r_lane, c_lane);
                    cp_async16_row(to, k + i * step, 16, policy);
                    cp_async16_row(to + 16 * ROW, v + i * step, 16, policy);
                }
            } else {
#pragma unroll
                for (int i = 0; i < INS; ++i) {
                    const int r = i * RPI + r_lane;
                    const uint32_t to = dst + piece_at<D>(r, c_lane);
                    const bool ok = r >= a && r < z;
                    cp_async16_row(to, ok ? k + i * step : P.k, ok ? 16 : 0, policy);
                    cp_async16_row(to + 16 * ROW, ok ? v + i * step : P.v, ok ? 16 : 0, policy);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < ST - 1; ++s) issue(s);
    int stage = 0;

    // ---- Q rows of a unit, read ahead of the unit that needs them (not where O needs the
    // registers): the B operands themselves, or a row of a warp's for shared memory
    constexpr bool kQInRegs = Cfg::kQInRegs;
    constexpr bool kQAhead = NT <= 2;
    constexpr int QPW = kQInRegs ? 1 : Cfg::kRows / W, QW = kQInRegs ? KK * 2 : D / 64;
    uint32_t qw[QPW][QW];
    auto q_row = [&](const SelUnit& x, int r) -> const uint32_t* {
        return reinterpret_cast<const uint32_t*>(
            P.q + (JOINED ? (int64_t)(x.row + r / g.G) * g.Hq + (int64_t)x.hk * g.G + r % g.G
                          : (int64_t)x.row * g.Hq + (int64_t)x.hk * g.G + r) * D);
    };
    auto load_q = [&](const SelUnit& x) {
#pragma unroll
        for (int i = 0; i < QPW; ++i) {
            const int r = kQInRegs ? gr : warp + i * W;
#pragma unroll
            for (int j = 0; j < QW; ++j) qw[i][j] = 0u;
            if (r < x.rows * g.G) {
                const uint32_t* src = q_row(x, r);
#pragma unroll
                for (int j = 0; j < QW; ++j) qw[i][j] = src[kQInRegs ? 4 * j + t4 : lane + 32 * j];
            }
        }
    };
    if constexpr (kQAhead) load_q(u);
    int buffer = 0;

    // (never 0, so that a masked score times it stays -inf)
    const float f = fmaxf(g.sm_scale * kLog2e, 1.2e-38f);
    // ---- units
    while (true) {
        const SelShare sh = share(u);
        const int R = u.rows * g.G;
        if constexpr (!kQAhead) load_q(u);
        uint32_t qf[kQInRegs ? QW : 1];
        if constexpr (kQInRegs) {
#pragma unroll
            for (int j = 0; j < QW; ++j) qf[j] = qw[0][j];
        } else {
#pragma unroll
            for (int i = 0; i < QPW; ++i)
#pragma unroll
                for (int j = 0; j < QW; ++j)
                    *reinterpret_cast<uint32_t*>(smem + Cfg::kOffQ + (warp + i * W) * Cfg::kQRow +
                                                 4 * (lane + 32 * j)) = qw[i][j];
            __syncthreads();
        }
        SelUnit nu = u;
        const bool has_next = next_unit<JOINED>(P, nu, hi);
        if (kQAhead && has_next) load_q(nu);

        float m[NT][2], l[NT][2];
        float o[OT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = kUnseen;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < OT; ++i)
                o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
        }
        // JOINED: lane i has row i's position; query row r is of row r / G = r * inv >> 16
        const int upos = JOINED ? row_pos(u) : 0;
        const int inv = JOINED ? 65535 / g.G + 1 : 0;
        // the B operands of two contraction steps: rows 8 nt + (lane & 7), piece 2 kk + lane / 8
        auto q_frag = [&](int nt, int kk, uint32_t* x) {
            ldsm_x4(qbase + (8 * nt + (lane & 7)) * Cfg::kQRow + (2 * kk + (lane >> 3)) * 16, x[0],
                    x[1], x[2], x[3]);
        };

#pragma unroll 1
        for (int tok = sh.a; tok < sh.z;) {
            cp_async_wait<ST - 2>();
            __syncwarp();
            const uint32_t mt = __shfl_sync(0xffffffffu, meta, stage);
            const int at = JOINED ? __shfl_sync(0xffffffffu, meta_at, stage) : 0;
            issue(stage == 0 ? ST - 1 : stage - 1);   // into the stage the last step left
            const uint32_t sk = ring + stage * Cfg::kStage, sv = sk + 16 * ROW;
            stage = stage + 1 == ST ? 0 : stage + 1;
            tok += 16;
            // (taken out of mt again where they are needed: kept, they and tok cost the widest
            // forms registers that they then spill; 128 sequences of 3 rows, 64 q heads 208 us,
            // so 204)
            auto first_key = [&]() { return (int)(mt & 31u); };
            auto end_key = [&]() { return (int)((mt >> 5) & 31u); };
            if (first_key() == end_key()) continue;   // no key of the step is there

            // ---- scores of 16 keys
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
            {
                // (few rows: even and odd contraction steps in two chains)
                constexpr bool kTwo = NT <= 2;
                float s1[kTwo ? NT : 1][4];
#pragma unroll
                for (int nt = 0; nt < (kTwo ? NT : 1); ++nt)
                    s1[nt][0] = s1[nt][1] = s1[nt][2] = s1[nt][3] = 0.f;
                const int r = lane & 15, c = lane >> 4;
#pragma unroll
                for (int kk = 0; kk < KK; kk += 2) {
                    uint32_t x[4], y[4];
                    ldsm_x4(sk + piece_at<D>(r, 2 * kk + c), x[0], x[1], x[2], x[3]);
                    ldsm_x4(sk + piece_at<D>(r, 2 * kk + 2 + c), y[0], y[1], y[2], y[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (kQInRegs) {
                            mma_bf16_16816(s[nt], x, qf[2 * kk], qf[2 * kk + 1]);
                            mma_bf16_16816(s1[nt], y, qf[2 * kk + 2], qf[2 * kk + 3]);
                        } else {
                            uint32_t b[4];
                            q_frag(nt, kk, b);
                            mma_bf16_16816(s[nt], x, b[0], b[1]);
                            mma_bf16_16816(kTwo ? s1[kTwo ? nt : 0] : s[nt], y, b[2], b[3]);
                        }
                    }
                }
                if constexpr (kTwo) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[nt][e] += s1[nt][e];
                }
            }
            const bool part_seen = JOINED ? !(mt >> 16 & 1u) : first_key() > 0 || end_key() < 16;
            if (part_seen) {
                const int a = first_key(), z = end_key();
                if constexpr (JOINED) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r = 8 * nt + 2 * t4 + e, i = r * inv >> 16;
                            const int p = __shfl_sync(0xffffffffu, upos, i & 31);
                            const bool listed = r < R && (mt >> (10 + i) & 1u) != 0;
                            // of keys gr and gr + 8 of the step
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int x = gr + 8 * h;
                                if (!(listed && x >= a && x < z && at + x <= p &&
                                      (g.window == 0 || at + x > p - g.window)))
                                    s[nt][2 * h + e] = -INFINITY;
                            }
                        }
                } else {
                    const bool k0 = gr >= a && gr < z, k1 = gr + 8 >= a && gr + 8 < z;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(e < 2 ? k0 : k1)) s[nt][e] = -INFINITY;
                }
            }
            // ---- exponents below the running max, which moves where one passes it by far
            float x[NT][4];
            auto exponents = [&]() -> float {
                float most = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[nt][e] = fmaf(s[nt][e], f, -m[nt][e & 1]);
                    most = fmax3(most, fmaxf(x[nt][0], x[nt][1]), fmaxf(x[nt][2], x[nt][3]));
                }
                return most;
            };
            if (__any_sync(0xffffffffu, exponents() > kRise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y = fmaxf(s[nt][e], s[nt][e + 2]) * f;
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                        if (y > m[nt][e]) {
                            const float al = m[nt][e] == kUnseen ? 0.f : ex2(m[nt][e] - y);
                            m[nt][e] = y;
                            l[nt][e] *= al;
#pragma unroll
                            for (int i = 0; i < OT; ++i) {
                                o[i][nt][e] *= al;
                                o[i][nt][e + 2] *= al;
                            }
                        }
                    }
                exponents();
            }
            // ---- probabilities, and their transposes as the B operand: rounded to bf16 (2^-8 of
            // each at most), since a product's operands are of one type, V's.  Their sum keeps 32
            // bits, for lse.  The roundings of different keys are independent: results are off by
            // 0.0023 of their rms, where rounding them to bf16 alone gives 0.0017.  A second
            // product, of what the first rounding left, would double the work that sets the pace
            // from 24 rows on.
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = ex2(x[nt][0]), p1 = ex2(x[nt][1]);
                const float p2 = ex2(x[nt][2]), p3 = ex2(x[nt][3]);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                pb[nt][0] = movmatrix_trans(pack_bf16x2(p0, p1));
                pb[nt][1] = movmatrix_trans(pack_bf16x2(p2, p3));
            }
            // ---- O^T += V^T P
            const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
            bool plain = true;
            if constexpr (JOINED) {
                if (part_seen) {
                    // is V finite?  (the largest magnitude of the lane's share of it)
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < OT; ++i) {
                        uint32_t y[4];
                        ldsm_x4(sv + piece_at<D>(vr, 2 * i + vc), y[0], y[1], y[2], y[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) top = max_bf16x2(top, y[j] & 0x7fff7fffu);
                    }
                    const uint32_t m1 = max(top & 0xffffu, top >> 16);
                    plain = !__any_sync(0xffffffffu, m1 >= 0x7f80u);
                }
            }
            if (plain) {
#pragma unroll
                for (int i = 0; i < OT; ++i) {
                    uint32_t x[4];
                    ldsm_x4_t(sv + piece_at<D>(vr, 2 * i + vc), x[0], x[1], x[2], x[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(o[i][nt], x, pb[nt][0], pb[nt][1]);
                }
            } else if constexpr (JOINED) {
                // row by row of the sequence: the keys it does not see are zeros in V, and
                // the product is added to its own columns only
                const int a = first_key(), z = end_key();
                for (int i0 = 0; i0 < u.rows; ++i0) {
                    const int p = __shfl_sync(0xffffffffu, upos, i0);
                    auto word = [&](int key) -> uint32_t {
                        auto seen = [&](int x) {
                            return (mt >> (10 + i0) & 1u) != 0 && x >= a && x < z && at + x <= p &&
                                   (g.window == 0 || at + x > p - g.window);
                        };
                        return (seen(key) ? 0xffffu : 0u) | (seen(key + 1) ? 0xffff0000u : 0u);
                    };
                    const uint32_t w0 = word(2 * t4), w1 = word(2 * t4 + 8);
#pragma unroll
                    for (int i = 0; i < OT; ++i) {
                        uint32_t x[4];
                        ldsm_x4_t(sv + piece_at<D>(vr, 2 * i + vc), x[0], x[1], x[2], x[3]);
                        x[0] &= w0;
                        x[1] &= w0;
                        x[2] &= w1;
                        x[3] &= w1;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float y[4];
                            mma_bf16_first(y, x, pb[nt][0], pb[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int r = 8 * nt + 2 * t4 + (e & 1);
                                if (r < R && r * inv >> 16 == i0) o[i][nt][e] += y[e];
                            }
                        }
                    }
                }
            }
        }

        // ---- merge the warps, a few rows at a time
        if (sh.t1 > sh.t0) {
            // the CTAs that hold parts of the unit
            auto owner = [&](int64_t x) { return (int)quotient((x + 1) * N - 1, C); };
            const int c_first = sh.t0 == 0 ? cta : owner(u.start + cost + 1);
            const int c_last = sh.t1 == u.n ? cta : owner(u.start + cost + u.n - 2);
            // where row r of the unit is among the outputs; -1: nowhere
            auto out_row = [&](int r) -> int64_t {
                if constexpr (JOINED) {
                    const int t = u.row + r / g.G, p = P.positions[t];
                    if (p < 0 || p >= g.max_ctx) return -1;
                    return (int64_t)t * g.Hq + (int64_t)u.hk * g.G + r % g.G;
                }
                return (int64_t)u.row * g.Hq + (int64_t)u.hk * g.G + r;
            };
            const int part = c_first == c_last ? -1 : 2 * cta + (cta == c_first ? 1 : 0);
            // (the stage that the next load goes to: what was in it has been used)
            int* s_free = reinterpret_cast<int*>(smem + Cfg::kOffFree);
            if (NT > 1 && lane == 0) s_free[warp] = stage == 0 ? ST - 1 : stage - 1;
#pragma unroll
            for (int r0 = 0; r0 < Cfg::kRows; r0 += MR) {
                if (r0 >= R) break;
                // row r is at r * D of a warp's area, its columns in eights turned by r / 2
                auto area = [&](int w) {
                    return reinterpret_cast<float*>(
                        NT == 1 ? smem + Cfg::kOffMerge + (buffer * W + w) * Cfg::kMergeWarp
                                : smem + (w * ST + s_free[w]) * Cfg::kStage);
                };
                float2* ml = reinterpret_cast<float2*>(smem + Cfg::kOffMl) + buffer * W * MR;
                float* mw = NT == 1 ? area(warp)
                                    : reinterpret_cast<float*>(
                                          smem + (warp * ST + (stage == 0 ? ST - 1 : stage - 1)) *
                                                     Cfg::kStage);
#pragma unroll
                for (int nt = r0 / 8; nt < NT && nt * 8 < r0 + MR; ++nt) {
                    if (8 * nt >= R) break;
                    // (of eight rows the four of r0 are with half of the lanes)
                    const bool mine = MR >= 8 || t4 / 2 == (r0 % 8) / 4;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = l[nt][e];
                        x += __shfl_xor_sync(0xffffffffu, x, 4);
                        x += __shfl_xor_sync(0xffffffffu, x, 8);
                        x += __shfl_xor_sync(0xffffffffu, x, 16);
                        const int r = (8 * nt + 2 * t4 + e) % MR;
                        if (mine) {
                            if (gr == 0) ml[warp * MR + r] = make_float2(m[nt][e], x);
                            float* to = mw + r * D + gr;
#pragma unroll
                            for (int i = 0; i < OT; ++i) {
                                to[(16 * i) ^ (8 * t4)] = o[i][nt][e];
                                to[(16 * i + 8) ^ (8 * t4)] = o[i][nt][e + 2];
                            }
                        }
                    }
                }
                __syncthreads();
                // a row a warp
#pragma unroll
                for (int rr = warp; rr < MR; rr += W) {
                    const int r = r0 + rr;
                    if (r >= R) break;
                    constexpr int DPL = D / 32;
                    float M = kUnseen;
#pragma unroll
                    for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w * MR + rr].x);
                    float den = 0.f, acc[DPL];
#pragma unroll
                    for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float2 z = ml[w * MR + rr];
                        const float* b = area(w) + rr * D + (lane * DPL ^ (8 * (r / 2 & 3)));
                        if (z.x == kUnseen && z.y == 0.f) continue;   // saw nothing
                        const float x = z.x == kUnseen ? 1.f : ex2(z.x - M);
                        den += x * z.y;
#pragma unroll
                        for (int e = 0; e < DPL; ++e) acc[e] += x * b[e];
                    }
                    // (a NaN sum is not "no visible key")
                    const bool none = den == 0.f;
                    const float inv = none ? 0.f : 1.f / den;
                    const float ln2 = none ? -INFINITY : (M == kUnseen ? den : (lg2(den) + M) * kLn2);
                    if (part < 0) {
                        const int64_t row = out_row(r);
                        if (row >= 0) {
                            __nv_bfloat16* dst = P.out + row * D + lane * DPL;
#pragma unroll
                            for (int e = 0; e < DPL; e += 2)
                                *reinterpret_cast<uint32_t*>(dst + e) =
                                    pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
                        }
                        if (P.lse != nullptr && lane == 0 && row >= 0) P.lse[row] = ln2;
                    } else {
                        const int64_t row = (int64_t)part * Cfg::kRows + r;
                        float* dst = P.part_o + row * D + lane * DPL;
#pragma unroll
                        for (int e = 0; e < DPL; e += 2)
                            *reinterpret_cast<float2*>(dst + e) =
                                make_float2(acc[e] * inv, acc[e + 1] * inv);
                        if (lane == 0) P.part_lse[row] = ln2;
                    }
                }
                // (two buffers: the next barrier comes before this one is written again)
                if constexpr (Cfg::kBuffers > 1)
                    buffer ^= 1;
                else
                    __syncthreads();
            }
            if (part >= 0) {
                // every row for itself: the last warp to leave a part of it joins them (nobody
                // waits for another); lane i counts the warp's i-th row
                const uint32_t others = (uint32_t)(c_last - c_first);
                bool last = false;
                __syncwarp();
                __threadfence();                 // the warp's parts are written
                if (warp + W * lane < R) {
                    int32_t* count = P.done + c_first * kDoneRows + warp + W * lane;
                    const uint32_t earlier = (uint32_t)atomicAdd(count, 1);
                    last = earlier == others;
                    if (last) *count = 0;        // as the next call finds it
                    // (nobody will come last: the workspace did not start as zeros)
                    if (earlier > others) flag_error(P.header + H_ERROR, PA_DEV_BAD_WORKSPACE);
                }
                __threadfence();
                uint32_t ends = __ballot_sync(0xffffffffu, last);
                __syncwarp();                    // (a vote orders no memory)
                // part c of the unit is in slot 2 c (the first in 2 c + 1)
                auto part_row = [&](int c, int r) {
                    return (int64_t)(2 * c + (c == c_first ? 1 : 0)) * Cfg::kRows + r;
                };
                // K of those rows, whose first B parts are under way together, and their lse
                // (one a lane); the weights of 32 parts at a time
                auto join_rows = [&](auto rows, auto batch) {
                    constexpr int K = decltype(rows)::value, B = decltype(batch)::value;
                    constexpr int DPL = D / 32;
                    int row_in[K];
                    bool there[K];
                    float x[K][B][DPL], lse[K];
                    auto load_parts = [&](int i, int c0) {
#pragma unroll
                        for (int j = 0; j < B; ++j) {
                            const float* src =
                                P.part_o + part_row(min(c0 + j, c_last), row_in[i]) * D + lane * DPL;
#pragma unroll
                            for (int e = 0; e < DPL; e += 2)
                                *reinterpret_cast<float2*>(x[i][j] + e) =
                                    __ldcg(reinterpret_cast<const float2*>(src + e));
                        }
                    };
                    auto load_lse = [&](int i, int c) {
                        return c <= c_last ? __ldcg(P.part_lse + part_row(c, row_in[i])) : -INFINITY;
                    };
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        there[i] = ends != 0;
                        row_in[i] = there[i] ? warp + W * (__ffs(ends) - 1) : row_in[0];
                        ends &= ends - 1;
                        lse[i] = load_lse(i, c_first + lane);
                        load_parts(i, c_first);
                    }
                    float M[K], den[K], acc[K][DPL];
                    bool poison[K];
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        M[i] = lse[i];
                        poison[i] = M[i] != M[i];
                        for (int c = c_first + lane + 32; c <= c_last; c += 32) {
                            const float y = load_lse(i, c);
                            poison[i] |= y != y;
                            M[i] = fmaxf(M[i], y);
                        }
#pragma unroll
                        for (int y = 16; y > 0; y >>= 1)
                            M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], y));
                        poison[i] = __any_sync(0xffffffffu, poison[i]);
                        den[i] = 0.f;
#pragma unroll
                        for (int e = 0; e < DPL; ++e) acc[i][e] = 0.f;
                    }
#pragma unroll 1
                    for (int cb = c_first; cb <= c_last; cb += 32) {
                        float y[K];
#pragma unroll
                        for (int i = 0; i < K; ++i) {
                            const float v = cb == c_first ? lse[i] : load_lse(i, cb + lane);
                            y[i] = cb + lane > c_last ? 0.f
                                   : poison[i]        ? NAN
                                   : v == -INFINITY   ? 0.f
                                                      : ex2((v - M[i]) * kLog2e);
                        }
#pragma unroll 1
                        for (int c0 = cb; c0 <= min(c_last, cb + 31); c0 += B) {
                            if (c0 > c_first)
#pragma unroll
                                for (int i = 0; i < K; ++i) load_parts(i, c0);
#pragma unroll
                            for (int i = 0; i < K; ++i)
#pragma unroll
                                for (int j = 0; j < B; ++j) {
                                    const float w = __shfl_sync(0xffffffffu, y[i], c0 - cb + j);
                                    den[i] += w;
#pragma unroll
                                    for (int e = 0; e < DPL; ++e)
                                        if (w != 0.f) acc[i][e] = fmaf(w, x[i][j][e], acc[i][e]);
                                }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        if (!there[i]) continue;
                        const bool none = den[i] == 0.f;
                        const float inv = none ? 0.f : 1.f / den[i];
                        const int64_t row = out_row(row_in[i]);
                        if (row >= 0) {
                            __nv_bfloat16* dst = P.out + row * D + lane * DPL;
#pragma unroll
                            for (int e = 0; e < DPL; e += 2)
                                *reinterpret_cast<uint32_t*>(dst + e) =
                                    pack_bf16x2(acc[i][e] * inv, acc[i][e + 1] * inv);
                        }
                        if (P.lse != nullptr && lane == 0 && row >= 0)
                            P.lse[row] = none ? -INFINITY : M[i] + lg2(den[i]) * kLn2;
                    }
                };
                while (ends != 0) {
                    if (NT > 1 && others < 4)
                        join_rows(Const<4>{}, Const<4>{});
                    else if (NT > 2)           // (O had the registers; with 16 rows it spills)
                        join_rows(Const<4>{}, Const<8>{});
                    else if (others < 8)
                        join_rows(Const<2>{}, Const<8>{});
                    else
                        join_rows(Const<1>{}, Const<16>{});
                }
            }
        }
        if (!has_next) break;
        if (!kQInRegs && sh.t1 <= sh.t0) __syncthreads();   // all have read this unit's Q rows
        u = nu;
    }
    cp_async_wait<0>();
}

template <int D, int NT, bool JOINED>
cudaError_t launch_variant(const SelectedParams& P, int grid, cudaStream_t stream) {
    using Cfg = SelCfg<D, NT>;
    const cudaError_t e = allow_smem<decode_selected_kernel<D, NT, JOINED>>(Cfg::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(decode_selected_kernel<D, NT, JOINED>, dim3(grid), dim3(Cfg::kThreads),
                            Cfg::kSmem, stream, P);
}
template <int D, int NT>
cudaError_t launch(const SelectedParams& P, bool joined, int grid, cudaStream_t stream) {
    return joined ? launch_variant<D, NT, true>(P, grid, stream)
                  : launch_variant<D, NT, false>(P, grid, stream);
}

}  // namespace

// Rows of a sequence that a unit takes, for groups of `heads` and at most max_q_len rows a
// sequence.
int selected_rows(int heads, int max_q_len) {
    return std::max(1, std::min({kMostRows, max_q_len, 32 / heads}));
}
// Row tiles (of 8) that are built: what holds `rows` query rows, -1 if none.
int selected_row_tiles(int D, int rows) {
    if (rows > (D == 128 ? 32 : 64)) return -1;
    return rows <= 32 ? (rows + 7) / 8 : 8;
}
int selected_ctas_per_sm() { return SelCfg<128, 1>::kCtas; }

cudaError_t launch_decode_selected(const SelectedParams& P0, int rows, int nt, int grid, int sms,
                                   cudaStream_t stream) {
    SelectedParams P = P0;
    if (rows > 1) {
        // a row's heads among CTAs until there is one an SM, and a CTA's warps among its heads
        int parts = 1, teams = 1;
        while (parts < kMostJoinParts && 2 * parts <= P.g.Hkv &&
               (int64_t)P.g.total_q * 2 * parts <= sms)
            parts *= 2;
        while (teams < kJoinWarps && teams * parts < P.g.Hkv) teams *= 2;
        P.join_parts = parts;
        P.join_team = kJoinWarps / teams;
        const cudaError_t e = launch_dependent(join_lists_kernel, dim3(P.g.total_q, parts),
                                               dim3(32 * kJoinWarps), 0, stream, P, rows);
        if (e != cudaSuccess) return e;
    }
    const bool joined = rows > 1;
    if (P.g.D == 128) {
        switch (nt) {
            case 1: return launch<128, 1>(P, joined, grid, stream);
            case 2: return launch<128, 2>(P, joined, grid, stream);
            case 3: return launch<128, 3>(P, joined, grid, stream);
            case 4: return launch<128, 4>(P, joined, grid, stream);
        }
    } else {
        switch (nt) {
            case 1: return launch<64, 1>(P, joined, grid, stream);
            case 2: return launch<64, 2>(P, joined, grid, stream);
            case 3: return launch<64, 3>(P, joined, grid, stream);
            case 4: return launch<64, 4>(P, joined, grid, stream);
            case 8: return launch_variant<64, 8, false>(P, grid, stream);   // (joined: 32 rows at most)
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
