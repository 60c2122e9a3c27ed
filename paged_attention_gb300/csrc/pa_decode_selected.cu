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
// a unit that spans CTAs leaves normalised parts in the workspace, and the last CTA
// to finish one joins them.
//
// What bounds it: 4 D bytes a listed key and head from HBM.  A page is 16 tokens or
// a multiple, so a step lies in one page, and one look at its list entry tells which
// of its keys are there: keys that the row does not see, or whose page is none, are
// not loaded but written as zeros, and their scores are -inf.  Nothing outside a
// row's sight reaches it.  Products are transposed (mma m16n8k16 with 16 keys, or 16
// columns of V, as rows): the G heads of a group cost ceil(G / 8) of them.
#include <algorithm>

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
    static constexpr int kMergeRows = 4;                   // rows merged at a time
    static constexpr int kMergeRow = D + 4;                // floats
    static constexpr int kMergeWarp = kMergeRows * kMergeRow + 2 * kMergeRows;
    static constexpr int kOffQ = kWarps * kStages * kStage;
    static constexpr int kOffMerge = kOffQ + kRows * kQRow;
    static constexpr int kOffFlag = kOffMerge + kWarps * kMergeWarp * 4;
    static constexpr int kSmem = kOffFlag + 16;
    static_assert((kSmem + 1024) * kCtas <= 233472, "shared memory");
    static_assert(kOffQ % 16 == 0 && kOffMerge % 16 == 0 && kOffFlag % 16 == 0, "alignment");
};

namespace {

// No CTA takes less than this of the flat line: joining a unit's parts costs more
// than the tiles it would spread.
constexpr int kMinShareSel = 2;

constexpr float kUnseen = -3.402823466e38f;   // running max of a row that has seen no key
constexpr float kRise = 8.f;                  // (log2) how far scores may pass the max before it moves

// A unit (row, KV head) as a CTA meets it.
struct SelUnit {
    int row, hk;
    int seq, pos;          // of the row
    int n;                 // tiles
    int tokens;            // of its list
    int64_t start;         // position of its fixed cost on the flat line
};

// Tokens of row t's list, 0 if it has none or is none of a sequence's.
__device__ __forceinline__ int list_tokens(const SelectedParams& P, int seq, int pos) {
    const CacheGeom& g = P.g;
    if (seq < 0 || seq >= g.B || pos < 0 || pos >= g.max_ctx) return 0;
    const int first = g.window > 0 ? max(0, pos - g.window + 1) >> g.ps_shift : 0;
    return min(P.budget, (pos >> g.ps_shift) + 1 - first) << g.ps_shift;
}
__device__ __forceinline__ int tiles_of(int tokens) {
    return (tokens + kDecodeTile - 1) / kDecodeTile;
}

__device__ __forceinline__ void load_row(const SelectedParams& P, SelUnit& u) {
    u.seq = P.row_seq[u.row];
    u.pos = P.positions[u.row];
    u.tokens = list_tokens(P, u.seq, u.pos);
    u.n = tiles_of(u.tokens);
}

// The unit after u (every lane the same); false past the last row.
__device__ __forceinline__ bool next_unit(const SelectedParams& P, SelUnit& u) {
    u.start += P.unit_cost + u.n;
    if (++u.hk < P.g.Hkv) return true;
    u.hk = 0;
    do {
        if (++u.row >= P.g.total_q) return false;
        load_row(P, u);
    } while (u.n == 0);
    return true;
}

// What warp w of W runs of unit u, of the CTA's share [lo, hi) of the flat line:
// tokens [a, z) of its list.
struct SelShare {
    int t0, t1;     // tiles of the unit in the CTA's share
    int a, z;
};
__device__ __forceinline__ SelShare share_of(const SelUnit& u, int cost, int64_t lo, int64_t hi,
                                             int w, int W) {
    SelShare s;
    const int64_t base = u.start + cost;
    s.t0 = (int)max((int64_t)0, min((int64_t)u.n, lo - base));
    s.t1 = (int)max((int64_t)0, min((int64_t)u.n, hi - base));
    const int tok0 = s.t0 * kDecodeTile, end = min(u.tokens, s.t1 * kDecodeTile);
    const int steps = s.t1 > s.t0 ? (end - tok0) / 16 : 0;
    s.a = tok0 + 16 * (steps * w / W);
    s.z = tok0 + 16 * (steps * (w + 1) / W);
    return s;
}

__device__ __forceinline__ void cp_async16_row(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(bytes)
                 : "memory");
}

// Byte offset of 16-byte piece c of row r of a step's K or V rows: ldmatrix takes
// eight rows' piece c, on eight bank groups.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    return (uint32_t)(r * 2 * D + ((c ^ (r & 7)) << 4));
}

template <int D, int NT>
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

    // ---- this CTA's share of the flat line
    auto row_cost = [&](int t) -> int64_t {
        const int n = tiles_of(list_tokens(P, P.row_seq[t], P.positions[t]));
        return n > 0 ? (int64_t)g.Hkv * (n + cost) : 0;
    };
    const int64_t C = flat_total(g.total_q, lane, row_cost);
    if (blockIdx.x == 0 && warp == 0) {
        bool bad = false;
        for (int t = lane; t < g.total_q; t += 32)
            bad |= P.row_seq[t] >= 0 && list_tokens(P, P.row_seq[t], P.positions[t]) == 0;
        if (bad) flag_error(P.header + H_ERROR, PA_DEV_BAD_LENGTHS);
    }
    const int64_t N = min((int64_t)gridDim.x, (C + kMinShareSel - 1) / kMinShareSel);
    const int cta = blockIdx.x;
    if (cta >= N) return;
    const int64_t lo = C * cta / N, hi = C * (cta + 1) / N;
    SelUnit u;
    {
        int64_t start;
        int none;
        u.row = flat_find(g.total_q, lane, lo, row_cost, [](int) { return 0; }, start, none);
        load_row(P, u);
        const int i = (int)((lo - start) / (u.n + cost));
        u.hk = i;
        u.start = start + (int64_t)i * (u.n + cost);
    }

    const uint32_t ring = smem_u32(smem) + warp * ST * Cfg::kStage;
    const uint32_t qbase = smem_u32(smem + Cfg::kOffQ);
    float* merge = reinterpret_cast<float*>(smem + Cfg::kOffMerge);
    volatile int* flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffFlag);

    // ---- the load side runs ST - 1 steps ahead, over unit boundaries
    constexpr int CH = ROW / 16, RPI = 32 / CH;   // pieces of a row, rows an instruction
    constexpr int INS = 16 / RPI;                 // instructions for a step's K (or V)
    const int page_rows = g.ps * g.Hkv;
    const int r_lane = lane / CH, c_lane = lane % CH;
    // list entry i + lane of a unit, as (page number, position of its first token); a page
    // number of -1: nothing is there
    auto entries = [&](const SelUnit& x, int i, int& base) -> int {
        base = 0;
        const int k = i + lane;
        if (k >= x.tokens >> g.ps_shift) return -1;
        const int s = P.selected[((int64_t)x.row * g.Hkv + x.hk) * P.budget + k];
        if (s < 0) {
            if (s < -1) flag_error(P.header + H_ERROR, PA_DEV_BAD_LENGTHS);
            return -1;
        }
        if (s > x.pos >> g.ps_shift) {
            flag_error(P.header + H_ERROR, PA_DEV_BAD_LENGTHS);
            return -1;
        }
        base = s << g.ps_shift;
        const int page = P.table[(int64_t)x.seq * g.mpps + s];
        if ((uint32_t)page < (uint32_t)g.num_pages) return page;
        flag_error(P.header + H_ERROR, PA_DEV_BAD_PAGE);
        return -1;
    };
    SelUnit ln = u;                          // the unit after the one being loaded
    SelUnit lu = u;                          // the one being loaded
    SelShare ls = share_of(u, cost, lo, hi, warp, W);
    bool more = true;
    int l_tok = ls.a, l_end = ls.z;
    int win_lo = l_tok >> g.ps_shift;        // 32 entries, and the next unit's
    int win_base, lnw_base = 0;
    int win = entries(u, win_lo, win_base), lnw = -1;
    uint32_t meta = 0;                       // per stage: the first key there is, and one past the last
    bool ln_ok = next_unit(P, ln) && ln.start < hi;
    if (ln_ok) lnw = entries(ln, share_of(ln, cost, lo, hi, warp, W).a >> g.ps_shift, lnw_base);
    auto issue = [&](int stage) {
        while (more && l_tok >= l_end) {
            more = ln_ok;
            if (!more) break;
            lu = ln;
            const SelShare x = share_of(ln, cost, lo, hi, warp, W);
            l_tok = x.a;
            l_end = x.z;
            win_lo = l_tok >> g.ps_shift;
            win = lnw;
            win_base = lnw_base;
            ln_ok = next_unit(P, ln) && ln.start < hi;
            if (ln_ok)
                lnw = entries(ln, share_of(ln, cost, lo, hi, warp, W).a >> g.ps_shift, lnw_base);
        }
        if (more) {
            const int tok = l_tok;
            l_tok += 16;
            const int p0 = tok >> g.ps_shift;
            if (p0 - win_lo >= 32) {
                win_lo += 32;
                win = entries(lu, win_lo, win_base);
            }
            const int page = __shfl_sync(0xffffffffu, win, p0 - win_lo);
            const int slot = tok & (g.ps - 1);
            const int at = __shfl_sync(0xffffffffu, win_base, p0 - win_lo) + slot;
            // keys a .. z - 1 of the step are there and seen
            int a = 0, z = 0;
            if (page >= 0) {
                a = g.window > 0 ? max(0, min(16, lu.pos - g.window + 1 - at)) : 0;
                z = max(a, min(16, lu.pos + 1 - at));
            }
            const int sh = 10 * stage;
            if constexpr (ST <= 3)
                meta = (meta & ~(1023u << sh)) | (uint32_t)(a | z << 5) << sh;
            else if (lane == stage)
                meta = (uint32_t)(a | z << 5);
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
                    cp_async16_row(to, k + i * step, 16);
                    cp_async16_row(to + 16 * ROW, v + i * step, 16);
                }
            } else {
#pragma unroll
                for (int i = 0; i < INS; ++i) {
                    const int r = i * RPI + r_lane;
                    const uint32_t to = dst + piece_at<D>(r, c_lane);
                    const bool ok = r >= a && r < z;
                    cp_async16_row(to, ok ? k + i * step : P.k, ok ? 16 : 0);
                    cp_async16_row(to + 16 * ROW, ok ? v + i * step : P.v, ok ? 16 : 0);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < ST - 1; ++s) issue(s);
    int stage = 0;

    // ---- Q rows of a unit, one warp a row: read ahead of the unit that needs them
    constexpr int QPW = Cfg::kRows / W, QW = D / 64;
    uint32_t qw[QPW][QW];
    auto load_q = [&](const SelUnit& x) {
#pragma unroll
        for (int i = 0; i < QPW; ++i) {
            const int r = warp + i * W;
#pragma unroll
            for (int j = 0; j < QW; ++j) qw[i][j] = 0u;
            if (r < g.G) {
                const uint32_t* src = reinterpret_cast<const uint32_t*>(
                    P.q + ((int64_t)x.row * g.Hq + (int64_t)x.hk * g.G + r) * D);
#pragma unroll
                for (int j = 0; j < QW; ++j) qw[i][j] = src[lane + 32 * j];
            }
        }
    };
    load_q(u);

    const float f = g.sm_scale * kLog2e;
    // ---- units
    while (true) {
        const SelShare sh = share_of(u, cost, lo, hi, warp, W);
#pragma unroll
        for (int i = 0; i < QPW; ++i)
#pragma unroll
            for (int j = 0; j < QW; ++j)
                *reinterpret_cast<uint32_t*>(smem + Cfg::kOffQ + (warp + i * W) * Cfg::kQRow +
                                             4 * (lane + 32 * j)) = qw[i][j];
        __syncthreads();
        SelUnit nu = u;
        const bool has_next = next_unit(P, nu) && nu.start < hi;
        if (has_next) load_q(nu);

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
        constexpr bool kQInRegs = NT == 1;
        uint32_t qf[kQInRegs ? KK : 1][2];
        // the B operands of two contraction steps: rows 8 nt + (lane & 7), piece 2 kk + lane / 8
        auto q_frag = [&](int nt, int kk, uint32_t* x) {
            ldsm_x4(qbase + (8 * nt + (lane & 7)) * Cfg::kQRow + (2 * kk + (lane >> 3)) * 16, x[0],
                    x[1], x[2], x[3]);
        };
        if constexpr (kQInRegs) {
#pragma unroll
            for (int kk = 0; kk < KK; kk += 2) {
                uint32_t x[4];
                q_frag(0, kk, x);
                qf[kk][0] = x[0];
                qf[kk][1] = x[1];
                qf[kk + 1][0] = x[2];
                qf[kk + 1][1] = x[3];
            }
        }

#pragma unroll 1
        for (int tok = sh.a; tok < sh.z; tok += 16) {
            cp_async_wait<ST - 2>();
            __syncwarp();
            uint32_t mt;
            if constexpr (ST <= 3)
                mt = meta >> (10 * stage);
            else
                mt = __shfl_sync(0xffffffffu, meta, stage);
            const int a = (int)(mt & 31u), z = (int)((mt >> 5) & 31u);
            issue(stage == 0 ? ST - 1 : stage - 1);   // into the stage the last step left
            const uint32_t sk = ring + stage * Cfg::kStage, sv = sk + 16 * ROW;
            stage = stage + 1 == ST ? 0 : stage + 1;
            if (z == a) continue;                     // no key of the step is there

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
                            mma_bf16_16816(s[nt], x, qf[kk][0], qf[kk][1]);
                            mma_bf16_16816(s1[nt], y, qf[kk + 1][0], qf[kk + 1][1]);
                        } else {
                            uint32_t b[4];
                            q_frag(nt, kk, b);
                            mma_bf16_16816(s[nt], x, b[0], b[1]);
                            mma_bf16_16816(kTwo ? s1[kTwo ? nt : 0] : s[nt], y, b[2], b[3]);
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[nt][e] = (kTwo ? s[nt][e] + s1[kTwo ? nt : 0][e] : s[nt][e]) * f;
            }
            if (a > 0 || z < 16) {
                // keys gr and gr + 8 of the step
                const bool k0 = gr >= a && gr < z, k1 = gr + 8 >= a && gr + 8 < z;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(e < 2 ? k0 : k1)) s[nt][e] = -INFINITY;
            }
            // ---- the running max moves where a score passes it by far
            bool far = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    far |= fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + kRise;
            if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(s[nt][e], s[nt][e + 2]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        if (x > m[nt][e]) {
                            const float al = m[nt][e] == kUnseen ? 0.f : ex2(m[nt][e] - x);
                            m[nt][e] = x;
                            l[nt][e] *= al;
#pragma unroll
                            for (int i = 0; i < OT; ++i) {
                                o[i][nt][e] *= al;
                                o[i][nt][e + 2] *= al;
                            }
                        }
                    }
            }
            // ---- probabilities, and their transposes as the B operand
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = ex2(s[nt][0] - m[nt][0]), p1 = ex2(s[nt][1] - m[nt][1]);
                const float p2 = ex2(s[nt][2] - m[nt][0]), p3 = ex2(s[nt][3] - m[nt][1]);
                l[nt][0] += p0 + p2;
                l[nt][1] += p1 + p3;
                pb[nt][0] = movmatrix_trans(pack_bf16x2(p0, p1));
                pb[nt][1] = movmatrix_trans(pack_bf16x2(p2, p3));
            }
            // ---- O^T += V^T P
            {
                const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
                for (int i = 0; i < OT; ++i) {
                    uint32_t x[4];
                    ldsm_x4_t(sv + piece_at<D>(r, 2 * i + c), x[0], x[1], x[2], x[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(o[i][nt], x, pb[nt][0], pb[nt][1]);
                }
            }
        }

        // ---- merge the warps, a few rows at a time
        if (sh.t1 > sh.t0) {
            const int64_t pos0 = u.start + cost;   // the CTAs that hold parts of the unit
            const int c_first = (int)(((pos0 + 1) * N - 1) / C);
            const int c_last = (int)(((pos0 + u.n) * N - 1) / C);
            const int part = c_first == c_last ? -1 : 2 * cta + (cta == c_first ? 1 : 0);
#pragma unroll
            for (int r0 = 0; r0 < Cfg::kRows; r0 += MR) {
                if (r0 >= g.G) break;
                const int nt = r0 / 8;
                float* mw = merge + warp * Cfg::kMergeWarp;
                // rows r0 .. r0 + 3 are with the lanes whose pairs are these columns
                const bool mine = t4 / 2 == (r0 % 8) / 4;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[nt][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    const int r = (2 * t4 + e) % MR;
                    if (mine) {
                        if (gr == 0) {
                            mw[MR * Cfg::kMergeRow + r] = m[nt][e];
                            mw[MR * Cfg::kMergeRow + MR + r] = x;
                        }
#pragma unroll
                        for (int i = 0; i < OT; ++i) {
                            mw[r * Cfg::kMergeRow + 16 * i + gr] = o[i][nt][e];
                            mw[r * Cfg::kMergeRow + 16 * i + 8 + gr] = o[i][nt][e + 2];
                        }
                    }
                }
                __syncthreads();
                // a warp a row
                static_assert(MR == W, "a warp a row");
                if (r0 + warp < g.G) {
                    const int mr = warp, r = r0 + warp;
                    constexpr int DPL = D / 32;
                    float M = kUnseen;
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        M = fmaxf(M, merge[w * Cfg::kMergeWarp + MR * Cfg::kMergeRow + mr]);
                    float den = 0.f, acc[DPL];
#pragma unroll
                    for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float* b = merge + w * Cfg::kMergeWarp;
                        const float mv = b[MR * Cfg::kMergeRow + mr];
                        const float lv = b[MR * Cfg::kMergeRow + MR + mr];
                        if (mv == kUnseen && lv == 0.f) continue;     // saw nothing
                        const float x = mv == kUnseen ? 1.f : ex2(mv - M);
                        den += x * lv;
#pragma unroll
                        for (int e = 0; e < DPL; ++e)
                            acc[e] += x * b[mr * Cfg::kMergeRow + lane * DPL + e];
                    }
                    // (a NaN sum is not "no visible key")
                    const bool none = den == 0.f;
                    const float inv = none ? 0.f : 1.f / den;
                    const float ln2 = none ? -INFINITY : (M == kUnseen ? den : (lg2(den) + M) * kLn2);
                    if (part < 0) {
                        const int64_t row = (int64_t)u.row * g.Hq + (int64_t)u.hk * g.G + r;
                        __nv_bfloat16* dst = P.out + row * D + lane * DPL;
#pragma unroll
                        for (int e = 0; e < DPL; e += 2)
                            *reinterpret_cast<uint32_t*>(dst + e) =
                                pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
                        if (P.lse != nullptr && lane == 0) P.lse[row] = ln2;
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
                __syncthreads();
            }
            if (part >= 0) {
                // the last of the unit's CTAs to come here joins the parts (nobody
                // waits for another CTA)
                if (threadIdx.x == 0) {
                    __threadfence();   // every warp's part is written (barrier above)
                    const uint32_t before = (uint32_t)atomicAdd(P.done + c_first, 1);
                    const bool last = before == (uint32_t)(c_last - c_first);
                    if (last) P.done[c_first] = 0;   // as the next call finds it
                    // (nobody will come last: the workspace did not start as zeros)
                    if (before > (uint32_t)(c_last - c_first))
                        flag_error(P.header + H_ERROR, PA_DEV_BAD_WORKSPACE);
                    __threadfence();
                    *flag = last ? 1 : 0;
                }
                __syncthreads();
                const bool last = *flag != 0;
                __threadfence();
                if (last) {
                    constexpr int DPL = D / 32;
                    for (int r = warp; r < g.G; r += W) {
                        // part c of the unit is in slot 2 c (the first in 2 c + 1); 32
                        // parts' lse at a time, one a lane
                        auto part_row = [&](int c) {
                            return (int64_t)(2 * c + (c == c_first ? 1 : 0)) * Cfg::kRows + r;
                        };
                        float M = -INFINITY;
                        bool poison = false;
                        for (int c = c_first + lane; c <= c_last; c += 32) {
                            const float x = __ldcg(P.part_lse + part_row(c));
                            poison |= x != x;
                            M = fmaxf(M, x);
                        }
#pragma unroll
                        for (int x = 16; x > 0; x >>= 1)
                            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
                        poison = __any_sync(0xffffffffu, poison);
                        float den = 0.f, acc[DPL];
#pragma unroll
                        for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
                        for (int c0 = c_first; c0 <= c_last; c0 += 32) {
                            float y = 0.f;
                            if (c0 + lane <= c_last) {
                                const float x = __ldcg(P.part_lse + part_row(c0 + lane));
                                y = poison ? NAN : x == -INFINITY ? 0.f : ex2((x - M) * kLog2e);
                            }
                            const int n = min(32, c_last - c0 + 1);
#pragma unroll 8
                            for (int j = 0; j < n; ++j) {
                                const float w = __shfl_sync(0xffffffffu, y, j);
                                const float* src = P.part_o + part_row(c0 + j) * D + lane * DPL;
                                float x[DPL];
#pragma unroll
                                for (int e = 0; e < DPL; e += 2)
                                    *reinterpret_cast<float2*>(x + e) =
                                        __ldcg(reinterpret_cast<const float2*>(src + e));
                                den += w;
#pragma unroll
                                for (int e = 0; e < DPL; ++e)
                                    if (w != 0.f) acc[e] = fmaf(w, x[e], acc[e]);
                            }
                        }
                        const bool none = den == 0.f;
                        const float inv = none ? 0.f : 1.f / den;
                        const int64_t row = (int64_t)u.row * g.Hq + (int64_t)u.hk * g.G + r;
                        __nv_bfloat16* dst = P.out + row * D + lane * DPL;
#pragma unroll
                        for (int e = 0; e < DPL; e += 2)
                            *reinterpret_cast<uint32_t*>(dst + e) =
                                pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
                        if (P.lse != nullptr && lane == 0)
                            P.lse[row] = none ? -INFINITY : M + lg2(den) * kLn2;
                    }
                }
            }
        }
        if (!has_next) break;
        if (sh.t1 <= sh.t0) __syncthreads();   // all have read this unit's Q rows
        u = nu;
    }
    cp_async_wait<0>();
}

template <int D, int NT>
cudaError_t launch(const SelectedParams& P, int grid, cudaStream_t stream) {
    using Cfg = SelCfg<D, NT>;
    const cudaError_t e = allow_smem<decode_selected_kernel<D, NT>>(Cfg::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(decode_selected_kernel<D, NT>, dim3(grid), dim3(Cfg::kThreads),
                            Cfg::kSmem, stream, P);
}

}  // namespace

// Row tiles (of 8) that are built: what holds a group of `heads`, -1 if none.
int selected_row_tiles(int D, int heads) {
    if (heads > (D == 128 ? 32 : 64)) return -1;
    return heads <= 8 ? 1 : heads <= 16 ? 2 : heads <= 32 ? 4 : 8;
}
int selected_ctas_per_sm() { return SelCfg<128, 1>::kCtas; }

cudaError_t launch_decode_selected(const SelectedParams& P, int nt, int grid, cudaStream_t stream) {
    if (P.g.D == 128) {
        switch (nt) {
            case 1: return launch<128, 1>(P, grid, stream);
            case 2: return launch<128, 2>(P, grid, stream);
            case 4: return launch<128, 4>(P, grid, stream);
        }
    } else {
        switch (nt) {
            case 1: return launch<64, 1>(P, grid, stream);
            case 2: return launch<64, 2>(P, grid, stream);
            case 4: return launch<64, 4>(P, grid, stream);
            case 8: return launch<64, 8>(P, grid, stream);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
