// pa_decode_mx4.cu -- decode attention over a PA_MX4 (4-bit) paged cache.
//
//   S^T = K Q^T,  P = exp2(S^T - m),  O^T += V^T P,  per KV head and sequence
//
// Persistent CTAs, a few per SM, take equal shares of the flat line of
// (sequence, KV head, 64-token tile); the warps of a CTA cut each unit's tokens
// between them in 32-token steps, every warp with its own running (max, sum, O), its
// own ring of cp.async stages that runs ahead over unit boundaries, and no
// barrier until the unit ends.  Then the warps' states merge through shared
// memory; a unit that spans CTAs leaves normalised parts in the workspace, and
// the last CTA to finish one joins them.
//
// What bounds it: 17/16 D bytes a key and head from HBM (136 at D = 128, K and
// V; with more rows than a block holds, every block of them reads the cache, two at
// most, also where a sequence's own rows fit one), and the instructions that
// turn 4-bit codes into operands.  So:
//   - products are transposed (mma m16n8k16 with 16 keys, or 16 columns of V,
//     as rows): R query rows cost ceil(R/8) products, no half-empty tiles;
//   - the contraction order is free, so each lane takes the bytes of a row as
//     they lie: 4 bytes = 8 codes of one 32-block for K, 16 codes of one block
//     for V; codes become f16 pairs by one conversion each, exactly;
//   - K's block scales multiply the fp32 block scores (a block is two mma
//     steps), V's multiply the f16 codes, relative to the largest scale its
//     columns met so far (moved as rarely as the running max);
//   - the running max moves only when a score passes it by 2^8, decided by one
//     vote; a row's max is otherwise never reduced over lanes;
//   - P carries a factor 2^7, which the division by its sum takes out: below 2^15
//     in f16, whose normal range then reaches down to 2^-21 of the row's largest
//     probability.  What is smaller rounds to multiples of 2^-31 of that, so keys
//     beside one that outweighs them all still count.
// Masked scores are -inf and V rows past the context are zero codes, so
// nothing outside a row's sight reaches it, nor a key whose page is none; a NaN
// block (scale 255) reaches exactly the rows that see its key.
#include "pa_cache_mma.cuh"

namespace pa {

struct Mx4Params {
    CacheGeom g;
    const __nv_bfloat16* q;
    const uint8_t* k;
    const uint8_t* ks;
    const uint8_t* v;
    const uint8_t* vs;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* ql;
    int32_t* header;     // error word at H_ERROR
    int32_t* done;       // completion counter of the unit a CTA begins
    float* part_o;       // [2 * grid][rows][D]
    float* part_lse;     // [2 * grid][rows]
    __nv_bfloat16* out;
    float* lse;
    int32_t unit_cost;   // fixed cost of a unit, in tiles (line_fits)
};

// No CTA takes less than this of the flat line: joining a unit's parts costs more
// than the tiles it would spread (3 sequences of 37 to 100 tokens: 11.7 us with 1,
// 6.5 with 4, 7.0 with 8; one of 4000 tokens, 8 heads: 13.8, 11.5 and 16.1).
constexpr int kMinShare = 4;

template <int D, int NT>
struct Mx4Cfg {
    // CTAs of an SM: what the registers of a thread (O alone takes NT D / 4)
    // leave room for.  Measured on 64 sequences of 128 to 32768 tokens: 8 rows, D =
    // 128, 3 CTAs of 4 warps (168 registers) 105 us, 4 (128 registers, and spills)
    // 112; 16 rows, D = 128, 2 CTAs (255 registers) 145 us, 3 (spills) 173; 32
    // rows, D = 64, 182 and 193
    static constexpr int kPerThread = NT * D;
    static constexpr int kCtas = kPerThread <= 128 ? 3 : 2;
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = kPerThread <= 128 ? 2 : 3;   // (8 rows, 3: 106 us)
    static constexpr int kStep = 32;                       // tokens of a warp's step
    static constexpr int kRow = D / 2;                     // code bytes of a row
    static constexpr int kStage = 2 * kStep * (kRow + 4);  // K, V, their scale words
    static constexpr int kRows = 8 * NT;
    static constexpr int kQPerWarp = kRows / kWarps;
    static constexpr int kQRow = 2 * D + kQPad;
    static constexpr bool kQInRegs = kPerThread <= 128;   // few enough rows to keep
    static constexpr int kMergeRow = D + 4;                // floats
    static constexpr int kMergeWarp = 8 * kMergeRow + 16;  // 8 rows, then up[8], l[8]
    static constexpr int kOffQ = kWarps * kStages * kStage;
    static constexpr int kOffInfo = kOffQ + kRows * kQRow;  // per row: score factor
    static constexpr int kOffMerge = kOffInfo + kRows * 4;
    static constexpr int kOffFlag = kOffMerge + kWarps * kMergeWarp * 4;
    static constexpr int kSmem = kOffFlag + 16;
    static_assert((kSmem + 1024) * kCtas <= 233472, "shared memory");
    static_assert(kOffQ % 16 == 0 && kOffMerge % 16 == 0, "alignment");
};

namespace {

// A row's state is up = kPBits - running max: P = exp2(score + up), at most 2^(kPBits
// + kPRise).  kUpNone: no key seen yet, any score passes the max.
constexpr float kPBits = 7.f, kPRise = 8.f, kUpNone = 3.402823466e38f;

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 2^(e - 127) of the first 2 N bytes of a word as bf16 pairs (exact; e = 255: NaN).
template <int N>
__device__ __forceinline__ void e8m0_to_bf16(uint32_t w, uint32_t* d) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(d[i]) : "h"((uint16_t)(w >> (16 * i))));
}

// A unit (sequence, KV head, block of query rows) as a CTA meets it.
struct Unit {
    int b, hk, blk;
    int ctx, ql, row0;     // lengths, first query row
    int n, first;          // tiles, the first tile any row sees
    int64_t start;         // position of its fixed cost on the flat line
};

// Tiles of 64 tokens that sequence b's rows see, 0 if it has none or bad lengths.
__device__ __forceinline__ int seq_tiles(const CacheGeom& g, int c, int q, int& first) {
    first = 0;
    if (q <= 0 || !good_lens(g, q, c)) return 0;
    first = window_first_tile(g.window, c - q, kDecodeTile);
    return (c + kDecodeTile - 1) / kDecodeTile - first;
}

__device__ __forceinline__ void load_seq(const Mx4Params& P, Unit& u) {
    u.ctx = P.ctx[u.b];
    u.ql = P.ql[u.b];
    u.n = seq_tiles(P.g, u.ctx, u.ql, u.first);
}

// The unit after u (every lane the same); false past the last sequence.
template <int RB>
__device__ __forceinline__ bool next_unit(const Mx4Params& P, Unit& u) {
    u.start += P.unit_cost + u.n;
    if (RB > 1 && ++u.blk < RB) return true;
    u.blk = 0;
    if (++u.hk < P.g.Hkv) return true;
    u.hk = 0;
    do {
        u.row0 += clamp_q(P.g, u.ql);
        if (++u.b >= P.g.B) return false;
        load_seq(P, u);
    } while (u.n == 0);
    return true;
}

// What warp w of W runs of unit u, of the CTA's share [lo, hi) of the flat line.
struct Share {
    int t0, t1;     // tiles of the unit in the CTA's share
    int s0, s1;     // the warp's 32-token steps, counted from token tok0
    int tok0;
};
__device__ __forceinline__ Share share_of(const Unit& u, int cost, int64_t lo, int64_t hi, int w,
                                          int W) {
    Share s;
    const int64_t base = u.start + cost;
    s.t0 = (int)max((int64_t)0, min((int64_t)u.n, lo - base));
    s.t1 = (int)max((int64_t)0, min((int64_t)u.n, hi - base));
    s.tok0 = (u.first + s.t0) * kDecodeTile;
    const int end = min(u.ctx, (u.first + s.t1) * kDecodeTile);
    const int steps = s.t1 > s.t0 ? (end - s.tok0 + 31) / 32 : 0;
    s.s0 = steps * w / W;
    s.s1 = steps * (w + 1) / W;
    return s;
}

// Row of a 16-key tile that operand row / contraction index i stands for.  Any
// bijection gives the same sums; this one keeps V's loads off one another's
// banks (four keys at a time, rows of 64 or 32 bytes).
template <int D>
__device__ __forceinline__ int tile_key(int i) {
    const int x = i & 7;
    const int y = D == 128 ? (x & 4) | ((x & 1) << 1) | ((x >> 1) & 1)
                           : (x >> 1) | ((x & 1) << 2);
    return (i & 8) | y;
}
// 16-byte chunk position of chunk c of row r
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
    return D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1);
}

// NT row tiles of 8 at a time; RB: blocks of that many rows, each a unit of its own.
template <int D, int NT, int RB>
__global__ void __launch_bounds__(Mx4Cfg<D, NT>::kThreads, Mx4Cfg<D, NT>::kCtas)
decode_mx4_kernel(const __grid_constant__ Mx4Params P) {
    using Cfg = Mx4Cfg<D, NT>;
    constexpr int W = Cfg::kWarps, ST = Cfg::kStages, ROW = Cfg::kRow;
    constexpr int KB = D / 32;      // blocks of a row
    constexpr int OT = D / 16;      // 16-column tiles of O
    constexpr int VW = D / 64;      // words of V codes a lane takes of a key
    extern __shared__ __align__(128) uint8_t smem[];
    const CacheGeom& g = P.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gr = lane >> 2, t4 = lane & 3;   // operand row, column pair
    const int cost = P.unit_cost;
    grid_dependency_wait();

    // ---- this CTA's share of the flat line
    auto seq_cost = [&](int b) -> int64_t {
        int first;
        const int n = seq_tiles(g, P.ctx[b], P.ql[b], first);
        return n > 0 ? (int64_t)g.Hkv * RB * (n + cost) : 0;
    };
    const int64_t C = flat_total(g.B, lane, seq_cost);
    if (blockIdx.x == 0 && warp == 0) check_lens(g, P.ctx, P.ql, lane, P.header + H_ERROR);
    const int64_t N = min((int64_t)gridDim.x, (C + kMinShare - 1) / kMinShare);
    const int cta = blockIdx.x;
    if (cta >= N) return;
    const int64_t lo = C * cta / N, hi = C * (cta + 1) / N;
    Unit u;
    {
        int64_t start;
        int rows;
        u.b = flat_find(g.B, lane, lo, seq_cost, [&](int b) { return clamp_q(g, P.ql[b]); }, start,
                        rows);
        load_seq(P, u);
        u.row0 = rows;
        const int i = (int)((lo - start) / (u.n + cost));
        u.hk = i / RB;
        u.blk = i % RB;
        u.start = start + (int64_t)i * (u.n + cost);
    }

    const uint32_t ring = smem_u32(smem) + warp * ST * Cfg::kStage;
    const uint32_t qbase = smem_u32(smem + Cfg::kOffQ);
    float* info = reinterpret_cast<float*>(smem + Cfg::kOffInfo);
    float* merge = reinterpret_cast<float*>(smem + Cfg::kOffMerge);
    volatile int* flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffFlag);

    // ---- the load side runs ST - 1 steps ahead, over unit boundaries
    constexpr int CH = ROW / 16, RPI = 32 / CH;   // chunks of a row, rows an instruction
    constexpr int HALF = 16 / RPI;                // instructions for 16 rows
    static_assert(RPI % 8 == 0, "the chunk order repeats every 8 rows");
    // a block of rows reads codes once; a sector of scales serves several heads
    uint64_t once, again;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(again));
    const int page_rows = g.ps * g.Hkv;
    const int64_t lane_off = (int64_t)(lane / CH) * g.tok_rows * ROW + (lane % CH) * 16;
    const int64_t ins_off = (int64_t)RPI * g.tok_rows * ROW;
    const uint32_t lane_at = (lane / CH) * ROW + chunk_at<D>(lane / CH, lane % CH) * 16;
    // page id p + lane of a sequence
    auto page_ids = [&](const Unit& x, int p) -> int {
        const int npg = (x.ctx + g.ps - 1) >> g.ps_shift;
        return p + lane < npg ? P.table[(int64_t)x.b * g.mpps + p + lane] : -1;
    };
    auto first_page = [&](const Share& x) { return (x.tok0 + 32 * x.s0) >> g.ps_shift; };
    Unit ln = u;                             // the unit after the one being loaded
    Share ls = share_of(u, cost, lo, hi, warp, W);
    bool more = true;
    int l_tok = ls.tok0 + 32 * ls.s0, l_end = ls.tok0 + 32 * ls.s1, l_ctx = u.ctx, l_hk = u.hk;
    int l_b = u.b;
    int win_lo = first_page(ls);             // 32 page ids, the 32 after them, the next unit's
    int win = page_ids(u, win_lo), nxt = page_ids(u, win_lo + 32), lnw = -1;
    uint32_t bad = 0;                        // two bits a stage: halves whose page is none
    bool ln_ok = next_unit<RB>(P, ln) && ln.start < hi;
    if (ln_ok) lnw = page_ids(ln, first_page(share_of(ln, cost, lo, hi, warp, W)));
    auto issue = [&](int stage) {
        while (more && l_tok >= l_end) {
            more = ln_ok;
            if (!more) break;
            const Share x = share_of(ln, cost, lo, hi, warp, W);
            l_tok = x.tok0 + 32 * x.s0;
            l_end = x.tok0 + 32 * x.s1;
            l_ctx = ln.ctx;
            l_hk = ln.hk;
            l_b = ln.b;
            win_lo = first_page(x);
            win = lnw;
            nxt = page_ids(ln, win_lo + 32);
            ln_ok = next_unit<RB>(P, ln) && ln.start < hi;
            if (ln_ok) lnw = page_ids(ln, first_page(share_of(ln, cost, lo, hi, warp, W)));
        }
        if (more) {
            const int tok = l_tok;
            l_tok += 32;
            const int p0 = tok >> g.ps_shift;
            if (p0 - win_lo >= 32) {         // (steps advance by at most two pages: p0 is next)
                win = nxt;
                win_lo += 32;
                const int p = win_lo + 32 + lane;
                nxt = p < (l_ctx + g.ps - 1) >> g.ps_shift ? P.table[(int64_t)l_b * g.mpps + p] : -1;
            }
            // rows where the step's two halves begin
            const int pa = __shfl_sync(0xffffffffu, win, p0 - win_lo);
            int64_t ra = (int64_t)pa * page_rows +
                         ((tok & (g.ps - 1)) * g.tok_rows + l_hk * g.head_rows);
            int64_t rb = ra + 16 * g.tok_rows;
            bool oka = (uint32_t)pa < (uint32_t)g.num_pages, okb = oka;
            if (g.ps == 16) {
                const int pb = __shfl_sync(0xffffffffu, win, p0 + 1 - win_lo);
                okb = (uint32_t)pb < (uint32_t)g.num_pages;
                rb = (int64_t)pb * page_rows + l_hk * g.head_rows;
            }
            const uint32_t dst = ring + stage * Cfg::kStage;
            const uint32_t dsc = dst + 64 * ROW + lane * 4;
            const int left = l_ctx - tok;       // tokens that exist
            // (D = 64: the word that holds the key's two bytes)
            const int64_t so = ((lane < 16 ? ra : rb) + (lane & 15) * g.tok_rows) * KB & ~(int64_t)3;
            if (left >= 32 && oka && okb) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t off = (h ? rb : ra) * ROW + lane_off;
                    const uint8_t* k = P.k + off;
                    const uint8_t* v = P.v + off;
#pragma unroll
                    for (int i = 0; i < HALF; ++i) {
                        const uint32_t at = dst + lane_at + (h * HALF + i) * RPI * ROW;
                        cp_async16(at, k, 16, once);
                        cp_async16(at + 32 * ROW, v, 16, once);
                        k += ins_off;
                        v += ins_off;
                    }
                }
                cp_async4(dsc, P.ks + so, 4, again);
                cp_async4(dsc + 128, P.vs + so, 4, again);
            } else {
                // keys that do not exist, or whose page does not: zero codes and scales
#pragma unroll
                for (int i = 0; i < 2 * HALF; ++i) {
                    const int r = i * RPI + lane / CH;
                    const bool second = i >= HALF;
                    const bool ok = r < left && (second ? okb : oka);
                    const int64_t off = ok ? (second ? rb : ra) * ROW + lane_off +
                                                 (i - (second ? HALF : 0)) * ins_off
                                           : 0;
                    const uint32_t at = dst + lane_at + i * RPI * ROW;
                    cp_async16(at, P.k + off, ok ? 16 : 0, once);
                    cp_async16(at + 32 * ROW, P.v + off, ok ? 16 : 0, once);
                }
                const bool ok = lane < left && (lane < 16 ? oka : okb);
                cp_async4(dsc, P.ks + (ok ? so : 0), ok ? 4 : 0, again);
                cp_async4(dsc + 128, P.vs + (ok ? so : 0), ok ? 4 : 0, again);
                const uint32_t none = (oka ? 0u : 1u) | (left > 16 && !okb ? 2u : 0u);
                bad |= none << (2 * stage);
                if (none != 0 && lane == 0) flag_error(P.header + H_ERROR, PA_DEV_BAD_PAGE);
            }
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < ST - 1; ++s) issue(s);
    int stage = 0;

    // ---- Q rows of a unit, one warp a row: read ahead of the unit that needs them
    uint32_t qw[Cfg::kQPerWarp][D / 64];
    // (rows past total_q_tokens, lengths that do not add up, are not there)
    auto rows_of = [&](const Unit& x) -> int {
        const int rows = x.row0 + x.ql <= g.total_q ? g.G * x.ql : 0;
        return RB > 1 ? max(0, min(Cfg::kRows, rows - x.blk * Cfg::kRows)) : rows;
    };
    auto load_q = [&](const Unit& x) {
        const int R = rows_of(x), r0 = x.blk * Cfg::kRows;
#pragma unroll
        for (int k = 0; k < Cfg::kQPerWarp; ++k) {
            const int r = warp + k * W;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) qw[k][j] = 0u;
            if (r < R) {
                const __nv_bfloat16* src =
                    P.q + ((int64_t)(x.row0 + (r0 + r) / g.G) * g.Hq + x.hk * g.G + (r0 + r) % g.G) * D;
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
                    qw[k][j] = reinterpret_cast<const uint32_t*>(src)[lane + 32 * j];
            }
        }
    };
    load_q(u);

    // ---- units
    while (true) {
        const int R = rows_of(u), r0 = u.blk * Cfg::kRows;
        const int ctx = u.ctx, pbase = u.ctx - u.ql;
        const Share sh = share_of(u, cost, lo, hi, warp, W);
        // Q rows as f16 with a power of two taken out of each: no element
        // leaves f16's range at the top, and what falls off the bottom is
        // 2^-25 of the row's largest
#pragma unroll
        for (int k = 0; k < Cfg::kQPerWarp; ++k) {
            const int r = warp + k * W;
            float x[D / 32], top = 0.f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                x[2 * j] = __uint_as_float(qw[k][j] << 16);
                x[2 * j + 1] = __uint_as_float(qw[k][j] & 0xffff0000u);
                top = fmaxf(top, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
            }
            // (magnitudes order like their bits)
            const uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            // exponent field of the largest, kept where both powers are normal
            const int e = max(8, min(247, (int)(tb >> 23)));
            const float down = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
                *reinterpret_cast<uint32_t*>(smem + Cfg::kOffQ + r * Cfg::kQRow +
                                             4 * (lane + 32 * j)) =
                    pack_f16x2(x[2 * j] * down, x[2 * j + 1] * down);
            // (never 0, so that a masked score times it stays -inf)
            if (lane == 0)
                info[r] = fmaxf(__uint_as_float((uint32_t)e << 23) * (g.sm_scale * kLog2e),
                                1.2e-38f);
        }
        __syncthreads();
        Unit nu = u;
        const bool has_next = next_unit<RB>(P, nu) && nu.start < hi;
        if (has_next) load_q(nu);

        float up[NT][2], l[NT][2], fq[NT][2];
        int pr[NT][2];              // last visible position of the thread's rows
        float o[OT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + 2 * t4 + e;
                up[nt][e] = kUpNone;
                l[nt][e] = 0.f;
                fq[nt][e] = info[r];
                pr[nt][e] = r < R ? pbase + (r0 + r) / g.G : -1;
            }
#pragma unroll
            for (int i = 0; i < OT; ++i)
                o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
        }
        uint4 qf[Cfg::kQInRegs ? NT : 1][KB];
        if constexpr (Cfg::kQInRegs) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
                    qf[nt][kb] = lds128(qbase + (8 * nt + gr) * Cfg::kQRow + kb * 64 + t4 * 16);
        }
        int vref = -1000;           // exponent that V's codes are scaled against

#pragma unroll 1
        for (int step = sh.s0; step < sh.s1; ++step) {
            cp_async_wait<ST - 2>();
            __syncwarp();
            issue(stage == 0 ? ST - 1 : stage - 1);   // into the stage the last step left
            const int tok = sh.tok0 + 32 * step;
            const uint32_t sk = ring + stage * Cfg::kStage, sv = sk + 32 * ROW;
            const uint32_t sks = sv + 32 * ROW, svs = sks + 128;
            // head_dim 64: which half of its scale word a key's two bytes are
            auto scale_shift = [&](int key) -> int {
                if constexpr (D == 128) return 0;
                const int x = (tok + key) & (g.ps - 1);
                return ((x * g.tok_rows + u.hk * g.head_rows) & 1) * 16;
            };
            auto visible = [&](int key, int nt, int e) -> bool {
                const int j = tok + key, p = pr[nt][e];
                return j <= p && (g.window == 0 || j > p - g.window);
            };

            // ---- scores of 2 x 16 keys (before the row's factor)
            float s[2][NT][4];
            const int key0 = tile_key<D>(gr);
            uint32_t kf[2][2][KB / 2];      // K's scales, pairs of blocks
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int key = key0 + 16 * mt + 8 * hh;
                    e8m0_to_bf16<KB / 2>(lds32(sks + key * 4) >> scale_shift(key), kf[mt][hh]);
                }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint4 b[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if constexpr (Cfg::kQInRegs)
                        b[nt] = qf[nt][kb];
                    else
                        b[nt] = lds128(qbase + (8 * nt + gr) * Cfg::kQRow + kb * 64 + t4 * 16);
                }
                const uint32_t at = sk + key0 * ROW + chunk_at<D>(key0, kb) * 16 + t4 * 4;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    uint32_t a[2][4];
                    e2m1x8_to_f16(lds32(at + 16 * mt * ROW), a[0][0], a[0][2], a[1][0], a[1][2]);
                    e2m1x8_to_f16(lds32(at + (16 * mt + 8) * ROW), a[0][1], a[0][3], a[1][1],
                                  a[1][3]);
                    const uint64_t f0 = pair2(__uint_as_float(
                        kb & 1 ? kf[mt][0][kb / 2] & 0xffff0000u : kf[mt][0][kb / 2] << 16));
                    const uint64_t f1 = pair2(__uint_as_float(
                        kb & 1 ? kf[mt][1][kb / 2] & 0xffff0000u : kf[mt][1][kb / 2] << 16));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float x[4];
                        mma_f16_first(x, a[0], b[nt].x, b[nt].y);
                        mma_f16_16816(x, a[1], b[nt].z, b[nt].w);
                        float* d = s[mt][nt];
                        if (kb == 0) {
                            mul2(d, x, f0);
                            mul2(d + 2, x + 2, f1);
                        } else {
                            fma2(d, x, f0);
                            fma2(d + 2, x + 2, f1);
                        }
                    }
                }
            }
            // the mask, where a row does not see the whole step
            if (!(tok + 31 <= pbase && (g.window == 0 || tok > ctx - 1 - g.window))) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!visible(16 * mt + 8 * (e >> 1) + key0, nt, e & 1))
                                s[mt][nt][e] = -INFINITY;
            }
            // nobody sees keys whose page is none
            if (bad != 0) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
                    if (bad >> (2 * stage + mt) & 1u) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[mt][nt][e] = -INFINITY;
                    }
                bad &= ~(3u << (2 * stage));
            }
            // ---- V's scale bytes of the thread's keys and columns
            int ve[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 16 * mt + 8 * (e >> 1) + tile_key<D>(2 * t4 + (e & 1));
                    ve[mt][e] = (int)lds8(svs + key * 4 + scale_shift(key) / 8 +
                                          (D == 128 ? gr / 2 : gr / 4));
                }
            const int vmax = max(max(max(max(ve[0][0], ve[0][1]), ve[0][2]), max(ve[0][3], ve[1][0])),
                                 max(max(ve[1][1], ve[1][2]), ve[1][3]));
            const int vmin = min(min(min(min(ve[0][0], ve[0][1]), ve[0][2]), min(ve[0][3], ve[1][0])),
                                 min(min(ve[1][1], ve[1][2]), ve[1][3]));
            // ---- what the plain course below does not cover: a score far above
            // its row's running max, a V scale outside [-14, 4] binary orders of
            // its columns' reference, or none
            bool odd_step = vmax > vref + 4 || vmin < vref - 14 || vmax == 255;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    odd_step |= fmaf(fmaxf(fmax3(s[0][nt][e], s[0][nt][e + 2], s[1][nt][e]),
                                           s[1][nt][e + 2]),
                                     fq[nt][e], up[nt][e]) > kPBits + kPRise;
            bool nan_v = false, wide_v = false;
            if (__any_sync(0xffffffffu, odd_step)) {
                int top = -1000;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        nan_v |= ve[mt][e] == 255;
                        if (ve[mt][e] != 255) top = max(top, ve[mt][e]);
                    }
                nan_v = __any_sync(0xffffffffu, nan_v);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                float vfac = 1.f;
                if (top > vref) {
                    vfac = vref < 0 ? 0.f : ex2((float)(vref - top));
                    vref = top;
                }
                wide_v = __any_sync(0xffffffffu, vmin < vref - 14) || nan_v;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(fmax3(s[0][nt][e], s[0][nt][e + 2], s[1][nt][e]),
                                        s[1][nt][e + 2]) * fq[nt][e];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        float al = 1.f;
                        if (kPBits - x < up[nt][e]) {
                            al = ex2(kPBits - x - up[nt][e]);
                            up[nt][e] = kPBits - x;
                        }
                        l[nt][e] *= al;
                        const float f = al * vfac;
#pragma unroll
                        for (int i = 0; i < OT; ++i) {
                            o[i][nt][e] *= f;
                            o[i][nt][e + 2] *= f;
                        }
                    }
            }
            // ---- probabilities, and their transposes as the B operand
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const float p0 = ex2(fmaf(s[mt][nt][0], fq[nt][0], up[nt][0]));
                    const float p1 = ex2(fmaf(s[mt][nt][1], fq[nt][1], up[nt][1]));
                    const float p2 = ex2(fmaf(s[mt][nt][2], fq[nt][0], up[nt][0]));
                    const float p3 = ex2(fmaf(s[mt][nt][3], fq[nt][1], up[nt][1]));
                    l[nt][0] += p0 + p2;
                    l[nt][1] += p1 + p3;
                    pb[mt][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
                    pb[mt][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
                }
            }
            // ---- O^T += V^T P
            // f16 scales of a pair of keys: exponent fields e - vref + 15, in 1 .. 19
            const uint32_t vbias = (uint32_t)(15 - vref) * 0x04000400u;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t sc[2];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                    sc[hh] = (uint32_t)ve[mt][2 * hh] * 0x400u +
                             ((uint32_t)ve[mt][2 * hh + 1] * 0x4000000u + vbias);
                if (wide_v) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        float f[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int x = ve[mt][2 * hh + e];
                            f[e] = x == 255 ? 0.f
                                            : __uint_as_float((uint32_t)max(0, x - vref + 127) << 23);
                        }
                        sc[hh] = pack_f16x2(f[0], f[1]);
                    }
                }
                uint32_t even[2][VW], odd[2][VW];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int ka = tile_key<D>(2 * t4), kb = tile_key<D>(2 * t4 + 1);
                    const uint32_t row = sv + (16 * mt + 8 * hh) * ROW;
                    uint32_t wa[VW], wb[VW];
                    if constexpr (D == 128) {
                        const uint2 x =
                            lds64(row + ka * ROW + chunk_at<D>(ka, gr >> 1) * 16 + (gr & 1) * 8);
                        const uint2 y =
                            lds64(row + kb * ROW + chunk_at<D>(kb, gr >> 1) * 16 + (gr & 1) * 8);
                        wa[0] = x.x;
                        wa[VW - 1] = x.y;
                        wb[0] = y.x;
                        wb[VW - 1] = y.y;
                    } else {
                        wa[0] = lds32(row + ka * ROW + chunk_at<D>(ka, gr >> 2) * 16 + (gr & 3) * 4);
                        wb[0] = lds32(row + kb * ROW + chunk_at<D>(kb, gr >> 2) * 16 + (gr & 3) * 4);
                    }
                    // bytes of (key a, key b) codes: even columns, odd columns
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        even[hh][w] = (wa[w] & 0x0f0f0f0fu) | ((wb[w] << 4) & 0xf0f0f0f0u);
                        odd[hh][w] = ((wa[w] >> 4) & 0x0f0f0f0fu) | (wb[w] & 0xf0f0f0f0u);
                    }
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    uint32_t a[4][4];
                    e2m1x8_to_f16(even[0][w], a[0][0], a[1][0], a[2][0], a[3][0]);
                    e2m1x8_to_f16(odd[0][w], a[0][1], a[1][1], a[2][1], a[3][1]);
                    e2m1x8_to_f16(even[1][w], a[0][2], a[1][2], a[2][2], a[3][2]);
                    e2m1x8_to_f16(odd[1][w], a[0][3], a[1][3], a[2][3], a[3][3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[j][0] = hmul2(a[j][0], sc[0]);
                        a[j][1] = hmul2(a[j][1], sc[0]);
                        a[j][2] = hmul2(a[j][2], sc[1]);
                        a[j][3] = hmul2(a[j][3], sc[1]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(o[4 * w + j][nt], a[j], pb[mt][nt][0], pb[mt][nt][1]);
                    }
                }
            }
            if (nan_v) {
                // a NaN block of V makes its columns NaN in the rows that see the key
#pragma unroll 1
                for (int key = 0; key < 32; ++key) {
                    if (lds8(svs + key * 4 + scale_shift(key) / 8 +
                             (D == 128 ? gr / 2 : gr / 4)) != 255u)
                        continue;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (visible(key, nt, e & 1))
#pragma unroll
                                for (int i = 0; i < OT; ++i) o[i][nt][e] = NAN;
                }
            }
            stage = stage + 1 == ST ? 0 : stage + 1;
        }

        // ---- merge the warps, eight rows at a time
        if (sh.t1 > sh.t0) {
            const float vmul = vref < 0 ? 0.f : e8m0_to_f32((uint32_t)vref);
            const int64_t pos0 = u.start + cost;   // the CTAs that hold parts of the unit
            const int c_first = (int)(((pos0 + 1) * N - 1) / C);
            const int c_last = (int)(((pos0 + u.n) * N - 1) / C);
            const int part = c_first == c_last ? -1 : 2 * cta + (cta == c_first ? 1 : 0);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (8 * nt < R) {
                    float* mw = merge + warp * Cfg::kMergeWarp;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = l[nt][e];
                        x += __shfl_xor_sync(0xffffffffu, x, 4);
                        x += __shfl_xor_sync(0xffffffffu, x, 8);
                        x += __shfl_xor_sync(0xffffffffu, x, 16);
                        if (gr == 0) {
                            mw[8 * Cfg::kMergeRow + 2 * t4 + e] =
                                sh.s1 > sh.s0 ? up[nt][e] : kUpNone;
                            mw[8 * Cfg::kMergeRow + 8 + 2 * t4 + e] = x;
                        }
                        // the thread's columns are consecutive: OT pairs from gr * D / 8
                        if (sh.s1 > sh.s0) {
                            float* row = mw + (2 * t4 + e) * Cfg::kMergeRow + gr * (D / 8);
#pragma unroll
                            for (int i = 0; i < OT; i += 2)
                                *reinterpret_cast<float4*>(row + 2 * i) =
                                    make_float4(o[i][nt][e] * vmul, o[i][nt][e + 2] * vmul,
                                                o[i + 1][nt][e] * vmul, o[i + 1][nt][e + 2] * vmul);
                        }
                    }
                    __syncthreads();
#pragma unroll 1
                    for (int mr = warp; mr < 8 && 8 * nt + mr < R; mr += W) {
                        const int r = 8 * nt + mr;
                        constexpr int DPL = D / 32;
                        float U = kUpNone;
#pragma unroll
                        for (int w = 0; w < W; ++w)
                            U = fminf(U, merge[w * Cfg::kMergeWarp + 8 * Cfg::kMergeRow + mr]);
                        float den = 0.f, acc[DPL];
#pragma unroll
                        for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
#pragma unroll 4
                        for (int w = 0; w < W; ++w) {
                            const float* b = merge + w * Cfg::kMergeWarp;
                            const float uv = b[8 * Cfg::kMergeRow + mr];
                            const float lv = b[8 * Cfg::kMergeRow + 8 + mr];
                            if (uv == kUpNone && lv == 0.f) continue;     // saw nothing
                            const float f = uv == kUpNone ? 1.f : ex2(U - uv);
                            den += f * lv;
#pragma unroll
                            for (int e = 0; e < DPL; ++e)
                                acc[e] += f * b[mr * Cfg::kMergeRow + lane * DPL + e];
                        }
                        // (a NaN sum is not "no visible key")
                        const bool none = den == 0.f;
                        const float inv = none ? 0.f : 1.f / den;
                        const float ln = none ? -INFINITY
                                              : (U == kUpNone ? den : (lg2(den) - U) * kLn2);
                        if (part < 0) {
                            const int64_t row =
                                (int64_t)(u.row0 + (r0 + r) / g.G) * g.Hq + u.hk * g.G + (r0 + r) % g.G;
                            __nv_bfloat16* dst = P.out + row * D + lane * DPL;
#pragma unroll
                            for (int e = 0; e < DPL; e += 2)
                                *reinterpret_cast<uint32_t*>(dst + e) =
                                    pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
                            if (P.lse != nullptr && lane == 0) P.lse[row] = ln;
                        } else {
                            const int64_t row = (int64_t)part * Cfg::kRows + r;
                            float* dst = P.part_o + row * D + lane * DPL;
                            if constexpr (DPL == 4)
                                *reinterpret_cast<float4*>(dst) = make_float4(
                                    acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
                            else
                                *reinterpret_cast<float2*>(dst) =
                                    make_float2(acc[0] * inv, acc[1] * inv);
                            if (lane == 0) P.part_lse[row] = ln;
                        }
                    }
                    __syncthreads();
                }
            }
            if (part >= 0 && R > 0) {
                // the last of the unit's CTAs to come here joins the parts (nobody
                // waits for another CTA): its first warp alone where there are few,
                // while the others go on to the next unit
                const bool alone = c_last - c_first < 8;
                bool last = false;
                if (threadIdx.x == 0) {
                    __threadfence();   // every warp's part is written (barrier above)
                    const uint32_t before = (uint32_t)atomicAdd(P.done + c_first, 1);
                    last = before == (uint32_t)(c_last - c_first);
                    if (last) P.done[c_first] = 0;   // as the next call finds it
                    // (nobody will come last: the workspace did not start as zeros)
                    if (before > (uint32_t)(c_last - c_first))
                        flag_error(P.header + H_ERROR, PA_DEV_BAD_WORKSPACE);
                    __threadfence();
                    *flag = last ? 1 : 0;
                }
                if (alone) {
                    last = warp == 0 && __any_sync(0xffffffffu, last);
                    __syncwarp();      // (a vote orders no memory: what thread 0 has seen
                                       // written, the warp sees from here on)
                } else {
                    __syncthreads();
                    last = *flag != 0;
                    __threadfence();
                    __syncthreads();
                }
                if (last) {
                    constexpr int DPL = D / 32;
                    for (int r = alone ? 0 : warp; r < R; r += alone ? 1 : W) {
                        // part c of the unit is in slot 2 c (the first in 2 c + 1); 32
                        // parts' lse at a time, one a lane
                        auto part_row = [&](int c) {
                            return (int64_t)(2 * c + (c == c_first ? 1 : 0)) * Cfg::kRows + r;
                        };
                        float M = -INFINITY;
                        bool poison = false;
                        for (int c = c_first + lane; c <= c_last; c += 32) {
                            const float v = __ldcg(P.part_lse + part_row(c));
                            poison |= v != v;
                            M = fmaxf(M, v);
                        }
#pragma unroll
                        for (int x = 16; x > 0; x >>= 1)
                            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
                        poison = __any_sync(0xffffffffu, poison);
                        float den = 0.f, acc[DPL];
#pragma unroll
                        for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
                        for (int c0 = c_first; c0 <= c_last; c0 += 32) {
                            float f = 0.f;
                            if (c0 + lane <= c_last) {
                                const float v = __ldcg(P.part_lse + part_row(c0 + lane));
                                f = poison ? NAN : v == -INFINITY ? 0.f : ex2((v - M) * kLog2e);
                            }
                            const int n = min(32, c_last - c0 + 1);
                            for (int j0 = 0; j0 < n; j0 += 16) {
                                float4 x[16];
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const float* src =
                                        P.part_o + part_row(c0 + min(j0 + j, n - 1)) * D + lane * DPL;
                                    if constexpr (DPL == 4) {
                                        x[j] = __ldcg(reinterpret_cast<const float4*>(src));
                                    } else {
                                        const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
                                        x[j] = make_float4(y.x, y.y, 0.f, 0.f);
                                    }
                                }
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const float w = __shfl_sync(0xffffffffu, f, (j0 + j) & 31);
                                    if (j0 + j >= n || w == 0.f) continue;
                                    den += w;
                                    acc[0] = fmaf(w, x[j].x, acc[0]);
                                    acc[1] = fmaf(w, x[j].y, acc[1]);
                                    if constexpr (DPL == 4) {
                                        acc[2] = fmaf(w, x[j].z, acc[2]);
                                        acc[3] = fmaf(w, x[j].w, acc[3]);
                                    }
                                }
                            }
                        }
                        const bool none = den == 0.f;
                        const float inv = none ? 0.f : 1.f / den;
                        const int64_t row = (int64_t)(u.row0 + (r0 + r) / g.G) * g.Hq + u.hk * g.G + (r0 + r) % g.G;
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
        if (R == 0 || sh.t1 <= sh.t0) __syncthreads();   // all have read this unit's Q rows
        u = nu;
    }
    cp_async_wait<0>();
}

template <int D, int NT, int RB = 1>
cudaError_t launch_mx4(const Mx4Params& P, int grid, cudaStream_t stream) {
    using Cfg = Mx4Cfg<D, NT>;
    const cudaError_t e = allow_smem<decode_mx4_kernel<D, NT, RB>>(Cfg::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(decode_mx4_kernel<D, NT, RB>, dim3(grid), dim3(Cfg::kThreads), Cfg::kSmem,
                            stream, P);
}

}  // namespace

// CTAs of an SM that the variant for `nt` row tiles is built for.
int mx4_ctas_per_sm(int D, int nt) {
    return D == 128 ? (nt == 1 ? Mx4Cfg<128, 1>::kCtas : nt == 2 ? Mx4Cfg<128, 2>::kCtas
                       : nt == 3 ? Mx4Cfg<128, 3>::kCtas : Mx4Cfg<128, 2>::kCtas)
                    : (nt == 1 ? Mx4Cfg<64, 1>::kCtas : nt == 2 ? Mx4Cfg<64, 2>::kCtas
                       : Mx4Cfg<64, 4>::kCtas);
}

// Row tiles (of 8) that are built: what holds `rows`, -1 if none.
int mx4_row_tiles(int D, int rows) {
    const int most = D == 128 ? 32 : 64;
    if (rows > most) return -1;
    if (D == 128) return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 4 : 8;
}

cudaError_t launch_decode_mx4(const CacheGeom& g, int nt, const void* q, const void* k,
                              const void* ks, const void* v, const void* vs, const int32_t* table,
                              const int32_t* ctx, const int32_t* ql, int32_t* header,
                              int32_t* done, float* part_o, float* part_lse, void* out, float* lse,
                              int unit_cost, int grid, cudaStream_t stream) {
    Mx4Params P;
    P.g = g;
    P.q = (const __nv_bfloat16*)q;
    P.k = (const uint8_t*)k;
    P.ks = (const uint8_t*)ks;
    P.v = (const uint8_t*)v;
    P.vs = (const uint8_t*)vs;
    P.table = table;
    P.ctx = ctx;
    P.ql = ql;
    P.header = header;
    P.done = done;
    P.part_o = part_o;
    P.part_lse = part_lse;
    P.out = (__nv_bfloat16*)out;
    P.lse = lse;
    P.unit_cost = unit_cost;
    if (g.D == 128) {
        switch (nt) {
            case 1: return launch_mx4<128, 1>(P, grid, stream);
            case 2: return launch_mx4<128, 2>(P, grid, stream);
            case 3: return launch_mx4<128, 3>(P, grid, stream);
            // (32 rows at a time spill: 64 sequences 288 us, two blocks of 16 260)
            case 4: return launch_mx4<128, 2, 2>(P, grid, stream);
        }
    } else {
        switch (nt) {
            case 1: return launch_mx4<64, 1>(P, grid, stream);
            case 2: return launch_mx4<64, 2>(P, grid, stream);
            case 4: return launch_mx4<64, 4>(P, grid, stream);
            // (64 rows at a time spill: 64 sequences 497 us, two blocks of 32 307)
            case 8: return launch_mx4<64, 4, 2>(P, grid, stream);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
