// pa_decode_mx4.cu -- decode attention over a PA_MX4 (4-bit) paged cache.
//
//   S^T = K Q^T,  P = exp2(S^T - m),  O^T += V^T P,  per KV head and sequence
//
// One persistent CTA per SM takes an equal share of the flat line of (sequence,
// KV head, 64-token tile); its warps cut each unit's tokens between them in
// 32-token steps, every warp with its own running (m, l, O), its own ring of
// cp.async stages and no barrier until the unit ends.  Then the warps' states
// merge through shared memory; a unit that spans CTAs leaves normalised parts
// in the workspace, and the last CTA to finish one joins them.
//
// What bounds it: 17/16 D bytes a key and head from HBM (136 at D = 128, K and
// V), and the instructions that turn 4-bit codes into operands.  So:
//   - products are transposed (mma m16n8k16 with 16 keys, or 16 columns of V,
//     as rows): R query rows cost ceil(R/8) products, no half-empty tiles;
//   - the contraction order is free, so each lane takes the bytes of a row as
//     they lie: 4 bytes = 8 codes of one 32-block for K, 16 codes of one block
//     for V; codes become f16 pairs by one conversion each, exactly;
//   - K's block scales multiply the fp32 block scores (a block is two mma
//     steps), V's multiply the f16 codes, relative to the largest scale its
//     columns met so far (moved as rarely as the running max);
//   - the running max moves only when a score passes it by 2^8, decided by one
//     vote; a row's max is otherwise never reduced over lanes.
// Masked scores are -inf and V rows past the context are zero codes, so
// nothing outside a row's sight reaches it; a NaN block (scale 255) reaches
// exactly the rows that see its key.
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
    int32_t unit_cost;   // fixed cost of a unit, in tiles
};

template <int D, int NT>
struct Mx4Cfg {
    static constexpr int kWarps = 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = 4;
    static constexpr int kStep = 32;                       // tokens of a warp's step
    static constexpr int kRow = D / 2;                     // code bytes of a row
    static constexpr int kStage = 2 * kStep * (kRow + 4);  // K, V, their scale words
    static constexpr int kRows = 8 * NT;
    static constexpr int kQRow = 2 * D + kQPad;
    static constexpr int kMergeRow = D + 4;                // floats
    static constexpr int kMergeWarp = 8 * kMergeRow + 16;  // 8 rows, then m[8], l[8]
    static constexpr int kOffQ = kWarps * kStages * kStage;
    static constexpr int kOffInfo = kOffQ + kRows * kQRow;  // per row: score factor
    static constexpr int kOffMerge = kOffInfo + kRows * 4;
    static constexpr int kOffFlag = kOffMerge + kWarps * kMergeWarp * 4;
    static constexpr int kSmem = kOffFlag + 16;
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kOffQ % 16 == 0 && kOffMerge % 16 == 0, "alignment");
};

namespace {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

// A unit (sequence, KV head) as a CTA meets it.
struct Unit {
    int b, hk;
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
__device__ __forceinline__ bool next_unit(const Mx4Params& P, Unit& u) {
    u.start += P.unit_cost + u.n;
    if (++u.hk < P.g.Hkv) return true;
    u.hk = 0;
    do {
        u.row0 += clamp_q(P.g, u.ql);
        if (++u.b >= P.g.B) return false;
        load_seq(P, u);
    } while (u.n == 0);
    return true;
}

// The token steps of unit u that warp w of W runs, of the CTA's share [lo, hi)
// of the flat line: steps [s0, s1) of 32 tokens, counted from token `tok0`.
struct Share {
    int t0, t1;     // tiles of the unit in the CTA's share
    int s0, s1;
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
    s.s0 = (int)((int64_t)steps * w / W);
    s.s1 = (int)((int64_t)steps * (w + 1) / W);
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

template <int D, int NT>
__global__ void __launch_bounds__(Mx4Cfg<D, NT>::kThreads, 1)
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

    // ---- this CTA's share of the flat line
    auto seq_cost = [&](int b) -> int64_t {
        int first;
        const int n = seq_tiles(g, P.ctx[b], P.ql[b], first);
        return n > 0 ? (int64_t)g.Hkv * (n + cost) : 0;
    };
    const int64_t C = flat_total(g.B, lane, seq_cost);
    if (blockIdx.x == 0 && warp == 0) check_lens(g, P.ctx, P.ql, lane, P.header + H_ERROR);
    const int64_t N = min((int64_t)gridDim.x, C);
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
        u.hk = (int)((lo - start) / (u.n + cost));
        u.start = start + (int64_t)u.hk * (u.n + cost);
    }

    const uint32_t ring = smem_u32(smem) + warp * ST * Cfg::kStage;
    const uint32_t qbase = smem_u32(smem + Cfg::kOffQ);
    float* info = reinterpret_cast<float*>(smem + Cfg::kOffInfo);
    float* merge = reinterpret_cast<float*>(smem + Cfg::kOffMerge);
    volatile int* flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffFlag);

    // ---- the load side runs up to ST - 1 steps ahead, over unit boundaries
    Unit lu = u;
    Share ls = share_of(lu, cost, lo, hi, warp, W);
    bool more = true;
    int lstep = ls.s0;
    int win_lo = 0, win = -1, nxt = -1;      // 32 page ids, and the next 32
    bool win_ok = false;
    auto issue = [&](int stage) {
        while (more && lstep >= ls.s1) {
            if (!next_unit(P, lu) || lu.start >= hi) {
                more = false;
                break;
            }
            ls = share_of(lu, cost, lo, hi, warp, W);
            lstep = ls.s0;
            win_ok = false;
        }
        if (more) {
            const int tok = ls.tok0 + 32 * lstep++;
            const int npg = (lu.ctx + g.ps - 1) >> g.ps_shift;
            const int32_t* row = P.table + (int64_t)lu.b * g.mpps;
            const int p0 = tok >> g.ps_shift;
            if (!win_ok || p0 - win_lo >= 32) {
                auto id = [&](int p) { return p < npg ? row[p] : -1; };
                win = win_ok && p0 == win_lo + 32 ? nxt : id(p0 + lane);
                win_lo = p0;
                nxt = id(p0 + 32 + lane);
                win_ok = true;
            }
            const uint32_t dk = ring + stage * Cfg::kStage, dv = dk + 32 * ROW;
            const uint32_t dks = dv + 32 * ROW, dvs = dks + 128;
            constexpr int CH = ROW / 16, RPI = 32 / CH;   // chunks of a row, rows an instruction
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 32 / RPI; ++i) {
                const int r = i * RPI + lane / CH, c = lane % CH, t = tok + r;
                const int page = __shfl_sync(0xffffffffu, win, (t >> g.ps_shift) - win_lo);
                const bool in = t < lu.ctx, ok = in && page >= 0 && page < g.num_pages;
                bad |= in && !ok;
                const int64_t off =
                    ok ? row_of(g, page, t & (g.ps - 1), lu.hk) * ROW + c * 16 : 0;
                const uint32_t at = r * ROW + chunk_at<D>(r, c) * 16;
                cp_async16(dk + at, P.k + off, ok ? 16 : 0);
                cp_async16(dv + at, P.v + off, ok ? 16 : 0);
            }
            {   // one scale word per key (head_dim 64: the word that holds its two bytes)
                const int t = tok + lane;
                const int page = __shfl_sync(0xffffffffu, win, (t >> g.ps_shift) - win_lo);
                const bool ok = t < lu.ctx && page >= 0 && page < g.num_pages;
                const int64_t off = ok ? row_of(g, page, t & (g.ps - 1), lu.hk) * KB & ~(int64_t)3 : 0;
                cp_async4(dks + lane * 4, P.ks + off, ok ? 4 : 0);
                cp_async4(dvs + lane * 4, P.vs + off, ok ? 4 : 0);
            }
            if (__any_sync(0xffffffffu, bad) && lane == 0)
                flag_error(P.header + H_ERROR, PA_DEV_BAD_PAGE);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) issue(s);
    int stage = 0;

    // ---- units
    while (true) {
        const int R = g.G * u.ql;
        const int pbase = u.ctx - u.ql;
        const Share sh = share_of(u, cost, lo, hi, warp, W);
        const bool any_tile = sh.t1 > sh.t0;
        if (any_tile && u.row0 + u.ql <= g.total_q) {
            // Q rows as f16 with a power of two taken out of each: no element
            // leaves f16's range at the top, and what falls off the bottom is
            // 2^-25 of the row's largest
            for (int r = warp; r < Cfg::kRows; r += W) {
                float x[D / 32];
                float top = 0.f;
                if (r < R) {
                    const __nv_bfloat16* src =
                        P.q + ((int64_t)(u.row0 + r / g.G) * g.Hq + u.hk * g.G + r % g.G) * D;
#pragma unroll
                    for (int j = 0; j < D / 64; ++j) {
                        const uint32_t w = reinterpret_cast<const uint32_t*>(src)[lane + 32 * j];
                        x[2 * j] = __uint_as_float(w << 16);
                        x[2 * j + 1] = __uint_as_float(w & 0xffff0000u);
                        top = fmaxf(top, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) x[j] = 0.f;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                // exponent field of the largest, kept where both powers are normal
                const int e = max(8, min(247, (int)(__float_as_uint(top) >> 23)));
                const float down = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
                    *reinterpret_cast<uint32_t*>(smem + Cfg::kOffQ + r * Cfg::kQRow +
                                                 4 * (lane + 32 * j)) =
                        pack_f16x2(x[2 * j] * down, x[2 * j + 1] * down);
                if (lane == 0)
                    info[r] = __uint_as_float((uint32_t)e << 23) * (g.sm_scale * kLog2e);
            }
            __syncthreads();

            float m[NT][2], l[NT][2], fq[NT][2];
            int pr[NT][2];              // last visible position of the thread's rows
            float o[OT][NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * nt + 2 * t4 + e;
                    m[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                    fq[nt][e] = info[r];
                    pr[nt][e] = r < R ? pbase + r / g.G : -1;
                }
#pragma unroll
                for (int i = 0; i < OT; ++i)
                    o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
            }
            uint4 qf[NT <= 2 ? NT : 1][KB];
            if constexpr (NT <= 2) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
                        qf[nt][kb] =
                            lds128(qbase + (8 * nt + gr) * Cfg::kQRow + kb * 64 + t4 * 16);
            }
            int vref = -1000;           // exponent that V's codes are scaled against

            for (int step = sh.s0; step < sh.s1; ++step) {
                cp_async_wait<ST - 2>();
                __syncwarp();
                const int tok = sh.tok0 + 32 * step;
                const uint32_t sk = ring + stage * Cfg::kStage, sv = sk + 32 * ROW;
                const uint32_t sks = sv + 32 * ROW, svs = sks + 128;
                // head_dim 64: which half of its scale word a key's two bytes are
                auto scale_shift = [&](int key) -> int {
                    if constexpr (D == 128) return 0;
                    const int s = (tok + key) & (g.ps - 1);
                    return ((s * g.tok_rows + u.hk * g.head_rows) & 1) * 16;
                };

                // ---- scores of 2 x 16 keys
                float s[2][NT][4];
                uint32_t kw[2][2];
                bool nan_k = false;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int key = 16 * mt + 8 * hh + tile_key<D>(gr);
                        uint32_t w = lds32(sks + key * 4) >> scale_shift(key);
                        if (D == 64) w &= 0xffffu;
                        kw[mt][hh] = w;
                        nan_k |= (((w & 0x7f7f7f7fu) + 0x01010101u) & w & 0x80808080u) != 0;
                    }
                nan_k = __any_sync(0xffffffffu, nan_k);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const int key0 = 16 * mt + tile_key<D>(gr), key1 = key0 + 8;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        uint32_t a[2][4];
                        e2m1x8_to_f16(lds32(sk + key0 * ROW + chunk_at<D>(key0, kb) * 16 + t4 * 4),
                                      a[0][0], a[0][2], a[1][0], a[1][2]);
                        e2m1x8_to_f16(lds32(sk + key1 * ROW + chunk_at<D>(key1, kb) * 16 + t4 * 4),
                                      a[0][1], a[0][3], a[1][1], a[1][3]);
                        const uint32_t e0 = (kw[mt][0] >> (8 * kb)) & 255u;
                        const uint32_t e1 = (kw[mt][1] >> (8 * kb)) & 255u;
                        float f0 = __uint_as_float(e0 << 23), f1 = __uint_as_float(e1 << 23);
                        if (nan_k) {
                            f0 = e8m0_to_f32(e0);
                            f1 = e8m0_to_f32(e1);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint4 b;
                            if constexpr (NT <= 2)
                                b = qf[nt][kb];
                            else
                                b = lds128(qbase + (8 * nt + gr) * Cfg::kQRow + kb * 64 + t4 * 16);
                            float x[4];
                            mma_f16_first(x, a[0], b.x, b.y);
                            mma_f16_16816(x, a[1], b.z, b.w);
                            float* d = s[mt][nt];
                            if (kb == 0) {
                                d[0] = x[0] * f0;
                                d[1] = x[1] * f0;
                                d[2] = x[2] * f1;
                                d[3] = x[3] * f1;
                            } else {
                                d[0] = fmaf(x[0], f0, d[0]);
                                d[1] = fmaf(x[1], f0, d[1]);
                                d[2] = fmaf(x[2], f1, d[2]);
                                d[3] = fmaf(x[3], f1, d[3]);
                            }
                        }
                    }
                }
                // log2 domain, then the mask where a row does not see the whole step
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][nt][e] *= fq[nt][e & 1];
                const bool clear = tok + 31 <= pbase && (g.window == 0 || tok > u.ctx - 1 - g.window);
                if (!clear) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = tok + 16 * mt + 8 * (e >> 1) + tile_key<D>(gr);
                                const int p = pr[nt][e & 1];
                                if (j > p || (g.window > 0 && j <= p - g.window))
                                    s[mt][nt][e] = -INFINITY;
                            }
                }
                // ---- V's scale bytes of the thread's keys and columns
                uint32_t ve[2][4];
                int vtop = -1000;
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = 16 * mt + 8 * (e >> 1) + tile_key<D>(2 * t4 + (e & 1));
                        ve[mt][e] = lds8(svs + key * 4 + scale_shift(key) / 8 +
                                         (D == 128 ? gr / 2 : gr / 4));
                        vtop = max(vtop, (int)ve[mt][e]);
                    }
                // ---- move the running max and V's reference where they must
                bool move = vtop > vref + 4 || vtop == 255;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]),
                                              fmaxf(s[1][nt][e], s[1][nt][e + 2]));
                        move |= x > m[nt][e] + 8.f;
                    }
                bool nan_v = false;
                if (__any_sync(0xffffffffu, move)) {
                    int top = -1000;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            nan_v |= ve[mt][e] == 255u;
                            if (ve[mt][e] != 255u) top = max(top, (int)ve[mt][e]);
                        }
                    nan_v = __any_sync(0xffffffffu, nan_v);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    float vfac = 1.f;
                    if (top > vref) {
                        vfac = vref < 0 ? 0.f : ex2((float)(vref - top));
                        vref = top;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]),
                                            fmaxf(s[1][nt][e], s[1][nt][e + 2]));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                            float al = 1.f;
                            if (x > m[nt][e]) {
                                al = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - x);
                                m[nt][e] = x;
                            }
                            l[nt][e] *= al;
                            const float f = al * vfac;
#pragma unroll
                            for (int i = 0; i < OT; ++i) {
                                // a poisoned sum stays poisoned
                                o[i][nt][e] = o[i][nt][e] * f;
                                o[i][nt][e + 2] = o[i][nt][e + 2] * f;
                            }
                        }
                }
                // ---- probabilities, and their transposes as the B operand
                uint32_t pb[2][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float mu0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
                    const float mu1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const float p0 = ex2(s[mt][nt][0] - mu0), p1 = ex2(s[mt][nt][1] - mu1);
                        const float p2 = ex2(s[mt][nt][2] - mu0), p3 = ex2(s[mt][nt][3] - mu1);
                        l[nt][0] += p0 + p2;
                        l[nt][1] += p1 + p3;
                        pb[mt][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
                        pb[mt][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
                    }
                }
                // ---- O^T += V^T P
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    uint32_t sc[2];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        float f[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x = ve[mt][2 * hh + e];
                            f[e] = __uint_as_float((uint32_t)max(0, (int)x - vref + 127) << 23);
                            if (nan_v && x == 255u) f[e] = 0.f;
                        }
                        sc[hh] = pack_f16x2(f[0], f[1]);
                    }
                    uint32_t even[2][VW], odd[2][VW];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const int ka = 16 * mt + 8 * hh + tile_key<D>(2 * t4);
                        const int kb = 16 * mt + 8 * hh + tile_key<D>(2 * t4 + 1);
                        uint32_t wa[VW], wb[VW];
                        if constexpr (D == 128) {
                            const uint2 x = lds64(sv + ka * ROW + chunk_at<D>(ka, gr >> 1) * 16 +
                                                  (gr & 1) * 8);
                            const uint2 y = lds64(sv + kb * ROW + chunk_at<D>(kb, gr >> 1) * 16 +
                                                  (gr & 1) * 8);
                            wa[0] = x.x;
                            wa[VW - 1] = x.y;
                            wb[0] = y.x;
                            wb[VW - 1] = y.y;
                        } else {
                            wa[0] = lds32(sv + ka * ROW + chunk_at<D>(ka, gr >> 2) * 16 +
                                          (gr & 3) * 4);
                            wb[0] = lds32(sv + kb * ROW + chunk_at<D>(kb, gr >> 2) * 16 +
                                          (gr & 3) * 4);
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
                    for (int key = 0; key < 32; ++key) {
                        const int j = tok + key;
                        if (lds8(svs + key * 4 + scale_shift(key) / 8 +
                                 (D == 128 ? gr / 2 : gr / 4)) != 255u)
                            continue;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int p = pr[nt][e & 1];
                                if (j <= p && (g.window == 0 || j > p - g.window))
#pragma unroll
                                    for (int i = 0; i < OT; ++i) o[i][nt][e] = NAN;
                            }
                    }
                }
                __syncwarp();
                issue(stage == 0 ? ST - 1 : stage - 1);
                stage = stage + 1 == ST ? 0 : stage + 1;
            }

            // ---- merge the warps, eight rows at a time
            const float vmul = vref < 0 ? 0.f : e8m0_to_f32((uint32_t)vref);
            // the unit's CTAs, and whether it is split over several
            const int64_t first_pos = u.start + cost;
            const int c_first = (int)(((first_pos + 1) * N - 1) / C);
            const int c_last = (int)(((first_pos + u.n) * N - 1) / C);
            const int slot = c_first == c_last ? -1 : 2 * cta + (cta == c_first ? 1 : 0);
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
                            mw[8 * Cfg::kMergeRow + 2 * t4 + e] = sh.s1 > sh.s0 ? m[nt][e] : -INFINITY;
                            mw[8 * Cfg::kMergeRow + 8 + 2 * t4 + e] = x;
                        }
                        // the thread's columns are consecutive: OT pairs from gr * D / 8
                        float* row = mw + (2 * t4 + e) * Cfg::kMergeRow + gr * (D / 8);
#pragma unroll
                        for (int i = 0; i < OT; i += 2)
                            *reinterpret_cast<float4*>(row + 2 * i) =
                                make_float4(o[i][nt][e] * vmul, o[i][nt][e + 2] * vmul,
                                            o[i + 1][nt][e] * vmul, o[i + 1][nt][e + 2] * vmul);
                    }
                    __syncthreads();
                    const int r = 8 * nt + warp;   // 8 warps, 8 rows
                    if (r < R) {
                        constexpr int DPL = D / 32;
                        float M = -INFINITY;
#pragma unroll
                        for (int w = 0; w < W; ++w)
                            M = fmaxf(M, merge[w * Cfg::kMergeWarp + 8 * Cfg::kMergeRow + warp]);
                        float den = 0.f, acc[DPL];
#pragma unroll
                        for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            const float* b = merge + w * Cfg::kMergeWarp;
                            const float mv = b[8 * Cfg::kMergeRow + warp];
                            const float lv = b[8 * Cfg::kMergeRow + 8 + warp];
                            if (mv == -INFINITY && lv == 0.f) continue;   // saw nothing
                            const float f = mv == -INFINITY ? 1.f : ex2(mv - M);
                            den += f * lv;
#pragma unroll
                            for (int e = 0; e < DPL; ++e)
                                acc[e] += f * b[warp * Cfg::kMergeRow + lane * DPL + e];
                        }
                        // (a NaN sum is not "no visible key")
                        const bool none = den == 0.f;
                        const float inv = none ? 0.f : 1.f / den;
                        const float ln = none ? -INFINITY : (M == -INFINITY ? den : (M + lg2(den)) * kLn2);
                        if (slot < 0) {
                            const int64_t row = (int64_t)(u.row0 + r / g.G) * g.Hq + u.hk * g.G + r % g.G;
                            __nv_bfloat16* dst = P.out + row * D + lane * DPL;
#pragma unroll
                            for (int e = 0; e < DPL; e += 2)
                                *reinterpret_cast<uint32_t*>(dst + e) =
                                    pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
                            if (P.lse != nullptr && lane == 0) P.lse[row] = ln;
                        } else {
                            const int64_t row = (int64_t)slot * Cfg::kRows + r;
#pragma unroll
                            for (int e = 0; e < DPL; ++e)
                                P.part_o[row * D + lane * DPL + e] = acc[e] * inv;
                            if (lane == 0) P.part_lse[row] = ln;
                        }
                    }
                    __syncthreads();
                }
            }
            if (slot >= 0) {
                // the last of the unit's CTAs to come here joins the parts;
                // nobody waits for another CTA
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0)
                    *flag = atomicAdd(P.done + c_first, 1) == c_last - c_first ? 1 : 0;
                __syncthreads();
                if (*flag != 0) {
                    __threadfence();
                    constexpr int DPL = D / 32;
                    for (int r = warp; r < R; r += W) {
                        float M = -INFINITY;
                        bool poison = false;
                        for (int c = c_first; c <= c_last; ++c) {
                            const int64_t row = (int64_t)(2 * c + (c == c_first ? 1 : 0)) * Cfg::kRows + r;
                            const float v = __ldcg(P.part_lse + row);
                            poison |= v != v;
                            M = fmaxf(M, v);
                        }
                        float den = 0.f, acc[DPL];
#pragma unroll
                        for (int e = 0; e < DPL; ++e) acc[e] = 0.f;
                        for (int c = c_first; c <= c_last; ++c) {
                            const int64_t row = (int64_t)(2 * c + (c == c_first ? 1 : 0)) * Cfg::kRows + r;
                            const float v = __ldcg(P.part_lse + row);
                            if (v == -INFINITY) continue;
                            const float f = poison ? NAN : ex2((v - M) * kLog2e);
                            den += f;
#pragma unroll
                            for (int e = 0; e < DPL; ++e)
                                acc[e] += f * __ldcg(P.part_o + row * D + lane * DPL + e);
                        }
                        const bool none = den == 0.f;
                        const float inv = none ? 0.f : 1.f / den;
                        const int64_t row = (int64_t)(u.row0 + r / g.G) * g.Hq + u.hk * g.G + r % g.G;
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
        } else if (any_tile) {
            // rows past total_q_tokens (lengths that do not add up): their
            // steps are loaded but not computed
            for (int step = sh.s0; step < sh.s1; ++step) {
                cp_async_wait<ST - 2>();
                __syncwarp();
                issue(stage == 0 ? ST - 1 : stage - 1);
                stage = stage + 1 == ST ? 0 : stage + 1;
            }
        }
        if (!next_unit(P, u) || u.start >= hi) break;
    }
    cp_async_wait<0>();
}

template <int D, int NT>
cudaError_t launch_mx4(const Mx4Params& P, int grid, cudaStream_t stream) {
    using Cfg = Mx4Cfg<D, NT>;
    auto kern = decode_mx4_kernel<D, NT>;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<grid, Cfg::kThreads, Cfg::kSmem, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

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
            case 4: return launch_mx4<128, 4>(P, grid, stream);
        }
    } else {
        switch (nt) {
            case 1: return launch_mx4<64, 1>(P, grid, stream);
            case 2: return launch_mx4<64, 2>(P, grid, stream);
            case 4: return launch_mx4<64, 4>(P, grid, stream);
            case 8: return launch_mx4<64, 8>(P, grid, stream);
        }
    }
    return cudaErrorInvalidValue;
}

}  // namespace pa
