// pa_key_weights_tc.cu -- pa_key_weights for many query rows, on tcgen05:
//     w_j += sum_r exp2(f q_r . k_j - lse_r log2 e).
//
// The scores of 256 keys (two accumulators of 128) by up to 128 query rows are
// computed transposed, keys as the rows of the product.  A key is then a lane
// of tensor memory: one thread sums all its exponentials, over all chunks of
// query rows, with no exchange between threads and no sum over keys to join.
// K stays in shared memory for all rows of an item; Q comes in chunks of 128
// rows, and stays from item to item where a head's rows fit in one chunk.
//
// Roles (21 warps): 8 take the accumulators (two groups of four, one for each
// 128 keys), 8 bring K (bf16 by cp.async; 4-bit codes through registers, as
// bf16 values), 4 bring Q, 1 issues the products.  All waits are bounded.
#include <mutex>

#include "pa_cache_mma.cuh"

namespace pa {

namespace {

constexpr int kTileKeys = 256, kChunk = 128;
constexpr int kEpiWarps = 8, kKWarps = 8, kQWarps = 4;
constexpr int kThreads = 32 * (kEpiWarps + kKWarps + kQWarps + 1);
constexpr int kQRing = 4;       // of row offsets, positions and full barriers (Q itself has 2)

struct ManyParams {
    CacheGeom g;
    const uint8_t* q;
    const uint8_t* k;
    const uint8_t* ks;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* ql;
    const float* lse;
    float* weights;
    int32_t* err;
};

template <int D>
struct ManySmem {
    static constexpr int kKBlock = kTileKeys * 128;     // 64 columns of K
    static constexpr int kQBlock = kChunk * 128;
    static constexpr int kK = 0;                        // two slots
    static constexpr int kQ = kK + 2 * (D / 64) * kKBlock;
    static constexpr int kOff = kQ + 2 * (D / 64) * kQBlock;
    static constexpr int kPos = kOff + kQRing * kChunk * 4;
    static constexpr int kBlind = kPos + kQRing * kChunk * 4;
    static constexpr int kBars = kBlind + kQRing * kQWarps * 4;
    static constexpr int kNumBars = 2 + 2 + kQRing + 2 + 4 + 4 + 1;
    static constexpr int kTmem = kBars + 8 * kNumBars;
    static constexpr int kBytes = kTmem + 16 + 1024;    // and the alignment of the slots
};

// Keys of a sequence: the first (a multiple of 32), how many tiles, and the
// chunks of its query rows.
__device__ __forceinline__ int many_tiles(const CacheGeom& g, int c, int q, int& first) {
    first = 0;
    if (q <= 0 || !good_lens(g, q, c)) return 0;
    first = window_first_tile(g.window, c - q, 32) * 32;
    return (c - first + kTileKeys - 1) / kTileKeys;
}
__device__ __forceinline__ int many_chunks(const CacheGeom& g, int q) {
    return (g.G * q + kChunk - 1) / kChunk;
}

// The CTA's items -- (sequence, KV head, tile of keys) -- in order.  Their cost
// is their chunks of rows; an item belongs to the CTA in whose share of the
// line it starts.
struct Walk {
    int64_t at, end;           // position of the item, end of the CTA's share
    int b, hk, tile, n, c, q, first, row0;
    bool same;                 // the item before had the same rows, in one chunk

    __device__ __forceinline__ bool more() const { return at < end; }
    __device__ __forceinline__ void read(const ManyParams& P) {
        c = P.ctx[b];
        q = P.ql[b];
        n = many_tiles(P.g, c, q, first);
    }
    // the next sequence with items; false when there is none
    __device__ __forceinline__ bool next_seq(const ManyParams& P) {
        do {
            row0 += clamp_q(P.g, q);
            if (++b >= P.g.B) {
                at = end;
                return false;
            }
            read(P);
        } while (n == 0);
        hk = tile = 0;
        return true;
    }
    __device__ __forceinline__ void init(const ManyParams& P, int lane) {
        const CacheGeom& g = P.g;
        auto cost = [&](int x) -> int64_t {
            int f;
            const int q_ = P.ql[x];
            return (int64_t)g.Hkv * many_tiles(g, P.ctx[x], q_, f) * many_chunks(g, q_);
        };
        same = false;
        const int64_t total = flat_total(g.B, lane, cost);
        const int64_t N = gridDim.x;
        const int64_t lo = total * blockIdx.x / N;
        end = total * (blockIdx.x + 1) / N;
        at = end;
        if (lo >= end) return;
        int64_t start;
        b = flat_find(g.B, lane, lo, cost, [&](int x) { return clamp_q(g, P.ql[x]); }, start, row0);
        read(P);
        const int w = many_chunks(g, q);
        const int64_t item = (lo - start + w - 1) / w;
        at = start + item * w;
        if (item < (int64_t)g.Hkv * n) {
            hk = (int)(item / n);
            tile = (int)(item % n);
        } else if (at < end) {
            next_seq(P);
        }
    }
    __device__ __forceinline__ void advance(const ManyParams& P) {
        const int w = many_chunks(P.g, q);
        at += w;
        same = w == 1;
        if (++tile < n) return;
        tile = 0;
        same = false;
        if (++hk < P.g.Hkv) return;
        if (at < end) next_seq(P);
    }
    __device__ __forceinline__ int key0() const { return first + tile * kTileKeys; }
    // chunks of rows that see some key of the tile
    __device__ __forceinline__ int2 chunks(const CacheGeom& g) const {
        const int n_ = many_chunks(g, q), p0 = c - q;
        int lo = 0, hi = n_;
        if (key0() > p0) lo = (int)((int64_t)(key0() - p0) * g.G / kChunk);
        if (g.window > 0) {
            // the last query that sees the tile's last key
            const int64_t last = (int64_t)key0() + kTileKeys - 1 + g.window - 1 - p0;
            if (last < q - 1) hi = (int)((max(last, (int64_t)0) * g.G + g.G - 1) / kChunk) + 1;
        }
        return make_int2(lo, max(hi, lo + 1));
    }
};

// E2M1 codes times a power of two, as bf16, by byte look-up: the eight
// magnitudes times the scale are four bf16x2 products; their high and their
// low bytes are two tables of eight that PRMT indexes with four codes at once.
struct ScaledCodes {
    uint32_t lo0, lo1, hi0, hi1;
    __device__ __forceinline__ explicit ScaledCodes(uint32_t e) {
        const uint32_t s = e == 0 ? 0x0040u : e == 255 ? 0x7fc0u : e << 7;
        const uint32_t s2 = s | (s << 16);
        uint32_t v[4];
        const uint32_t mag[4] = {0x3f000000u, 0x3fc03f80u, 0x40404000u, 0x40c04080u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(mag[i]), "r"(s2));
        lo0 = prmt(v[0], v[1], 0x6420);
        hi0 = prmt(v[0], v[1], 0x7531);
        lo1 = prmt(v[2], v[3], 0x6420);
        hi1 = prmt(v[2], v[3], 0x7531);
    }
    // four codes (the low 16 bits of w) -> two words
    __device__ __forceinline__ void four(uint32_t w, uint32_t m, uint32_t& a, uint32_t& b) const {
        const uint32_t l = prmt(lo0, lo1, m), h = prmt(hi0, hi1, m);
        // a selector's top bit spreads the byte's sign: 0x80 becomes 0xff for
        // a negative code, whose bit 6 is the sign wanted in bit 7
        const uint32_t s = prmt(0x80808080u, 0x80808080u, w);
        const uint32_t hs = h | ((s << 1) & 0x80808080u);
        a = prmt(l, hs, 0x5140);
        b = prmt(l, hs, 0x7362);
    }
    __device__ __forceinline__ uint4 eight(uint32_t w) const {
        const uint32_t m = w & 0x77777777u;
        uint4 d;
        four(w, m, d.x, d.y);
        four(w >> 16, m >> 16, d.z, d.w);
        return d;
    }
};

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 ldg_once16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::64B.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_many_kernel(const __grid_constant__ ManyParams P) {
    using S = ManySmem<D>;
    constexpr int NB = D / 64;                  // blocks of 64 columns
    extern __shared__ uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    float* off = reinterpret_cast<float*>(smem + S::kOff);      // -lse log2 e
    int* pos = reinterpret_cast<int*>(smem + S::kPos);          // query position, -1: sees nothing
    int* blind = reinterpret_cast<int*>(smem + S::kBlind);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kBars);
    uint64_t* k_empty = k_full + 2;
    uint64_t* q_full = k_empty + 2;
    uint64_t* q_empty = q_full + kQRing;
    uint64_t* s_full = q_empty + 2;             // [buffer][half]
    uint64_t* s_empty = s_full + 4;
    uint64_t* done = s_empty + 4;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kTmem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const CacheGeom& g = P.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 32 * kKWarps);
            mbar_init(&k_empty[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < kQRing; ++i) mbar_init(&q_full[i], 32 * kQWarps);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 128);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    constexpr int kMmaWarp = kEpiWarps + kKWarps + kQWarps;
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (blockIdx.x == 0 && warp == 0) check_lens(g, P.ctx, P.ql, lane, P.err);
    Walk t;
    t.init(P, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // true, or the CTA gives up
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        if (mbar_wait_or_abort(bar, parity, kWaitLimitNs, abort_flag)) return true;
        *abort_flag = 1;
        flag_error(P.err, PA_DEV_WAIT_TIMEOUT);
        return false;
    };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait(bar, parity));
    };

    if (warp < kEpiWarps) {
        // ------------------------------------------------ exponentials and sums
        const int half = warp >> 2, quad = warp & 3;
        const int my = 128 * half + 32 * quad;          // of the tile's keys
        const float factor = g.sm_scale * kLog2e;
        const uint64_t factor2 = pair2(factor);
        auto page_of = [&](const Walk& x) -> int {
            const int key = x.key0() + my + lane;
            return key < x.c ? P.table[(int64_t)x.b * g.mpps + (key >> g.ps_shift)] : -1;
        };
        uint32_t fill = 0, n = 0;
        int page = t.more() ? page_of(t) : -1;
        bool ok = true;
        while (ok && t.more()) {
            Walk next = t;
            next.advance(P);
            const int next_page = next.more() ? page_of(next) : -1;
            const int tok = t.key0() + my, key = tok + lane, p0 = t.c - t.q;
            const bool there = t.key0() + 128 * half < t.c;
            const int R = g.G * t.q;
            const int2 ch = t.chunks(g);
            uint64_t sum0 = 0, sum1 = 0;
            if (!t.same) fill += 1;
            for (int k = ch.x; k < ch.y; ++k, ++n) {
                if (k > ch.x) fill += 1;
                const uint32_t f = fill - 1;
                const int nr = min(kChunk, R - k * kChunk);
                const int buf = n & 1;
                ok = warp_wait(&s_full[2 * buf + half], (n >> 1) & 1) &&
                     warp_wait(&q_full[f % kQRing], (f / kQRing) & 1);
                if (!ok) break;
                tc_fence_after();
                if (there) {
                    const float* of = off + (f % kQRing) * kChunk;
                    const int* ps = pos + (f % kQRing) * kChunk;
                    const int4 bl = *reinterpret_cast<const int4*>(blind + (f % kQRing) * kQWarps);
                    const int lo_pos = p0 + k * kChunk / g.G;
                    const int hi_pos = p0 + (k * kChunk + nr - 1) / g.G;
                    const bool clear = (bl.x | bl.y | bl.z | bl.w) == 0 && tok + 31 <= lo_pos &&
                                       (g.window == 0 || tok > hi_pos - g.window);
                    const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) +
                                         (uint32_t)(2 * half + buf) * kChunk;
                    for (int c0 = 0; c0 < nr; c0 += 32) {
                        float v[32];
                        tmem_ld32(acc + c0, v);
                        tmem_wait_ld();
                        reg_fence32(v);
                        if (clear && c0 + 32 <= nr) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const ulonglong2 o =
                                    *reinterpret_cast<const ulonglong2*>(of + c0 + i);
                                const float2 x = split2(fma2(make2(v[i], v[i + 1]), factor2, o.x));
                                const float2 y =
                                    split2(fma2(make2(v[i + 2], v[i + 3]), factor2, o.y));
                                sum0 = add2(sum0, make2(ex2(x.x), ex2(x.y)));
                                sum1 = add2(sum1, make2(ex2(y.x), ex2(y.y)));
                            }
                        } else {
                            float s = 0.f;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const int p = ps[c0 + i];
                                const float e = ex2(fmaf(v[i], factor, of[c0 + i]));
                                s += key > p || (g.window > 0 && key <= p - g.window) ? 0.f : e;
                            }
                            sum0 = add2(sum0, make2(s, 0.f));
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(&s_empty[2 * buf + half]);
            }
            if (ok && key < t.c && (uint32_t)page < (uint32_t)g.num_pages) {
                const float2 a = split2(sum0), b = split2(sum1);
                atomicAdd(P.weights + ((int64_t)page * g.Hkv + t.hk) * g.ps + (key & (g.ps - 1)),
                          (a.x + a.y) + (b.x + b.y));
            }
            t = next;
            page = next_page;
        }
    } else if (warp < kEpiWarps + kKWarps) {
        // ------------------------------------------------------------------- K
        constexpr int ROW = MX4 ? D / 2 : 2 * D;        // bytes of a key's row
        constexpr int CH = ROW / 16, RPI = 32 / CH, NI = 32 / RPI;
        constexpr int KB = D / 32;
        const int kw = warp - kEpiWarps;                // keys 32 kw .. 32 kw + 31
        const int page_rows = g.ps * g.Hkv;
        auto look_up = [&](const Walk& x) -> int2 {     // the pages of two runs of 16 keys
            const int32_t* row = P.table + (int64_t)x.b * g.mpps;
            const int key = x.key0() + 32 * kw;
            int2 p = make_int2(-1, -1);
            if (key < x.c) p.x = p.y = row[key >> g.ps_shift];
            if (g.ps == 16) p.y = key + 16 < x.c ? row[(key >> 4) + 1] : -1;
            return p;
        };
        const int c16 = lane % CH;                      // this lane's 16 bytes of a row
        // row r of the warp's 32: its index, or -1
        auto row_at = [&](const Walk& x, int2 p, int r) -> int64_t {
            const int key = x.key0() + 32 * kw;
            const int pg = r < 16 ? p.x : p.y;
            if (key + r >= x.c || (uint32_t)pg >= (uint32_t)g.num_pages) return -1;
            return (int64_t)pg * page_rows + (int64_t)((key + r) & (g.ps - 1)) * g.tok_rows +
                   (int64_t)x.hk * g.head_rows;
        };
        auto check_pages = [&](const Walk& x, int2 p) {
            const int left = x.c - (x.key0() + 32 * kw);
            if (lane == 0 && ((left > 0 && (uint32_t)p.x >= (uint32_t)g.num_pages) ||
                              (left > 16 && (uint32_t)p.y >= (uint32_t)g.num_pages)))
                flag_error(P.err, PA_DEV_BAD_PAGE);
        };
        int2 page = t.more() ? look_up(t) : make_int2(-1, -1);
        if constexpr (MX4) {
            uint4 code[2][NI];
            uint32_t scale[2][NI];
            auto load = [&](const Walk& x, int2 p, uint4* cd, uint32_t* sc) {
                check_pages(x, p);
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const int64_t row = row_at(x, p, j * RPI + lane / CH);
                    cd[j] = make_uint4(0, 0, 0, 0);
                    sc[j] = 127;
                    if (row >= 0) {
                        cd[j] = ldg_once16(P.k + row * ROW + c16 * 16);
                        sc[j] = P.ks[row * KB + c16];
                    }
                }
            };
            if (t.more()) load(t, page, code[0], scale[0]);
            uint32_t n = 0;
            bool ok = true;
            while (ok && t.more()) {
                Walk next = t;
                next.advance(P);
                if (next.more()) load(next, look_up(next), code[1], scale[1]);
                const int slot = n & 1;
                ok = wait(&k_empty[slot], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                const int kb = c16 >> 1, turn = c16 & 2;
                const uint32_t base = sbase + S::kK + (uint32_t)(slot * NB + kb) * S::kKBlock;
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const int r = 32 * kw + j * RPI + lane / CH;
                    const ScaledCodes tab(scale[0][j]);
                    uint4 w = code[0][j];
                    // the second block's lanes store in another order: no bank twice
                    if (turn) w = make_uint4(w.z, w.w, w.x, w.y);
                    const uint32_t at = base + r * 128;
                    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sts128(at + ((((c16 & 1) * 4 + (i ^ turn)) ^ (r & 7)) << 4),
                               tab.eight(word[i]));
                }
                fence_proxy_async_smem();
                mbar_arrive(&k_full[slot]);
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    code[0][j] = code[1][j];
                    scale[0][j] = scale[1][j];
                }
                t = next;
                ++n;
            }
        } else {
            uint64_t once;
            asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
            uint32_t n = 0;
            while (t.more()) {
                Walk next = t;
                next.advance(P);
                const int2 next_page = next.more() ? look_up(next) : make_int2(-1, -1);
                const int slot = n & 1;
                if (!wait(&k_empty[slot], ((n >> 1) & 1) ^ 1)) break;
                check_pages(t, page);
                const uint32_t base = sbase + S::kK + (uint32_t)(slot * NB + (c16 >> 3)) * S::kKBlock;
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const int rw = j * RPI + lane / CH, r = 32 * kw + rw;
                    const int64_t row = row_at(t, page, rw);
                    cp_async16(base + r * 128 + (((c16 & 7) ^ (r & 7)) << 4),
                               P.k + (row >= 0 ? row * ROW + c16 * 16 : 0), row >= 0 ? 16 : 0, once);
                }
                cp_async_commit();
                cp_async_wait<0>();
                fence_proxy_async_smem();
                mbar_arrive(&k_full[slot]);
                t = next;
                page = next_page;
                ++n;
            }
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------------- Q
        constexpr int CH = D / 8, RPI = 32 / CH;
        const int qw = warp - kEpiWarps - kKWarps;      // rows 32 qw .. 32 qw + 31 of a chunk
        const int c16 = lane % CH;
        uint64_t keep;
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
        uint32_t fill = 0;
        bool ok = true;
        while (ok && t.more()) {
            if (!t.same) {
                const int R = g.G * t.q, p0 = t.c - t.q;
                const int2 ch = t.chunks(g);
                const bool rows_ok = t.row0 + t.q <= g.total_q;
                for (int k = ch.x; k < ch.y; ++k, ++fill) {
                    const int slot = fill & 1, ring = fill % kQRing;
                    ok = warp_wait(&q_empty[slot], ((fill >> 1) & 1) ^ 1);
                    if (!ok) break;
                    const int r = k * kChunk + 32 * qw + lane;
                    const bool real = r < R && rows_ok;
                    const int tq = r / g.G;
                    const int64_t row =
                        real ? (int64_t)(t.row0 + tq) * g.Hq + t.hk * g.G + (r - tq * g.G) : -1;
                    const uint32_t base =
                        sbase + S::kQ + (uint32_t)(slot * NB + (c16 >> 3)) * S::kQBlock;
#pragma unroll 4
                    for (int j = 0; j < 32 / RPI; ++j) {
                        const int rw = j * RPI + lane / CH, rr = 32 * qw + rw;
                        const int64_t x = __shfl_sync(0xffffffffu, row, rw);
                        cp_async16(base + rr * 128 + (((c16 & 7) ^ (rr & 7)) << 4),
                                   P.q + (x >= 0 ? x * 2 * D + c16 * 16 : 0), x >= 0 ? 16 : 0, keep);
                    }
                    cp_async_commit();
                    const float l = real ? P.lse[row] : -INFINITY;
                    off[ring * kChunk + 32 * qw + lane] = -l * kLog2e;
                    pos[ring * kChunk + 32 * qw + lane] = l == -INFINITY ? -1 : p0 + tq;
                    // (rows behind the last are left out by their number)
                    const bool none = __any_sync(0xffffffffu, r < R && l == -INFINITY);
                    if (lane == 0) blind[ring * kQWarps + qw] = none;
                    cp_async_wait<0>();
                    fence_proxy_async_smem();
                    mbar_arrive(&q_full[ring]);
                }
            }
            t.advance(P);
        }
    } else if (lane == 0) {
        // ------------------------------------------------------------- products
        uint32_t fill = 0, n = 0, m = 0;
        bool ok = true;
        while (ok && t.more()) {
            Walk next = t;
            next.advance(P);
            const int R = g.G * t.q;
            const int2 ch = t.chunks(g);
            const bool keep = next.more() && next.same;     // these rows serve the next item too
            const uint32_t kbase = sbase + S::kK + (uint32_t)((m & 1) * NB) * S::kKBlock;
            const bool second = t.key0() + 128 < t.c;
            ok = wait(&k_full[m & 1], (m >> 1) & 1);
            for (int k = ch.x; ok && k < ch.y; ++k, ++n) {
                if (k > ch.x || !t.same) {
                    ok = wait(&q_full[fill % kQRing], (fill / kQRing) & 1);
                    if (!ok) break;
                    ++fill;
                }
                const uint32_t slot = (fill - 1) & 1;
                const uint32_t qbase = sbase + S::kQ + slot * NB * S::kQBlock;
                const int cols = (min(kChunk, R - k * kChunk) + 31) & ~31;
                const uint32_t idesc = idesc_bf16_f32(128, 0, false, false) | ((uint32_t)(cols >> 3) << 17);
                const int buf = n & 1;
                for (int half = 0; half < 2; ++half) {
                    ok = wait(&s_empty[2 * buf + half], ((n >> 1) & 1) ^ 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (half == 0 || second) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma_ss(tmem + (uint32_t)(2 * half + buf) * kChunk,
                                      smem_desc_sw128(kbase + (kk >> 2) * S::kKBlock +
                                                          half * 128 * 128 + (kk & 3) * 32,
                                                      0, 1024),
                                      smem_desc_sw128(qbase + (kk >> 2) * S::kQBlock + (kk & 3) * 32,
                                                      0, 1024),
                                      idesc, kk > 0);
                    }
                    tc_commit(&s_full[2 * buf + half]);
                }
                if (!ok) break;
                if (k + 1 < ch.y || !keep) tc_commit(&q_empty[slot]);
            }
            if (ok) tc_commit(&k_empty[m & 1]);
            t = next;
            ++m;
        }
        // every product has ended before tensor memory is given back
        tc_commit(done);
        mbar_wait(done, 0, kDrainLimitNs);
    }
    cp_async_wait<0>();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool MX4>
cudaError_t launch_many(const ManyParams& P, int sms, cudaStream_t stream) {
    auto kern = key_weights_many_kernel<D, MX4>;
    constexpr int smem = ManySmem<D>::kBytes;
    static_assert(smem <= 232448, "shared memory of an SM");
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev >= 64 || !ready[dev]) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            if (dev < 64) ready[dev] = true;
        }
    }
    kern<<<sms, kThreads, smem, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights_many(const CacheGeom& g, bool mx4, const void* q, const void* k,
                                    const void* ks, const int32_t* table, const int32_t* ctx,
                                    const int32_t* ql, const float* lse, float* weights,
                                    int32_t* err, int sms, cudaStream_t stream) {
    ManyParams P;
    P.g = g;
    P.q = (const uint8_t*)q;
    P.k = (const uint8_t*)k;
    P.ks = (const uint8_t*)ks;
    P.table = table;
    P.ctx = ctx;
    P.ql = ql;
    P.lse = lse;
    P.weights = weights;
    P.err = err;
    if (g.D == 128)
        return mx4 ? launch_many<128, true>(P, sms, stream) : launch_many<128, false>(P, sms, stream);
    return mx4 ? launch_many<64, true>(P, sms, stream) : launch_many<64, false>(P, sms, stream);
}

}  // namespace pa
