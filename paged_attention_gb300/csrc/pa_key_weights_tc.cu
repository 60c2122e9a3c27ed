// pa_key_weights_tc.cu -- pa_key_weights for many query rows, on tcgen05:
//     w_j += sum_r exp2(f q_r . k_j - lse_r log2 e).
//
// The scores of 256 keys (two halves of 128) by up to 128 query rows are
// computed transposed, keys as the rows of the product.  A key is then a lane
// of tensor memory: one thread sums all its exponentials, over all chunks of
// query rows, with no exchange between threads and no sum over keys to join.
// 4-bit keys are turned into bf16 values by the thread that holds their lane,
// which stores them into tensor memory: the product then reads only Q from
// shared memory (whose bandwidth bound it with both operands there).  bf16 keys
// stay in shared memory.  Q comes in chunks of 128 rows, and stays from item to
// item where a head's rows fit in one chunk.
//
// Roles: two groups of 4 warps take the accumulators, one group for each half;
// two groups of 4 bring K, 2 warps bring Q, 2 issue the products.  All waits
// are bounded.
//
// 8 prompts of 4096 .. 16384 keys, 8 heads, 128 rows: 36 us 4-bit (80 on mma.sync,
// 41 with both operands in shared memory), of which 9 are the tensor cores', 7 the
// exponentials'; the conversion of K and the steps between the roles set the pace,
// about 2 us for 256 keys by 128 rows.  With 512 rows it is 1.5 us.
#include <type_traits>

#include "pa_cache_mma.cuh"

namespace pa {

namespace {

constexpr int kTileKeys = 256, kChunk = 128;
constexpr int kEpiWarps = 8, kKWarps = 8, kQWarps = 2;
constexpr int kMmaWarp = kEpiWarps + kKWarps + kQWarps;
constexpr int kThreads = 32 * (kMmaWarp + 2);
constexpr int kAccs = 3;        // accumulators of 128 x 128, taken in turn
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
    // Test hook: CTA 0 never announces item `skip` of half 0 (-1: none), and waits
    // are shorter.
    int32_t skip;
    uint64_t wait_limit_ns;
};

template <int D, bool MX4>
struct ManySmem {
    static constexpr int kKBlock = 128 * 128;           // 128 keys, 64 columns of K
    static constexpr int kQBlock = kChunk * 128;
    static constexpr int kSlots = MX4 ? 1 : 2;          // of a half of K
    static constexpr int kHalf = (D / 64) * kKBlock;
    // bf16: K's slots [slot][half]; 4-bit: each K warp's ring of places for 32
    // keys' rows and scale words
    static constexpr int kRing = 3, kPlace = 32 * (D / 2 + 4);
    static constexpr int kK = 0;
    static constexpr int kQ = kK + (MX4 ? (kKWarps * kRing * kPlace + 1023) / 1024 * 1024
                                        : kSlots * 2 * kHalf);
    static constexpr int kOff = kQ + 2 * (D / 64) * kQBlock;
    static constexpr int kPos = kOff + kQRing * kChunk * 4;
    static constexpr int kBlind = kPos + kQRing * kChunk * 4;
    static constexpr int kBars = kBlind + kQRing * 16;
    static constexpr int kNumBars = 4 + 4 + kQRing + 2 + 4 * kAccs + 1;
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
// line it starts.  Within the tiles of one head, the next item is a matter of
// two additions: every role walks the items by itself, many of them in a single
// thread or warp, where each instruction costs its latency.
struct Walk {
    int left;                  // items of this head that are the CTA's, this one included
    int key0;                  // first key of the tile
    int nch;                   // chunks of the head's rows
    bool same;                 // the item before had the same rows, in one chunk
    int b, hk, c, q, row0;
    int64_t at, end;           // position behind the items of this head; end of the share

    __device__ __forceinline__ bool more() const { return left > 0; }
    // enter a head at one of its n tiles, whose position is `at`
    __device__ __forceinline__ void enter(int tile, int n, int first) {
        const int64_t mine = (end - at + nch - 1) / nch;
        left = (int)min((int64_t)(n - tile), mine);
        key0 = first + tile * kTileKeys;
        at += (int64_t)left * nch;
        same = false;
    }
    // the next head with items of this CTA
    __device__ __forceinline__ void next_head(const ManyParams& P) {
        const CacheGeom& g = P.g;
        left = 0;
        if (at >= end) return;
        if (++hk == g.Hkv) {
            hk = 0;
            do {
                row0 += clamp_q(g, q);
                if (++b >= g.B) return;
                c = P.ctx[b];
                q = P.ql[b];
                int f;
                nch = many_tiles(g, c, q, f);
            } while (nch == 0);
        }
        int first;
        const int n = many_tiles(g, c, q, first);
        nch = many_chunks(g, q);
        enter(0, n, first);
    }
    __device__ __forceinline__ void init(const ManyParams& P, int lane) {
        const CacheGeom& g = P.g;
        auto cost = [&](int x) -> int64_t {
            int f;
            const int q_ = P.ql[x];
            return (int64_t)g.Hkv * many_tiles(g, P.ctx[x], q_, f) * many_chunks(g, q_);
        };
        left = 0;
        same = false;
        const int64_t total = flat_total(g.B, lane, cost);
        const int64_t N = gridDim.x;
        at = total * blockIdx.x / N;
        end = total * (blockIdx.x + 1) / N;
        if (at >= end) return;
        int64_t start;
        b = flat_find(g.B, lane, at, cost, [&](int x) { return clamp_q(g, P.ql[x]); }, start, row0);
        c = P.ctx[b];
        q = P.ql[b];
        int first;
        const int n = many_tiles(g, c, q, first);
        nch = many_chunks(g, q);
        const int64_t item = (at - start + nch - 1) / nch;
        at = start + item * nch;
        hk = (int)(item / n);
        if (at >= end) return;
        if (hk < g.Hkv) {
            enter((int)(item % n), n, first);
        } else {
            hk = g.Hkv - 1;
            next_head(P);
        }
    }
    __device__ __forceinline__ void advance(const ManyParams& P) {
        key0 += kTileKeys;
        same = nch == 1;
        if (--left == 0) next_head(P);
    }
    // chunks of rows that see some key of the tile
    __device__ __forceinline__ int2 chunks(const CacheGeom& g) const {
        int lo = 0, hi = nch;
        if (nch > 1) {
            const int p0 = c - q;
            if (key0 > p0) lo = (int)((int64_t)(key0 - p0) * g.G / kChunk);
            if (g.window > 0) {
                // the last query that sees the tile's last key
                const int64_t last = (int64_t)key0 + kTileKeys - 1 + g.window - 1 - p0;
                if (last < q - 1) hi = (int)((max(last, (int64_t)0) * g.G + g.G - 1) / kChunk) + 1;
            }
            hi = max(hi, lo + 1);
        }
        return make_int2(lo, hi);
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

template <int D, bool MX4>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_many_kernel(const __grid_constant__ ManyParams P) {
    using S = ManySmem<D, MX4>;
    constexpr int NB = D / 64;                  // blocks of 64 columns
    extern __shared__ uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    float* off = reinterpret_cast<float*>(smem + S::kOff);      // -lse log2 e
    int* pos = reinterpret_cast<int*>(smem + S::kPos);          // query position, -1: sees nothing
    int* blind = reinterpret_cast<int*>(smem + S::kBlind);      // of 32 rows each
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + S::kBars);    // [slot][half]
    uint64_t* k_empty = k_full + 4;
    uint64_t* q_full = k_empty + 4;
    uint64_t* q_empty = q_full + kQRing;
    uint64_t* s_full = q_empty + 2;
    uint64_t* s_empty = s_full + 2 * kAccs;                             // [half][accumulator]
    uint64_t* done = s_empty + 2 * kAccs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kTmem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const CacheGeom& g = P.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&k_full[i], 128);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&q_empty[i], 2);
        for (int i = 0; i < kQRing; ++i) mbar_init(&q_full[i], 32 * kQWarps);
        for (int i = 0; i < 2 * kAccs; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 128);
        }
        mbar_init(done, 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
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
    constexpr uint32_t kKCol = kAccs * kChunk;  // 4-bit: columns of K's halves, D / 2 each

    // true, or the CTA gives up
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        if (mbar_wait_or_abort(bar, parity, P.wait_limit_ns, abort_flag)) return true;
        *abort_flag = 1;
        flag_error(P.err, PA_DEV_WAIT_TIMEOUT);
        return false;
    };
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait(bar, parity));
    };

    if (warp < kEpiWarps) {
        // ------------------------------------------------ exponentials and sums
        // Group grp has half grp of every tile; the product of chunk n of all
        // is in accumulator (2 n + half) % kAccs, after the other half's of
        // chunk n - 2 + half.  (Barriers of their own for the halves: their
        // order in time is not fixed.)
        const int grp = warp >> 2, quad = warp & 3;
        const int my = 128 * grp + 32 * quad;
        const float factor = g.sm_scale * kLog2e;
        const uint64_t factor2 = pair2(factor);
        uint32_t fill = 0, n = 0;
        bool ok = true;
        for (; ok && t.more(); t.advance(P)) {
            const int tok = t.key0 + my, key = tok + lane, p0 = t.c - t.q;
            const bool there = t.key0 + 128 * grp < t.c;
            const int page =
                key < t.c ? P.table[(int64_t)t.b * g.mpps + (key >> g.ps_shift)] : -1;
            const int R = g.G * t.q;
            const int2 ch = t.chunks(g);
            uint64_t sum0 = 0, sum1 = 0;
            if (!t.same) fill += 1;
            for (int k = ch.x; k < ch.y; ++k, ++n) {
                if (k > ch.x) fill += 1;
                const uint32_t ring = (fill - 1) % kQRing, buf = (2 * n + grp) % kAccs;
                const int nr = min(kChunk, R - k * kChunk);
                ok = warp_wait(&s_full[grp * kAccs + buf], (n / kAccs) & 1) &&
                     warp_wait(&q_full[ring], ((fill - 1) / kQRing) & 1);
                if (!ok) break;
                tc_fence_after();
                const float* of = off + ring * kChunk;
                const int* ps = pos + ring * kChunk;
                const int4 bl = *reinterpret_cast<const int4*>(blind + ring * 4);
                // all of the chunk's queries see all of the warp's keys
                const bool clear = (bl.x | bl.y | bl.z | bl.w) == 0 &&
                                   (tok + 31 <= p0 || tok + 31 <= p0 + k * kChunk / g.G) &&
                                   (g.window == 0 ||
                                    tok > p0 + (k * kChunk + nr - 1) / g.G - g.window);
                const uint32_t acc = tmem + ((uint32_t)(32 * quad) << 16) + buf * kChunk;
                if (there) {
#pragma unroll 1
                    for (int c0 = 0; c0 < nr; c0 += 32) {
                        float v[32];
                        tmem_ld32(acc + c0, v);
                        tmem_wait_ld();
                        reg_fence32(v);
                        // (columns behind the last row are left out, not multiplied
                        // by nothing: their scores can be NaN)
                        auto take = [&](auto whole) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const ulonglong2 o =
                                    *reinterpret_cast<const ulonglong2*>(of + c0 + i);
                                const float2 x = split2(fma2(make2(v[i], v[i + 1]), factor2, o.x));
                                const float2 y =
                                    split2(fma2(make2(v[i + 2], v[i + 3]), factor2, o.y));
                                float e[4] = {ex2(x.x), ex2(x.y), ex2(y.x), ex2(y.y)};
                                if constexpr (!decltype(whole)::value) {
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        if (c0 + i + j >= nr) e[j] = 0.f;
                                }
                                sum0 = add2(sum0, make2(e[0], e[1]));
                                sum1 = add2(sum1, make2(e[2], e[3]));
                            }
                        };
                        if (clear && c0 + 32 <= nr) {
                            take(std::true_type());
                        } else if (clear) {
                            take(std::false_type());
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
                mbar_arrive(&s_empty[grp * kAccs + buf]);
            }
            if (ok && key < t.c && (uint32_t)page < (uint32_t)g.num_pages) {
                const float2 a = split2(sum0), b = split2(sum1);
                atomicAdd(P.weights + ((int64_t)page * g.Hkv + t.hk) * g.ps + (key & (g.ps - 1)),
                          (a.x + a.y) + (b.x + b.y));
            }
        }
    } else if (warp < kEpiWarps + kKWarps) {
        // ------------------------------------------------------------------- K
        // Group grp brings half grp of every tile, a warp 32 keys of it.
        constexpr int ROW = MX4 ? D / 2 : 2 * D;        // bytes of a key's row
        constexpr int CH = ROW / 16, RPI = 32 / CH, NI = 32 / RPI;
        constexpr int KB = D / 32;
        const int grp = (warp - kEpiWarps) >> 2, quad = warp & 3;
        const int my = 128 * grp + 32 * quad;
        const int page_rows = g.ps * g.Hkv;
        const int c16 = lane % CH, lr = lane / CH;      // this lane's 16 bytes, and row of RPI
        uint64_t once;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        // the pages of the warp's two runs of 16 keys; -1: no keys
        auto look_up = [&](const Walk& x) -> int2 {
            const int32_t* row = P.table + (int64_t)x.b * g.mpps;
            const int key = x.key0 + my;
            int2 p = make_int2(-1, -1);
            if (key < x.c) p.x = p.y = row[key >> g.ps_shift];
            if (g.ps == 16) p.y = key + 16 < x.c ? row[(key >> 4) + 1] : -1;
            return p;
        };
        // The two runs' pages and first rows in them (a page's rows are fewer
        // than 2^23, their bytes than 2^32).  Keys that do not exist, or whose
        // page does not, get rows that do: their sums go nowhere.
        struct Runs {
            uint32_t page_a, page_b, row_a, row_b;
        };
        auto runs_of = [&](const Walk& x, int2 p) -> Runs {
            const int key = x.key0 + my, left = x.c - key;
            const bool oka = (uint32_t)p.x < (uint32_t)g.num_pages;
            const bool okb = (uint32_t)p.y < (uint32_t)g.num_pages;
            if (lane == 0 && ((left > 0 && !oka) || (left > 16 && !okb)))
                flag_error(P.err, PA_DEV_BAD_PAGE);
            const int head = x.hk * g.head_rows;
            Runs r;
            r.page_a = oka ? p.x : 0;
            r.page_b = okb ? p.y : 0;
            r.row_a = (key & (g.ps - 1)) * g.tok_rows + head;
            r.row_b = ((key + 16) & (g.ps - 1)) * g.tok_rows + head;
            return r;
        };
        const uint32_t page_bytes = (uint32_t)page_rows * ROW;
        auto at_row = [&](uint32_t pg, uint32_t row) -> const uint8_t* {
            return P.k + ((uint64_t)pg * page_bytes + row * ROW);
        };
        const uint32_t lane_off = (uint32_t)(lr * g.tok_rows) * ROW + c16 * 16;
        const uint32_t step = (uint32_t)(RPI * g.tok_rows) * ROW;
        const int skip = blockIdx.x == 0 && grp == 0 ? P.skip : -1;
        int2 page = t.more() ? look_up(t) : make_int2(-1, -1);
        if constexpr (MX4) {
            // Rows come into the warp's ring by cp.async, coalesced, and from
            // there to the lane that holds the key: 16 bytes of a row (4 words
            // of codes, one scale) become 16 words of tensor memory.
            const uint32_t ring =
                sbase + S::kK + (uint32_t)(warp - kEpiWarps) * S::kRing * S::kPlace;
            // where chunk c of row r goes: eight lanes of a load meet no bank twice
            auto chunk_at = [&](int r, int c) -> int {
                if constexpr (CH == 4) return c ^ ((r >> 1) & 3);
                else return c ^ ((r >> 2) & 1);
            };
            uint32_t put = 0, get = 0;
            Walk ahead = t;                             // the item to fetch
            auto fetch = [&]() {
                if (ahead.more()) {
                    const Runs r = runs_of(ahead, page);
                    const uint32_t place = ring + put * S::kPlace;
                    const uint8_t* ka = at_row(r.page_a, r.row_a) + lane_off;
                    const uint8_t* kb = at_row(r.page_b, r.row_b) + lane_off;
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        const int x = j * RPI + lr;
                        cp_async16(place + x * ROW + chunk_at(x, c16) * 16,
                                   (j * RPI < 16 ? ka : kb) + (j * RPI & 15) / RPI * step,
                                   16, once);
                    }
                    // (head_dim 64: the word that holds the key's two bytes)
                    const uint32_t row =
                        (lane < 16 ? r.row_a : r.row_b) + (lane & 15) * (uint32_t)g.tok_rows;
                    const uint64_t so = (uint64_t)(lane < 16 ? r.page_a : r.page_b) *
                                            ((uint32_t)page_rows * KB) + (row * KB & ~3u);
                    cp_async4(place + 32 * ROW + lane * 4, P.ks + so, 4, once);
                    ahead.advance(P);
                    if (ahead.more()) page = look_up(ahead);
                }
                cp_async_commit();
                put = put + 1 == S::kRing ? 0 : put + 1;
            };
            for (int i = 0; i < S::kRing - 1; ++i) fetch();
            const uint32_t dst = tmem + ((uint32_t)(32 * quad) << 16) + kKCol + grp * (D / 2);
            for (uint32_t n = 0; t.more(); ++n, t.advance(P)) {
                cp_async_wait<S::kRing - 2>();
                __syncwarp();
                fetch();
                const uint32_t place = ring + get * S::kPlace;
                get = get + 1 == S::kRing ? 0 : get + 1;
                uint32_t e;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(e) : "r"(place + 32 * ROW + lane * 4));
                if constexpr (D == 64) {
                    const int slot = (t.key0 + my + lane) & (g.ps - 1);
                    e >>= ((slot * g.tok_rows + t.hk * g.head_rows) & 1) * 16;
                }
                auto convert = [&](int c, uint32_t* out) {
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                 : "r"(place + lane * ROW + chunk_at(lane, c) * 16));
                    const ScaledCodes tab((e >> (8 * c)) & 255u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 v = tab.eight(w[i]);
                        out[4 * i] = v.x;
                        out[4 * i + 1] = v.y;
                        out[4 * i + 2] = v.z;
                        out[4 * i + 3] = v.w;
                    }
                };
                // all but the last chunk while the item before is still in use
                uint32_t out[CH - 1][16];
#pragma unroll
                for (int c = 0; c < CH - 1; ++c) convert(c, out[c]);
                if (!warp_wait(&k_empty[grp], (n & 1) ^ 1)) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < CH - 1; ++c) tmem_st16(dst + 16 * c, out[c]);
                convert(CH - 1, out[0]);
                tmem_st16(dst + 16 * (CH - 1), out[0]);
                tmem_wait_st();
                tc_fence_before();
                if ((int)n != skip) mbar_arrive(&k_full[grp]);
            }
        } else {
            for (uint32_t n = 0; t.more(); ++n) {
                const uint32_t slot = n & 1;
                const Runs r = runs_of(t, page);
                t.advance(P);
                if (t.more()) page = look_up(t);
                if (!warp_wait(&k_empty[2 * slot + grp], ((n >> 1) & 1) ^ 1)) break;
                const uint32_t dst =
                    sbase + S::kK + (uint32_t)((2 * slot + grp) * NB + (c16 >> 3)) * S::kKBlock;
                const uint8_t* ka = at_row(r.page_a, r.row_a) + lane_off;
                const uint8_t* kb = at_row(r.page_b, r.row_b) + lane_off;
#pragma unroll 8
                for (int j = 0; j < NI; ++j) {
                    const int y = 32 * quad + j * RPI + lr;
                    cp_async16(dst + y * 128 + (((c16 & 7) ^ (y & 7)) << 4),
                               (j * RPI < 16 ? ka : kb) + (j * RPI & 15) / RPI * step,
                               16, once);
                }
                cp_async_commit();
                cp_async_wait<0>();
                fence_proxy_async_smem();
                if ((int)n != skip) mbar_arrive(&k_full[2 * slot + grp]);
            }
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------------- Q
        constexpr int CH = D / 8, RPI = 32 / CH;
        const int qw = warp - kEpiWarps - kKWarps;
        const int c16 = lane % CH;
        uint64_t keep;
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
        uint32_t fill = 0;
        bool ok = true;
        for (; ok && t.more(); t.advance(P)) {
            if (t.same) continue;
            const int R = g.G * t.q, p0 = t.c - t.q;
            const int2 ch = t.chunks(g);
            const bool rows_ok = t.row0 + t.q <= g.total_q;
            for (int k = ch.x; k < ch.y; ++k, ++fill) {
                const int slot = fill & 1, ring = fill % kQRing;
                ok = warp_wait(&q_empty[slot], ((fill >> 1) & 1) ^ 1);
                if (!ok) break;
                const uint32_t base = sbase + S::kQ + (uint32_t)(slot * NB + (c16 >> 3)) * S::kQBlock;
                constexpr int kParts = kChunk / 32 / kQWarps;   // of 32 rows, a warp
                int64_t row[kParts];
                float l[kParts];
                int tq[kParts];
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const int r = k * kChunk + 32 * (qw * kParts + i) + lane;
                    const bool real = r < R && rows_ok;
                    tq[i] = r / g.G;
                    row[i] = real ? (int64_t)(t.row0 + tq[i]) * g.Hq + t.hk * g.G + (r - tq[i] * g.G)
                                  : -1;
                    l[i] = real ? P.lse[row[i]] : -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < kParts; ++i)
#pragma unroll 4
                    for (int j = 0; j < 32 / RPI; ++j) {
                        const int rw = j * RPI + lane / CH, rr = 32 * (qw * kParts + i) + rw;
                        const int64_t x = __shfl_sync(0xffffffffu, row[i], rw);
                        cp_async16(base + rr * 128 + (((c16 & 7) ^ (rr & 7)) << 4),
                                   P.q + (x >= 0 ? x * 2 * D + c16 * 16 : 0), x >= 0 ? 16 : 0, keep);
                    }
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const int r = 32 * (qw * kParts + i) + lane;
                    off[ring * kChunk + r] = -l[i] * kLog2e;
                    pos[ring * kChunk + r] = l[i] == -INFINITY ? -1 : p0 + tq[i];
                    // (rows behind the last are left out by their number)
                    const bool none =
                        __any_sync(0xffffffffu, k * kChunk + r < R && l[i] == -INFINITY);
                    if (lane == 0) blind[ring * 4 + qw * kParts + i] = none;
                }
                cp_async_commit();
                cp_async_wait<0>();
                fence_proxy_async_smem();
                mbar_arrive(&q_full[ring]);
            }
        }
    } else if (lane == 0) {
        // ------------------------------------------------------------- products
        // One thread for each half: what lies between its products (waits,
        // commits, the next item) is as long as the products.
        // shared-memory descriptors: rows of 128 bytes with the 128-byte swizzle
        const int half = warp - kMmaWarp;
        const uint64_t kdesc =
            smem_desc_sw128(sbase + S::kK, 0, 1024) + half * (S::kHalf >> 4);
        const uint64_t qdesc = smem_desc_sw128(sbase + S::kQ, 0, 1024);
        const uint32_t ktmem = tmem + kKCol + half * (D / 2);
        uint32_t fill = 0, m = 0, n = 0;
        bool ok = true;
        for (; ok && t.more(); ++m) {
            const int R = g.G * t.q;
            const int2 ch = t.chunks(g);
            const bool same = t.same, there = t.key0 + 128 * half < t.c;
            t.advance(P);
            const bool keep = t.more() && t.same;     // these rows serve the next item too
            const uint32_t kslot = m % S::kSlots;
            const uint64_t kd = kdesc + kslot * (2 * S::kHalf >> 4);
            ok = wait(&k_full[2 * kslot + half], (m / S::kSlots) & 1);
            for (int k = ch.x; ok && k < ch.y; ++k, ++n) {
                if (k > ch.x || !same) {
                    ok = wait(&q_full[fill % kQRing], (fill / kQRing) & 1);
                    if (!ok) break;
                    ++fill;
                }
                const uint32_t qslot = (fill - 1) & 1;
                const uint64_t qd = qdesc + qslot * (NB * S::kQBlock >> 4);
                const int cols = (min(kChunk, R - k * kChunk) + 15) & ~15;
                const uint32_t idesc =
                    idesc_bf16_f32(128, 0, false, false) | ((uint32_t)(cols >> 3) << 17);
                const uint32_t buf = (2 * n + half) % kAccs, before = n - 2 + half;
                if (n + half >= 2) ok = wait(&s_empty[(half ^ 1) * kAccs + buf], (before / kAccs) & 1);
                if (!ok) break;
                tc_fence_after();
                if (there) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t q = qd + (((kk >> 2) * S::kQBlock + (kk & 3) * 32) >> 4);
                        if constexpr (MX4)
                            tc_mma_ts(tmem + buf * kChunk, ktmem + kk * 8, q, idesc, kk > 0);
                        else
                            tc_mma_ss(tmem + buf * kChunk,
                                      kd + (((kk >> 2) * S::kKBlock + (kk & 3) * 32) >> 4), q,
                                      idesc, kk > 0);
                    }
                }
                tc_commit(&s_full[half * kAccs + buf]);
                if (k + 1 == ch.y) tc_commit(&k_empty[2 * kslot + half]);
                if (k + 1 < ch.y || !keep) tc_commit(&q_empty[qslot]);
            }
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
    constexpr int smem = ManySmem<D, MX4>::kBytes;
    static_assert(smem <= 232448, "shared memory of an SM");
    const cudaError_t e = allow_smem<key_weights_many_kernel<D, MX4>>(smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(sms), dim3(kThreads), smem, stream, P);
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
    take_test_hook(&P.skip, &P.wait_limit_ns);
    if (g.D == 128)
        return mx4 ? launch_many<128, true>(P, sms, stream) : launch_many<128, false>(P, sms, stream);
    return mx4 ? launch_many<64, true>(P, sms, stream) : launch_many<64, false>(P, sms, stream);
}

}  // namespace pa
