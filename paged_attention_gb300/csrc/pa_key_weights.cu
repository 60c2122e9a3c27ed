// pa_key_weights.cu -- adds to every cached key the softmax weight that a set
// of queries gives it:  w_j += sum_r exp2(f q_r . k_j - lse_r log2 e), over the
// rows r (query, q head of the key's group) that see key j.  This is the kernel
// for up to 16 such rows; pa_key_weights_tc.cu has the one for more.
//
// No sum runs over keys, so there is nothing to join: a warp owns 32 keys of one
// KV head at a time, copies their rows into its own shared memory (cp.async) and
// from there into the operand registers of mma.sync; while it passes over the
// query rows, eight a product, the next 32 keys' rows are on their way into the
// same place.  Keys are the rows of the product and the contraction order is
// free, so a lane takes 16 consecutive bytes of a bf16 row (4 of codes).  The
// sum over query rows stays in a thread and its three neighbours: a fixed order,
// no atomics.
// Bound by HBM (K once).
#include <type_traits>

#include "pa_cache_mma.cuh"

namespace pa {

struct WeightParams {
    CacheGeom g;
    const __nv_bfloat16* q;
    const uint8_t* k;
    const uint8_t* ks;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* ql;
    const float* lse;
    float* weights;
    int32_t* err;
};

namespace {

constexpr int kWeightWarps = 8, kCtas = 2;    // of an SM
constexpr int kWeightThreads = 32 * kWeightWarps;

// Up to this many query rows (of the longest q_len) this kernel runs; above,
// the one on tcgen05 (16 sequences of 8000 keys, 8 KV heads, here / there: 8 rows
// bf16 46 / 48 us, 4-bit 35 / 35; 16 rows 49 / 48 and 50 / 55; 24 rows 53 / 46
// and 64 / 51; 64 rows 88 / 46 and 136 / 49).
constexpr int kFewRows = 16;

// Bytes of a warp's place for 32 keys' rows (and scale words).
template <int D, bool MX4>
__host__ __device__ constexpr int weight_stage() {
    return MX4 ? 32 * (D / 2 + 4) : 32 * 2 * D;
}

// Where those places begin: behind Q and what belongs to its rows, on a whole
// line of banks.
template <int D>
__host__ __device__ constexpr int weight_rows_at() {
    return (kFewRows * (2 * D + kQPad + 12) + 127) / 128 * 128;
}

// First key (a multiple of 32) of the items of a sequence, and how many items.
__device__ __forceinline__ int seq_items(const CacheGeom& g, int c, int q, int keys, int& first) {
    first = 0;
    if (q <= 0 || !good_lens(g, q, c)) return 0;
    first = window_first_tile(g.window, c - q, 32) * 32;
    return (c - first + keys - 1) / keys;
}

// K becomes an operand as it is (bf16), or as f16 codes, the block scales
// applied to the block scores.
template <int D, bool MX4>
__global__ void __launch_bounds__(kWeightThreads, kCtas)
key_weights_kernel(const __grid_constant__ WeightParams P) {
    constexpr int KB = D / 32;                 // blocks of 32 columns
    constexpr int QROW = 2 * D + kQPad;
    constexpr int MT = 2;                      // 16-key tiles of a warp
    constexpr int kKeys = 32 * kWeightWarps;   // of one item
    constexpr int ROW = MX4 ? D / 2 : 2 * D;  // bytes of a key's row
    constexpr int CH = ROW / 16, RPI = 32 / CH;   // its chunks, rows a copy instruction
    extern __shared__ __align__(128) uint8_t smem[];
    float* off = reinterpret_cast<float*>(smem + kFewRows * QROW);   // -lse * log2 e
    float* fac = off + kFewRows;                                     // score factor
    int* pos = reinterpret_cast<int*>(fac + kFewRows);               // query position
    const uint32_t rows = smem_u32(smem) + weight_rows_at<D>() + (threadIdx.x >> 5) * weight_stage<D, MX4>();
    const CacheGeom& g = P.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gr = lane >> 2, t4 = lane & 3;
    grid_dependency_wait();

    auto cost = [&](int b) -> int64_t {
        int first;
        return (int64_t)g.Hkv * seq_items(g, P.ctx[b], P.ql[b], kKeys, first);
    };
    const int64_t total = flat_total(g.B, lane, cost);
    if (blockIdx.x == 0 && warp == 0) check_lens(g, P.ctx, P.ql, lane, P.err);
    const int64_t N = min((int64_t)gridDim.x, total);
    if (blockIdx.x >= N) return;
    int64_t i = total * blockIdx.x / N;
    const int64_t i_end = total * (blockIdx.x + 1) / N;

    // an item: keys of one KV head of one sequence
    struct Item {
        int b, hk, chunk, n, c, q, first, row0;
    };
    Item t;
    {
        int64_t start;
        t.b = flat_find(g.B, lane, i, cost, [&](int x) { return clamp_q(g, P.ql[x]); }, start,
                        t.row0);
        t.c = P.ctx[t.b];
        t.q = P.ql[t.b];
        t.n = seq_items(g, t.c, t.q, kKeys, t.first);
        t.hk = (int)((i - start) / t.n);
        t.chunk = (int)((i - start) % t.n);
    }
    auto advance = [&](Item& x) {
        if (++x.chunk < x.n) return;
        x.chunk = 0;
        if (++x.hk < g.Hkv) return;
        x.hk = 0;
        do {
            x.row0 += clamp_q(g, x.q);
            ++x.b;
            x.c = P.ctx[x.b];
            x.q = P.ql[x.b];
            x.n = seq_items(g, x.c, x.q, kKeys, x.first);
        } while (x.n == 0);
    };
    auto first_key = [&](const Item& x) { return x.first + x.chunk * kKeys + 32 * warp; };
    // the pages of a warp's two runs of 16 keys
    auto look_up = [&](const Item& x) -> int2 {
        const int32_t* row = P.table + (int64_t)x.b * g.mpps;
        const int key = first_key(x);
        int2 p = make_int2(-1, -1);
        if (key < x.c) p.x = p.y = row[key >> g.ps_shift];
        if (g.ps == 16) p.y = key + 16 < x.c ? row[(key >> 4) + 1] : -1;
        return p;
    };
    uint64_t once;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    const int page_rows = g.ps * g.Hkv;
    // where chunk c of row r goes: eight lanes of a load meet no bank twice
    auto chunk_at = [&](int r, int c) -> int {
        if constexpr (CH >= 8) return c ^ ((r & 1) << 2);        // bf16: 64 bytes of two rows
        else if constexpr (CH == 4) return c ^ ((r >> 1) & 3);   // codes: 16 bytes of eight
        else return c ^ ((r >> 2) & 1);
    };
    // the rows of an item's 32 keys, and their scales, on their way; keys that
    // do not exist, or whose page does not, become zeros
    auto issue = [&](const Item& x, int2 p) {
        const int key = first_key(x), left = x.c - key;
        const bool oka = (uint32_t)p.x < (uint32_t)g.num_pages;
        const bool okb = (uint32_t)p.y < (uint32_t)g.num_pages;
        const int64_t ra = (int64_t)p.x * page_rows +
                           ((key & (g.ps - 1)) * g.tok_rows + x.hk * g.head_rows);
        const int64_t rb = g.ps == 16 ? (int64_t)p.y * page_rows + x.hk * g.head_rows
                                      : ra + 16 * g.tok_rows;
        if (lane == 0 && ((left > 0 && !oka) || (left > 16 && !okb)))
            flag_error(P.err, PA_DEV_BAD_PAGE);
#pragma unroll
        for (int j = 0; j < 32 / RPI; ++j) {
            const int r = j * RPI + lane / CH, c = lane % CH;
            const bool ok = r < left && (r < 16 ? oka : okb);
            const int64_t row = (r < 16 ? ra : rb) + (r & 15) * g.tok_rows;
            cp_async16(rows + r * ROW + chunk_at(r, c) * 16, P.k + (ok ? row * ROW + c * 16 : 0),
                       ok ? 16 : 0, once);
        }
        if constexpr (MX4) {
            const bool ok = lane < left && (lane < 16 ? oka : okb);
            const int64_t row = (lane < 16 ? ra : rb) + (lane & 15) * g.tok_rows;
            // (head_dim 64: the word that holds the key's two bytes)
            cp_async4(rows + 32 * ROW + lane * 4, P.ks + (ok ? row * KB & ~(int64_t)3 : 0),
                      ok ? 4 : 0, once);
        }
        cp_async_commit();
    };
    int2 page = look_up(t);
    issue(t, page);
    Item next = t;
    int2 next_page = make_int2(-1, -1);
    if (i + 1 < i_end) {
        advance(next);
        next_page = look_up(next);
    }
    bool fresh = true;                         // Q of the item is not in shared memory
    bool blind = false;                        // some of its rows see nothing (padding, lse -inf)

    for (; i < i_end; ++i) {
        const int R = g.G * t.q, c = t.c, q = t.q;
        const bool rows_ok = t.row0 + q <= g.total_q;
        // ---- this warp's keys; lane (gr, t4) adds up key 8 t4 + gr
        const int tok = first_key(t), my_tok = tok + 8 * t4 + gr;
        const int my_page = t4 < 2 ? page.x : page.y;
        const bool mine_ok = my_tok < c && (uint32_t)my_page < (uint32_t)g.num_pages;
        float* dst = P.weights + ((int64_t)(mine_ok ? my_page : 0) * g.Hkv + t.hk) * g.ps +
                     (my_tok & (g.ps - 1));
        const float before = mine_ok ? *dst : 0.f;
        cp_async_wait<0>();
        __syncwarp();
        uint32_t a[MT][KB][2][4];              // (4-bit: a[..][0][hh] only, the codes)
        uint32_t e[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int r = 16 * mt + 8 * hh + gr;
                if constexpr (MX4) {
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
                        asm volatile("ld.shared.b32 %0, [%1];"
                                     : "=r"(a[mt][kb][0][hh])
                                     : "r"(rows + r * ROW + chunk_at(r, kb) * 16 + t4 * 4));
                    asm volatile("ld.shared.b32 %0, [%1];"
                                 : "=r"(e[mt][hh])
                                 : "r"(rows + 32 * ROW + r * 4));
                    if constexpr (D == 64) {
                        const int x = (tok + r) & (g.ps - 1);
                        e[mt][hh] >>= ((x * g.tok_rows + t.hk * g.head_rows) & 1) * 16;
                    }
                } else {
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(a[mt][kb][0][hh]), "=r"(a[mt][kb][0][2 + hh]),
                                       "=r"(a[mt][kb][1][hh]), "=r"(a[mt][kb][1][2 + hh])
                                     : "r"(rows + r * ROW + chunk_at(r, 4 * kb + t4) * 16));
                }
            }
        __syncwarp();
        // ---- the next item's rows into the same place, the one after's pages
        const Item done = t;
        if (i + 1 < i_end) {
            issue(next, next_page);
            t = next;
            page = next_page;
            if (i + 2 < i_end) {
                advance(next);
                next_page = look_up(next);
            }
        }
        float w[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) w[mt][0] = w[mt][1] = 0.f;
        const bool clear =
            tok + 16 * MT - 1 <= c - q && (g.window == 0 || tok > c - 1 - g.window);
        if (fresh) {
            // ---- the item's query rows, padded to a multiple of 8
            __syncthreads();
            bool none = false;
            for (int r = warp; r < ((R + 7) & ~7); r += kWeightWarps) {
                float x[D / 32];
                const bool real = r < R && rows_ok;
                const int64_t qrow = real ? (int64_t)(done.row0 + r / g.G) * g.Hq + done.hk * g.G + r % g.G
                                          : 0;
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const uint32_t v =
                        real ? reinterpret_cast<const uint32_t*>(P.q + qrow * D)[lane + 32 * j]
                             : 0u;
                    x[2 * j] = __uint_as_float(v << 16);
                    x[2 * j + 1] = __uint_as_float(v & 0xffff0000u);
                    top = fmaxf(top, fmaxf(fabsf(x[2 * j]), fabsf(x[2 * j + 1])));
                }
                float factor = g.sm_scale * kLog2e;
                float down = 1.f;
                if constexpr (MX4) {
                    // f16 rows with a power of two taken out (as in pa_decode_mx4)
                    const uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
                    const int ex = max(8, min(247, (int)(tb >> 23)));
                    down = __uint_as_float((uint32_t)(254 - ex) << 23);
                    factor *= __uint_as_float((uint32_t)ex << 23);
                }
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
                    *reinterpret_cast<uint32_t*>(smem + r * QROW + 4 * (lane + 32 * j)) =
                        MX4 ? pack_f16x2(x[2 * j] * down, x[2 * j + 1] * down)
                            : pack_bf16x2(x[2 * j], x[2 * j + 1]);
                const float v = real ? P.lse[qrow] : -INFINITY;
                none |= v == -INFINITY;
                if (lane == 0) {
                    off[r] = -v * kLog2e;
                    fac[r] = factor;
                    pos[r] = v == -INFINITY ? -1 : c - q + r / g.G;
                }
            }
            blind = __syncthreads_or(none);
            fresh = false;
        }
        const uint32_t qbase = smem_u32(smem) + gr * QROW + t4 * 16;
        const float factor = g.sm_scale * kLog2e;
        // eight rows against the warp's keys
        auto score = [&](int nt, auto mask) {
            constexpr bool masked = decltype(mask)::value;
            float s[MT][4];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint32_t b0, b1, b2, b3;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3)
                             : "r"(qbase + nt * QROW + kb * 64));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float* d = s[mt];
                    if constexpr (MX4) {
                        // converted anew for every eight rows: a row's codes as
                        // f16 beside all else do not fit 128 registers
                        // (64 sequences, 8 rows: 98 us, with 300 bytes spilled 108)
                        uint32_t h[2][4], ex[2];
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t code = a[mt][kb][0][hh];
                            ex[hh] = e[mt][hh];
                            asm volatile("" : "+r"(code), "+r"(ex[hh]));
                            e2m1x8_to_f16(code, h[0][hh], h[0][2 + hh], h[1][hh], h[1][2 + hh]);
                        }
                        float x[4];
                        mma_f16_first(x, h[0], b0, b1);
                        mma_f16_16816(x, h[1], b2, b3);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const float f = e8m0_to_f32((ex[hh] >> (8 * kb)) & 255u);
#pragma unroll
                            for (int v = 2 * hh; v < 2 * hh + 2; ++v)
                                d[v] = kb == 0 ? x[v] * f : fmaf(x[v], f, d[v]);
                        }
                    } else {
                        if (kb == 0)
                            mma_bf16_first(d, a[mt][kb][0], b0, b1);
                        else
                            mma_bf16_16816(d, a[mt][kb][0], b0, b1);
                        mma_bf16_16816(d, a[mt][kb][1], b2, b3);
                    }
                }
            }
            const int r = nt + 2 * t4;
            const float2 of = *reinterpret_cast<const float2*>(off + r);
            float2 fc = make_float2(factor, factor);
            if constexpr (MX4) fc = *reinterpret_cast<const float2*>(fac + r);
            int2 pp = make_int2(0, 0);
            if constexpr (masked) pp = *reinterpret_cast<const int2*>(pos + r);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float* d = s[mt] + 2 * hh;
                    float p0 = ex2(fmaf(d[0], fc.x, of.x));
                    float p1 = ex2(fmaf(d[1], fc.y, of.y));
                    if constexpr (masked) {
                        const int j = tok + 16 * mt + 8 * hh + gr;
                        if (j > pp.x || (g.window > 0 && j <= pp.x - g.window)) p0 = 0.f;
                        if (j > pp.y || (g.window > 0 && j <= pp.y - g.window)) p1 = 0.f;
                    }
                    w[mt][hh] += p0 + p1;
                }
        };
        if (!clear || blind) {
#pragma unroll 1
            for (int nt = 0; nt < R; nt += 8) score(nt, std::true_type());
        } else {
#pragma unroll 1
            for (int nt = 0; nt < R; nt += 8) score(nt, std::false_type());
        }
        // ---- over the four lanes that hold a key's rows; lane (gr, t4) adds key 8 t4 + gr
        float mine = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float x = w[mt][hh];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (t4 == 2 * mt + hh) mine = x;
            }
        if (mine_ok) *dst = before + mine;
        fresh = t.hk != done.hk || t.b != done.b;
    }
}

template <int D, bool MX4>
cudaError_t launch_weights(const WeightParams& P, int sms, cudaStream_t stream) {
    constexpr int smem = weight_rows_at<D>() + kWeightWarps * weight_stage<D, MX4>();
    const cudaError_t e = allow_smem<key_weights_kernel<D, MX4>>(smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(key_weights_kernel<D, MX4>, dim3(sms * kCtas), dim3(kWeightThreads),
                            smem, stream, P);
}

}  // namespace

cudaError_t launch_key_weights_many(const CacheGeom& g, bool mx4, const void* q, const void* k,
                                    const void* ks, const int32_t* table, const int32_t* ctx,
                                    const int32_t* ql, const float* lse, float* weights,
                                    int32_t* err, int sms, cudaStream_t stream);

cudaError_t launch_key_weights(const CacheGeom& g, bool mx4, const void* q, const void* k,
                               const void* ks, const int32_t* table, const int32_t* ctx,
                               const int32_t* ql, const float* lse, float* weights, int32_t* err,
                               int sms, cudaStream_t stream) {
    if (g.G * g.max_q_len > kFewRows)
        return launch_key_weights_many(g, mx4, q, k, ks, table, ctx, ql, lse, weights, err, sms,
                                       stream);
    WeightParams P;
    P.g = g;
    P.q = (const __nv_bfloat16*)q;
    P.k = (const uint8_t*)k;
    P.ks = (const uint8_t*)ks;
    P.table = table;
    P.ctx = ctx;
    P.ql = ql;
    P.lse = lse;
    P.weights = weights;
    P.err = err;
    if (g.D == 128)
        return mx4 ? launch_weights<128, true>(P, sms, stream)
                   : launch_weights<128, false>(P, sms, stream);
    return mx4 ? launch_weights<64, true>(P, sms, stream)
               : launch_weights<64, false>(P, sms, stream);
}

}  // namespace pa
