// pa_key_weights.cu -- adds to every cached key the softmax weight that a set
// of queries gives it:  w_j += sum_r exp2(f q_r . k_j - lse_r log2 e), over the
// rows r (query, q head of the key's group) that see key j.
//
// No sum runs over keys, so there is nothing to join: a warp owns 32 keys of
// one KV head, loads their rows once straight into the operand registers of
// mma.sync (keys are the rows of the product, the contraction order is free,
// so a lane takes 16 consecutive bytes of a bf16 row), and passes over the
// query rows, eight a product, from shared memory.  The sum over rows stays in
// a thread and its three neighbours: a fixed order, no atomics.
// Bound by HBM (K once) for a decode step's few rows; with many rows by the
// exponentials and products, which share the SM's issue slots.
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

constexpr int kWeightWarps = 8;
constexpr int kWeightThreads = 32 * kWeightWarps;
constexpr int kWeightKeys = 32 * kWeightWarps;   // keys of one item
constexpr int kQBlock = 128;                     // query rows in shared memory at a time

// First key (a multiple of 32) of the items of a sequence, and how many items.
__device__ __forceinline__ int seq_items(const CacheGeom& g, int c, int q, int& first) {
    first = 0;
    if (q <= 0 || !good_lens(g, q, c)) return 0;
    first = window_first_tile(g.window, c - q, 32) * 32;
    return (c - first + kWeightKeys - 1) / kWeightKeys;
}

template <int D, bool MX4>
__global__ void __launch_bounds__(kWeightThreads)
key_weights_kernel(const __grid_constant__ WeightParams P) {
    constexpr int KB = D / 32;                 // blocks of 32 columns
    constexpr int QROW = 2 * D + kQPad;
    extern __shared__ __align__(128) uint8_t smem[];
    float* off = reinterpret_cast<float*>(smem + kQBlock * QROW);   // lse * log2 e
    float* fac = off + kQBlock;                                     // score factor
    int* pos = reinterpret_cast<int*>(fac + kQBlock);               // query position
    const CacheGeom& g = P.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gr = lane >> 2, t4 = lane & 3;

    auto cost = [&](int b) -> int64_t {
        int first;
        return (int64_t)g.Hkv * seq_items(g, P.ctx[b], P.ql[b], first);
    };
    const int64_t total = flat_total(g.B, lane, cost);
    if (blockIdx.x == 0 && warp == 0) check_lens(g, P.ctx, P.ql, lane, P.err);
    const int64_t N = min((int64_t)gridDim.x, total);
    if (blockIdx.x >= N) return;
    int64_t i = total * blockIdx.x / N;
    const int64_t i_end = total * (blockIdx.x + 1) / N;
    int64_t start;
    int row0;
    int b = flat_find(g.B, lane, i, cost, [&](int x) { return clamp_q(g, P.ql[x]); }, start, row0);
    int c = P.ctx[b], q = P.ql[b], first;
    int n = seq_items(g, c, q, first);
    int hk = (int)((i - start) / n), chunk = (int)((i - start) % n);
    bool fresh = true;                         // Q of (b, hk) is not in shared memory
    bool blind = false;                        // some of its rows see nothing (padding, lse -inf)

    for (; i < i_end; ++i) {
        const int R = g.G * q;
        const bool rows_ok = row0 + q <= g.total_q;
        // ---- this warp's 32 keys
        const int tok = first + chunk * kWeightKeys + 32 * warp;
        const int my_tok = tok + 8 * t4 + gr;  // the key this lane adds up for
        const bool in = my_tok < c;
        int page = in ? P.table[(int64_t)b * g.mpps + (my_tok >> g.ps_shift)] : -1;
        if (in && (page < 0 || page >= g.num_pages)) {
            flag_error(P.err, PA_DEV_BAD_PAGE);
            page = -1;
        }
        const int slot = my_tok & (g.ps - 1);
        float* dst = P.weights + ((int64_t)max(page, 0) * g.Hkv + hk) * g.ps + slot;
        const float before = page >= 0 ? *dst : 0.f;
        const int64_t my_row = page >= 0 ? row_of(g, page, slot, hk) : -1;
        uint32_t a[2][KB][2][4];
        float f[2][2][KB];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                // row of key 16 mt + 8 hh + gr, found by lane (gr, 2 mt + hh)
                const int64_t row = __shfl_sync(0xffffffffu, my_row, gr * 4 + 2 * mt + hh);
                if constexpr (MX4) {
                    uint32_t w[KB], e = 0;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
                        w[kb] = row >= 0 ? *reinterpret_cast<const uint32_t*>(
                                               P.k + row * (D / 2) + kb * 16 + t4 * 4)
                                         : 0u;
                    if (row >= 0)
                        e = D == 128 ? *reinterpret_cast<const uint32_t*>(P.ks + row * 4)
                                     : *reinterpret_cast<const uint16_t*>(P.ks + row * 2);
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        e2m1x8_to_f16(w[kb], a[mt][kb][0][hh], a[mt][kb][0][2 + hh],
                                      a[mt][kb][1][hh], a[mt][kb][1][2 + hh]);
                        f[mt][hh][kb] = e8m0_to_f32((e >> (8 * kb)) & 255u);
                    }
                } else {
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (row >= 0)
                            x = *reinterpret_cast<const uint4*>(P.k + row * (2 * D) + kb * 64 +
                                                                t4 * 16);
                        a[mt][kb][0][hh] = x.x;
                        a[mt][kb][0][2 + hh] = x.y;
                        a[mt][kb][1][hh] = x.z;
                        a[mt][kb][1][2 + hh] = x.w;
                    }
                }
            }
        float w[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
        const bool clear = tok + 31 <= c - q && (g.window == 0 || tok > c - 1 - g.window);
        for (int r0 = 0; r0 < R; r0 += kQBlock) {
            const int nr = min(kQBlock, R - r0);
            if (fresh || R > kQBlock) {
                // ---- query rows r0 .. r0 + nr, padded to a multiple of 8
                __syncthreads();
                bool none = false;
                for (int r = warp; r < ((nr + 7) & ~7); r += kWeightWarps) {
                    float x[D / 32];
                    const bool real = r < nr && rows_ok;
                    const int64_t qrow = real ? (int64_t)(row0 + (r0 + r) / g.G) * g.Hq +
                                                    hk * g.G + (r0 + r) % g.G
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
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int e = max(8, min(247, (int)(__float_as_uint(top) >> 23)));
                        down = __uint_as_float((uint32_t)(254 - e) << 23);
                        factor *= __uint_as_float((uint32_t)e << 23);
                    }
#pragma unroll
                    for (int j = 0; j < D / 64; ++j)
                        *reinterpret_cast<uint32_t*>(smem + r * QROW + 4 * (lane + 32 * j)) =
                            MX4 ? pack_f16x2(x[2 * j] * down, x[2 * j + 1] * down)
                                : pack_bf16x2(x[2 * j], x[2 * j + 1]);
                    const float v = real ? P.lse[qrow] : -INFINITY;
                    none |= v == -INFINITY;
                    if (lane == 0) {
                        off[r] = v * kLog2e;
                        fac[r] = factor;
                        pos[r] = v == -INFINITY ? -1 : c - q + (r0 + r) / g.G;
                    }
                }
                blind = __syncthreads_or(none);
                fresh = false;
            }
            const uint32_t qbase = smem_u32(smem);
            for (int nt = 0; nt < nr; nt += 8) {
                float s[2][4];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    uint32_t b0, b1, b2, b3;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3)
                                 : "r"(qbase + (nt + gr) * QROW + kb * 64 + t4 * 16));
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        if constexpr (MX4) {
                            float x[4];
                            mma_f16_first(x, a[mt][kb][0], b0, b1);
                            mma_f16_16816(x, a[mt][kb][1], b2, b3);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                s[mt][e] = kb == 0 ? x[e] * f[mt][e >> 1][0]
                                                   : fmaf(x[e], f[mt][e >> 1][kb], s[mt][e]);
                        } else {
                            if (kb == 0) s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;
                            mma_bf16_16816(s[mt], a[mt][kb][0], b0, b1);
                            mma_bf16_16816(s[mt], a[mt][kb][1], b2, b3);
                        }
                    }
                }
                const float2 fc = *reinterpret_cast<const float2*>(fac + nt + 2 * t4);
                const float2 of = *reinterpret_cast<const float2*>(off + nt + 2 * t4);
                const int2 pp = *reinterpret_cast<const int2*>(pos + nt + 2 * t4);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = fmaf(s[mt][e], e & 1 ? fc.y : fc.x, -(e & 1 ? of.y : of.x));
                        if (!clear || blind) {
                            const int j = tok + 16 * mt + 8 * (e >> 1) + gr;
                            const int p = e & 1 ? pp.y : pp.x;
                            if (j > p || (g.window > 0 && j <= p - g.window)) x = -INFINITY;
                        }
                        w[mt][e >> 1] += ex2(x);
                    }
            }
        }
        // ---- over the four lanes that hold a key's rows; lane (gr, t4) adds key 8 t4 + gr
        float mine = 0.f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float x = w[mt][hh];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (t4 == 2 * mt + hh) mine = x;
            }
        if (page >= 0) *dst = before + mine;
        // ---- the next item
        if (++chunk == n) {
            chunk = 0;
            fresh = true;
            if (++hk == g.Hkv) {
                hk = 0;
                if (i + 1 < i_end) {
                    do {
                        row0 += clamp_q(g, q);
                        ++b;
                        c = P.ctx[b];
                        q = P.ql[b];
                        n = seq_items(g, c, q, first);
                    } while (n == 0);
                }
            }
        }
    }
}

template <int D, bool MX4>
cudaError_t launch_weights(const WeightParams& P, int sms, cudaStream_t stream) {
    constexpr int smem = kQBlock * (2 * D + kQPad) + 3 * kQBlock * 4;
    auto kern = key_weights_kernel<D, MX4>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kWeightThreads, smem);
    if (e != cudaSuccess) return e;
    kern<<<sms * (per_sm > 0 ? per_sm : 1), kWeightThreads, smem, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights(const CacheGeom& g, bool mx4, const void* q, const void* k,
                               const void* ks, const int32_t* table, const int32_t* ctx,
                               const int32_t* ql, const float* lse, float* weights, int32_t* err,
                               int sms, cudaStream_t stream) {
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
