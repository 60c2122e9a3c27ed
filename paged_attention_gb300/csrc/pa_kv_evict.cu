// pa_kv_evict.cu -- which keys of a paged cache to keep, by their accumulated
// weights, and moving the kept rows into other pages.
//
// Select, one CTA per sequence and KV head: the budget-th largest key by a radix
// select, eight bits a pass over an order-preserving integer form of the
// weights, then one ordered pass that lists the kept positions (ties to the
// lower one).  Move, a second launch over all SMs: 64 kept rows of K and V a
// CTA, 16 bytes a thread.  The move is bound by HBM, the selection by the
// latency of its passes and, with two CTAs an SM, by their instructions: 32
// sequences of 8192 .. 32768 keys, 8 heads, 2048 kept: 130 us, 85 of them the move,
// where reading the weights and moving the rows takes 83 us of HBM time.  Past
// kMaxCached keys every pass reads the weights through the block table again: 4
// sequences of 60000 keys 60 us, of 131071 314 us.
#include "pa_cache_common.cuh"

namespace pa {

struct EvictParams {
    CacheGeom g;
    int32_t budget, num_first, num_recent;
    uint8_t* k;
    uint8_t* ks;
    uint8_t* v;
    uint8_t* vs;
    float* weights;
    const int32_t* table;
    const int32_t* dst_table;
    int32_t dst_mpps;
    const int32_t* ctx;
    int32_t* kept;
    int32_t* new_ctx;
    int32_t* err;
};

namespace {

constexpr int kBins = 256;
// Copies of the histogram, which lanes spread over: fewer are cheaper to clear
// and to add up, more meet less often.
constexpr int copies_of(bool few) { return few ? 8 : 32; }
constexpr int hist_bytes(bool few) { return kBins * copies_of(few) * 4; }
// Keys (as position and value) whose upper half is the threshold's, at most
constexpr int kListed = 1024;
// Keys whose upper halves shared memory holds
constexpr int kMaxCached = (227 * 1024 - hist_bytes(false) - kListed * 8 - 4096) / 2;
constexpr int kFewKeys = 12288;    // longest sequence that few threads select from
constexpr int kMoveRows = 64;

constexpr int kMoveThreads = 256;

// kMoveRows rows of a kept list into their new pages.  PIECES: 16-byte pieces of a
// row (D / 8 of bf16, D / 32 of 4-bit codes).
template <int PIECES>
__global__ void __launch_bounds__(kMoveThreads)
move_kernel(const __grid_constant__ EvictParams P, int chunks, int scale_bytes) {
    __shared__ struct {
        int64_t src[kMoveRows], dst[kMoveRows];
    } at;
    const CacheGeom& g = P.g;
    grid_dependency_wait();
    const int unit = blockIdx.x / chunks, r0 = blockIdx.x % chunks * kMoveRows;
    const int b = unit / g.Hkv, hk = unit % g.Hkv, c = P.ctx[b], tid = threadIdx.x;
    if (c <= P.budget || c > g.max_ctx) return;
    const int n = min(kMoveRows, P.budget - r0);
    if (tid < n) {
        const int from = P.kept[(int64_t)unit * P.budget + r0 + tid], to = r0 + tid;
        const bool listed = from >= 0 && from < c;
        const int sp = listed ? P.table[(int64_t)b * g.mpps + (from >> g.ps_shift)] : -1;
        const int dp = P.dst_table[(int64_t)b * P.dst_mpps + (to >> g.ps_shift)];
        const bool ok = sp >= 0 && sp < g.num_pages && dp >= 0 && dp < g.num_pages;
        const int ss = from & (g.ps - 1), ds = to & (g.ps - 1);
        const int64_t s = ok ? row_of(g, sp, ss, hk) : -1, d = ok ? row_of(g, dp, ds, hk) : 0;
        at.src[tid] = s;
        at.dst[tid] = d;
        if (ok) {
            P.weights[((int64_t)dp * g.Hkv + hk) * g.ps + ds] =
                P.weights[((int64_t)sp * g.Hkv + hk) * g.ps + ss];
            if (scale_bytes == 4) {
                reinterpret_cast<uint32_t*>(P.ks)[d] = reinterpret_cast<const uint32_t*>(P.ks)[s];
                reinterpret_cast<uint32_t*>(P.vs)[d] = reinterpret_cast<const uint32_t*>(P.vs)[s];
            } else if (scale_bytes == 2) {
                reinterpret_cast<uint16_t*>(P.ks)[d] = reinterpret_cast<const uint16_t*>(P.ks)[s];
                reinterpret_cast<uint16_t*>(P.vs)[d] = reinterpret_cast<const uint16_t*>(P.vs)[s];
            }
        } else {
            flag_error(P.err, PA_DEV_BAD_PAGE);
        }
    }
    __syncthreads();
    // pieces of K, then of V; every load of a thread before its stores
    constexpr int kPer = (2 * PIECES * kMoveRows + kMoveThreads - 1) / kMoveThreads;
    uint4 x[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid + j * kMoveThreads, kv = i / (PIECES * kMoveRows);
        const int r = (i / PIECES) % kMoveRows, p = i % PIECES;
        x[j] = make_uint4(0u, 0u, 0u, 0u);
        if (kv < 2 && r < n && at.src[r] >= 0)
            x[j] = __ldcs(reinterpret_cast<const uint4*>(kv ? P.v : P.k) + at.src[r] * PIECES + p);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = tid + j * kMoveThreads, kv = i / (PIECES * kMoveRows);
        const int r = (i / PIECES) % kMoveRows, p = i % PIECES;
        if (kv < 2 && r < n && at.src[r] >= 0)
            __stcs(reinterpret_cast<uint4*>(kv ? P.v : P.k) + at.dst[r] * PIECES + p, x[j]);
    }
}

// Larger weights get larger keys; NaN the smallest, a protected position the largest.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);   // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The upper halves of the keys stay in shared memory.  Where the first two passes leave few keys
// that share the threshold's upper half, those are read again, all at once, and
// decide the rest; where many do (equal weights), or the keys do not fit, every
// later step reads them where they are.
template <int kSelectThreads, bool FEW>
__global__ void __launch_bounds__(kSelectThreads)
select_kernel(const __grid_constant__ EvictParams P, int cached_cap) {
    grid_dependency_wait();
    constexpr int kSelectWarps = kSelectThreads / 32, kCopies = copies_of(FEW);
    extern __shared__ __align__(128) uint8_t smem[];
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem);
    uint2* list = reinterpret_cast<uint2*>(smem + hist_bytes(FEW));     // (position, key)
    uint16_t* cached = reinterpret_cast<uint16_t*>(smem + hist_bytes(FEW) + kListed * 8);
    __shared__ int s_listed;
    __shared__ uint32_t bins[kBins];
    __shared__ uint32_t s_digit, s_left;
    __shared__ int2 s_count[kSelectWarps];
    const CacheGeom& g = P.g;
    const int b = blockIdx.x / g.Hkv, hk = blockIdx.x % g.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = P.ctx[b];
    const bool bad = c < 0 || c > g.max_ctx;
    if (hk == 0 && tid == 0) {
        P.new_ctx[b] = bad ? 0 : min(c, P.budget);
        if (bad) flag_error(P.err, PA_DEV_BAD_LENGTHS);
    }
    if (bad || c <= P.budget) return;
    const int32_t* row = P.table + (int64_t)b * g.mpps;
    // (no branches: the loads of a loop's iterations run together; a page that
    // is none counts as the smallest key, and the first pass flags it)
    auto key_at = [&](int i) -> uint32_t {
        const int page = row[i >> g.ps_shift];
        const bool ok = (uint32_t)page < (uint32_t)g.num_pages;
        const float w =
            P.weights[((int64_t)(ok ? page : 0) * g.Hkv + hk) * g.ps + (i & (g.ps - 1))];
        const uint32_t x = ok ? order_key(w) : 0u;
        return i < P.num_first || i >= c - P.num_recent ? 0xffffffffu : x;
    };
    const bool in_smem = c <= cached_cap;
    auto upper = [&](int i) -> uint32_t { return in_smem ? cached[i] : key_at(i) >> 16; };
    // the upper halves of eight keys that shared memory holds (i a multiple of 8;
    // behind the last key: anything)
    auto eight = [&](int i, uint32_t* u) {
        const uint4 v = *reinterpret_cast<const uint4*>(cached + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[2 * j] = w[j] & 0xffffu;
            u[2 * j + 1] = w[j] >> 16;
        }
    };
    auto clear = [&]() {
        for (int i = tid; i < kBins * kCopies / 4; i += kSelectThreads)
            reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    };
    auto count = [&](uint32_t digit) {
        atomicAdd(&hist[digit * kCopies + lane % kCopies], 1u);
    };

    // ---- the budget-th largest key
    bool listed = false;
    if (tid == 0) s_listed = 0;
    uint32_t prefix = 0, left = (uint32_t)P.budget;   // rank from the top among equal prefixes
    for (int shift = 24; shift >= 0; shift -= 8) {
        clear();
        // (eight keys are read before the first is counted: no load passes an
        // atomic operation by itself)
        if (shift == 24) {
            // a warp takes 256 keys at a time; lane l < 16 has the page of their
            // l-th run of 16, looked up a turn ahead
            auto look_up = [&](int i) -> int {
                const int k = i + 16 * (lane & 15);
                return k < c ? row[k >> g.ps_shift] : -1;
            };
            int page = look_up(256 * warp);
            bool none = false;
            for (int i = 256 * warp; i < c; i += 8 * kSelectThreads) {
                const int now = page;
                none |= i + 16 * (lane & 15) < c && (uint32_t)now >= (uint32_t)g.num_pages;
                page = look_up(i + 8 * kSelectThreads);
                float w[8];
                bool ok[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int p = __shfl_sync(0xffffffffu, now, 2 * j + (lane >> 4));
                    ok[j] = (uint32_t)p < (uint32_t)g.num_pages;
                    w[j] = P.weights[((int64_t)(ok[j] ? p : 0) * g.Hkv + hk) * g.ps +
                                     ((i + 32 * j + lane) & (g.ps - 1))];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = i + 32 * j + lane;
                    if (k < c) {
                        uint32_t x = ok[j] ? order_key(w[j]) : 0u;
                        if (k < P.num_first || k >= c - P.num_recent) x = 0xffffffffu;
                        if (in_smem) cached[k] = (uint16_t)(x >> 16);
                        count(x >> 24);
                    }
                }
            }
            if (none) flag_error(P.err, PA_DEV_BAD_PAGE);
        } else if (shift == 16) {
            for (int i = tid; i < c; i += 8 * kSelectThreads) {
                uint32_t x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = upper(min(i + j * kSelectThreads, c - 1));
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i + j * kSelectThreads < c && x[j] >> 8 == prefix) count(x[j] & 255u);
            }
        } else if (listed) {
            for (int i = tid; i < s_listed; i += kSelectThreads) {
                const uint32_t x = list[i].y;
                if (x >> (shift + 8) == prefix) count((x >> shift) & 255u);
            }
        } else {
            for (int i = tid; i < c; i += kSelectThreads)
                if (upper(i) == prefix >> (8 - shift)) {
                    const uint32_t x = key_at(i);
                    if (x >> (shift + 8) == prefix) count((x >> shift) & 255u);
                }
        }
        __syncthreads();
        if (tid < kBins) {
            uint32_t s = 0;
#pragma unroll
            for (int j = 0; j < kCopies / 4; ++j) {
                const uint4 v = reinterpret_cast<const uint4*>(
                    hist)[tid * (kCopies / 4) + (j + tid) % (kCopies / 4)];
                s += v.x + v.y + v.z + v.w;
            }
            bins[tid] = s;
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds digits 255 - 8 l downwards
            uint32_t v[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = bins[255 - 8 * lane - j];
                sum += v[j];
            }
            const uint32_t inc = (uint32_t)warp_inclusive((int)sum, lane);
            uint32_t above = inc - sum;
            if (above < left && left <= inc) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (left > above && left <= above + v[j]) {
                        s_digit = 255 - 8 * lane - j;
                        s_left = left - above;
                    }
                    above += v[j];
                }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | s_digit;
        left = s_left;
        if (shift == 16 && in_smem) {
            listed = bins[prefix & 255u] <= kListed;
            if (listed) {
                for (int i = 8 * tid; i < c; i += 8 * kSelectThreads) {
                    uint32_t u[8];
                    eight(i, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (u[j] == prefix && i + j < c) list[atomicAdd(&s_listed, 1)].x = i + j;
                }
                __syncthreads();
                for (int i = tid; i < s_listed; i += kSelectThreads)
                    list[i].y = key_at((int)list[i].x);
                // (read after the next barrier)
            }
        }
    }
    if (listed) {
        // from now on an upper half tells a key's side of the threshold: 0xffff
        // and 0 are the halves of one key each, the largest and the smallest
        for (int i = tid; i < s_listed; i += kSelectThreads) {
            const uint2 x = list[i];
            if (x.y != prefix) cached[x.x] = x.y > prefix ? 0xffffu : 0u;
        }
        __syncthreads();
    }
    // kept: keys above `prefix`, and the first `left` that equal it

    // ---- list the kept positions; a warp owns a run of positions, a lane eight
    // neighbours of it at a time
    const int per_warp = (c + 256 * kSelectWarps - 1) / (256 * kSelectWarps) * 256;
    const int i0 = min(c, warp * per_warp), i1 = min(c, i0 + per_warp);
    int32_t* out = P.kept + (int64_t)blockIdx.x * P.budget;
    // sides(i, x): of keys i .. i + 7, 1 above the threshold, 0 equal, -1 below
    auto sweep = [&](auto sides) {
        uint32_t mine = 0;                            // above, and equal << 16, of a warp's turn
        int above = 0, equal = 0;
        auto tally = [&](const int* x) {
            mine = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) mine += x[j] > 0 ? 1u : x[j] == 0 ? 0x10000u : 0u;
        };
        for (int i = i0 + 8 * lane; i < i1; i += 256) {
            int x[8];
            sides(i, x);
            tally(x);
            above += (int)(mine & 0xffffu);
            equal += (int)(mine >> 16);
        }
        above = __reduce_add_sync(0xffffffffu, above);
        equal = __reduce_add_sync(0xffffffffu, equal);
        if (lane == 0) s_count[warp] = make_int2(above, equal);
        __syncthreads();
        const int2 all = lane < kSelectWarps ? s_count[lane] : make_int2(0, 0);
        const int ea = warp_inclusive(all.x, lane) - all.x;
        const int ee = warp_inclusive(all.y, lane) - all.y;
        int na = __shfl_sync(0xffffffffu, ea, warp);  // kept before this warp's turn
        int ne = __shfl_sync(0xffffffffu, ee, warp);
        for (int k = i0; k < i1; k += 256) {
            const int i = k + 8 * lane;
            int x[8] = {-1, -1, -1, -1, -1, -1, -1, -1};
            if (i < i1) sides(i, x);
            tally(x);
            const uint32_t inc = (uint32_t)warp_inclusive((int)mine, lane);
            int a = na + (int)((inc - mine) & 0xffffu), e = ne + (int)((inc - mine) >> 16);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (x[j] > 0 || (x[j] == 0 && e < (int)left)) out[a + min(e, (int)left)] = i + j;
                a += x[j] > 0;
                e += x[j] == 0;
            }
            const uint32_t turn = __shfl_sync(0xffffffffu, inc, 31);
            na += (int)(turn & 0xffffu);
            ne += (int)(turn >> 16);
        }
    };
    if (listed) {
        const uint32_t pu = prefix >> 16;
        sweep([&](int i, int* x) {
            uint32_t u[8];
            eight(i, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = i + j < c ? (u[j] > pu) - (u[j] < pu) : -1;
        });
    } else {
        sweep([&](int i, int* x) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t k = key_at(min(i + j, c - 1));
                x[j] = i + j < c ? (k > prefix) - (k < prefix) : -1;
            }
        });
    }
}

template <int kSelectThreads, bool FEW>
cudaError_t launch_select(const EvictParams& P, int cap, int units, int smem, cudaStream_t stream) {
    const cudaError_t e = allow_smem<select_kernel<kSelectThreads, FEW>>(
        hist_bytes(FEW) + kListed * 8 + (FEW ? kFewKeys : kMaxCached) * 2 + 16);
    if (e != cudaSuccess) return e;
    return launch_dependent(select_kernel<kSelectThreads, FEW>, dim3(units), dim3(kSelectThreads),
                            smem, stream, P, cap);
}

}  // namespace

cudaError_t launch_evict(const CacheGeom& g, bool mx4, int budget, int num_first, int num_recent,
                         void* k, void* ks, void* v, void* vs, float* weights,
                         const int32_t* table, const int32_t* dst_table, int dst_mpps,
                         const int32_t* ctx, int32_t* kept, int32_t* new_ctx, int32_t* err, int sms,
                         cudaStream_t stream) {
    EvictParams P;
    P.g = g;
    P.budget = budget;
    P.num_first = num_first;
    P.num_recent = num_recent;
    P.k = (uint8_t*)k;
    P.ks = (uint8_t*)ks;
    P.v = (uint8_t*)v;
    P.vs = (uint8_t*)vs;
    P.weights = weights;
    P.table = table;
    P.dst_table = dst_table;
    P.dst_mpps = dst_mpps;
    P.ctx = ctx;
    P.kept = kept;
    P.new_ctx = new_ctx;
    P.err = err;
    // the longest sequence's keys fit shared memory, or are read from L2 every pass
    const int cap = g.max_ctx <= kMaxCached ? g.max_ctx : kMaxCached;
    const int units = g.B * g.Hkv;
    const int pieces = mx4 ? g.D / 32 : g.D / 8, scale_bytes = mx4 ? g.D / 32 : 0;
    // Few threads a CTA where an SM gets several (512 pairs, 64 keys kept of 1000 /
    // 4000 / 6000 / 12000: 17 / 25 / 29 / 46 us with 256 threads, 25 / 31 / 38 / 52
    // with 512), 1024 where it gets one and the sequence is long (64 pairs of 6000:
    // 18.6 us with 256, 17.4 with 512, 16.6 with 1024; of 20000: 29 with 512, 25
    // with 1024).
    const bool one = units <= sms, few = cap <= (one ? 4096 : kFewKeys), wide = !few && one;
    const int smem = hist_bytes(few) + kListed * 8 + (cap * 2 + 15) / 16 * 16;
    const int chunks = (budget + kMoveRows - 1) / kMoveRows;
    const int64_t grid = (int64_t)units * chunks;
    if (g.max_ctx > budget && grid > 0x7fffffff) return cudaErrorInvalidValue;
    cudaError_t e = few    ? launch_select<256, true>(P, cap, units, smem, stream)
                    : wide ? launch_select<1024, false>(P, cap, units, smem, stream)
                           : launch_select<512, false>(P, cap, units, smem, stream);
    if (e != cudaSuccess || g.max_ctx <= budget) return e;
    auto move = pieces == 16  ? move_kernel<16>
                : pieces == 8 ? move_kernel<8>
                : pieces == 4 ? move_kernel<4>
                              : move_kernel<2>;
    return launch_dependent(move, dim3((unsigned)grid), dim3(kMoveThreads), 0, stream, P, chunks,
                            scale_bytes);
}

}  // namespace pa
