// pa_cache_mma.cuh -- what pa_decode_mx4 and pa_key_weights share: the scores
// of a 16-key tile against 8 query rows on mma.sync, transposed (keys are the
// rows of the product), and the division of flat work over the CTAs.
//
// Transposed, a unit of R query rows costs ceil(R / 8) products of 16 x 8
// instead of ceil(R / 16) of 16 x 16, a thread holds whole rows of keys (so a
// key's block scales belong to the thread), and the sum over query rows stays
// in a thread and its three neighbours.
#pragma once

#include "pa_cache_common.cuh"

namespace pa {

// D = A * B (f16, fp32 out), no accumulator input
__device__ __forceinline__ void mma_f16_first(float* d, const uint32_t* a, uint32_t b0,
                                              uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The same, bf16
__device__ __forceinline__ void mma_bf16_first(float* d, const uint32_t* a, uint32_t b0,
                                               uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two fp32 products or sums in one instruction.
__device__ __forceinline__ void fma2(float* d, const float* a, uint64_t b) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "fma.rn.f32x2 x, y, %4, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(d[0]), "+f"(d[1])
        : "f"(a[0]), "f"(a[1]), "l"(b));
}
__device__ __forceinline__ void mul2(float* d, const float* a, uint64_t b) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, y, %4;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "l"(b));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t make2(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 split2(uint64_t x) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
    return d;
}
__device__ __forceinline__ uint64_t pair2(float x) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(x));
    return d;
}

// Asynchronous copies with an L2 eviction priority; `bytes` 0 writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes,
                                           uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::64B [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes,
                                          uint64_t policy) {
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], 4, %2, %3;" ::"r"(dst),
                 "l"(src), "r"(bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A row of Q in shared memory is D f16 (or bf16) and this much padding: 8
// lanes of a 16-byte load (two rows of four chunks) then meet no bank twice.
constexpr int kQPad = 64;   // bytes

// Sequences' shares of a flat line of work, found by one warp without a table:
// cost(b) >= 0 units of work each, the total, and the sequence that holds a
// position.
template <typename Cost>
__device__ __forceinline__ int64_t flat_total(int B, int lane, Cost cost) {
    int64_t sum = 0;
    for (int b = lane; b < B; b += 32) sum += cost(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// The sequence b with start <= x < start + cost(b), for 0 <= x < total, and
// the sum `extra` of add(b') over the sequences before it (their query rows).
template <typename Cost, typename Add>
__device__ __forceinline__ int flat_find(int B, int lane, int64_t x, Cost cost, Add add,
                                         int64_t& start, int& extra) {
    int64_t run = 0;
    int rows = 0;
    for (int c0 = 0; c0 < B; c0 += 32) {
        const int b = c0 + lane;
        const int64_t v = b < B ? cost(b) : 0;
        const int q = b < B ? add(b) : 0;
        int64_t inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const int qinc = warp_inclusive(q, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, run + inc > x);
        if (past != 0) {
            const int i = __ffs(past) - 1;
            start = run + __shfl_sync(0xffffffffu, inc - v, i);
            extra = rows + __shfl_sync(0xffffffffu, qinc - q, i);
            return c0 + i;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
        rows += __shfl_sync(0xffffffffu, qinc, 31);
    }
    start = run;
    extra = rows;
    return B;
}

}  // namespace pa
