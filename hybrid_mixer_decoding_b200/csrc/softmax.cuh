// What the attention kernels' softmax warps share: two-lane fp32 arithmetic, the exponential on
// the FMA pipe, and the bounded wait of a warp-specialised CTA.
#pragma once
#include "ptx.cuh"

namespace hmd {

// ---- two fp32 lanes per instruction (sm_100 f32x2 arithmetic) ----------------------------------
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x for two lanes on the FMA pipe, for x <= 8: 2^x = 2^n 2^f with n = x rounded to the
// nearest integer (adding 1.5 * 2^23 rounds it into the low mantissa bits) and f = x - n in
// [-1/2, 1/2], 2^f by a cubic fitted to it on that interval (iteratively reweighted least
// squares at Chebyshev nodes; largest relative error 7.5e-5, below the rounding of P to bf16 or fp16).
// n is added to the exponent field straight from the rounded sum's bits (its low bits hold n,
// the bits above them drop out of the shift). x is clamped at -125, where 2^x is below 1e-37
// and its share of a row sum that holds an entry >= 1 is nil. Splitting the exponentials
// between this and ex2.approx keeps the softmax off a single pipe.
__device__ __forceinline__ uint64_t exp2_fma_x2(uint64_t x2) {
    float a, b;
    f2_split(x2, a, b);
    x2 = f2(fmaxf(a, -125.f), fmaxf(b, -125.f));
    const uint64_t j = f2_add(x2, f2(12582912.f, 12582912.f));
    const uint64_t n = f2_add(j, f2(-12582912.f, -12582912.f));
    const uint64_t f = f2_fma(n, f2(-1.f, -1.f), x2);
    uint64_t p = f2_fma(f2(0.05517588f, 0.05517588f), f, f2(0.24261151f, 0.24261151f));
    p = f2_fma(p, f, f2(0.6932602f, 0.6932602f));
    p = f2_fma(p, f, f2(0.999928f, 0.999928f));
    float p0, p1, j0, j1;
    f2_split(p, p0, p1);
    f2_split(j, j0, j1);
    return f2(__uint_as_float(__float_as_uint(p0) + (__float_as_uint(j0) << 23)),
              __uint_as_float(__float_as_uint(p1) + (__float_as_uint(j1) << 23)));
}

// Bounded wait that also gives up as soon as another thread of the CTA raised `abort`.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
}

// One lane of a converged warp. The warps that issue tcgen05.mma run converged, take their
// branches by warp votes and issue under this predicate: operands that the compiler can see are
// the same in the whole warp cost one instruction each, others about 140 cycles per product
// (measured; a 64 x 64 x 16 product takes 32, a 128 x 128 x 16 one 64).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

}  // namespace hmd
