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

// 2^x for two lanes on the FMA pipe, for x <= 15: 2^x = 2^n 2^f with n = x rounded to the
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

// A value that is the same in the whole warp, in a form in which the compiler knows it.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// tcgen05.mma and commit by a whole converged warp, of which only the lane with `lead` issues:
// without a branch around them, and with the descriptors' changing low words as 32-bit values
// equal in the warp, a product issues in the time it runs (32 cycles at 64 x 64 x 16, measured).
// One lane in a branch of its own took 48 to 140.
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ explicit Desc(uint64_t d) : lo((uint32_t)d), hi((uint32_t)(d >> 32)) {}
    __device__ __forceinline__ Desc at(uint32_t bytes) const {  // below 256 KiB: no carry
        Desc d = *this;
        d.lo += bytes >> 4;
        return d;
    }
};
__device__ __forceinline__ void umma_if(bool lead, uint32_t d_tmem, Desc a, Desc b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %7, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}"
        ::"r"(d_tmem), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate),
          "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void umma_ts_if(bool lead, uint32_t d_tmem, uint32_t a_tmem, Desc b,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate),
          "r"((uint32_t)lead)
        : "memory");
}
// Whether phase `parity` of a barrier is complete, asked by the lanes with `asks` (others: false).
__device__ __forceinline__ bool mbar_test_if(bool asks, uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %3, 0;\n\t"
        "setp.ne.b32 p, 0, 0;\n\t"
        "@q mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"((uint32_t)asks)
        : "memory");
    return ok != 0;
}
// The same for a whole converged warp, asked by its lane or lanes with `lead`, of which each may
// name a barrier of its own: all of them have to be complete.
__device__ __forceinline__ bool mbar_test_warp(bool lead, uint32_t bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, mbar_test_if(lead, bar, parity) || !lead);
    __syncwarp();  // what the asking lane has seen is seen by all: a vote alone orders nothing
    return ok;
}
// wait_or_abort for a whole converged warp: the lanes with `asks` ask, each for a barrier of its own.
// The warp stays converged (it asks and votes in turn): a lane that waits in a branch of its own
// leaves the others free to reach the next product before it. A wait that gave up shows in `abort`
// too; a caller that goes on (over what memory holds, with waits that return at once) looks at the
// flag before it writes results.
__device__ __forceinline__ bool wait_warp(bool asks, uint32_t bar, uint32_t parity, volatile int *abort,
                                          unsigned long long limit_ns = kWaitLimitNs) {
    if (mbar_test_warp(asks, bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    while (true) {
        if (mbar_test_warp(asks, bar, parity)) return true;
        const bool late = globaltimer_ns() - t0 > limit_ns;
        if (late) *abort = 1;
        if (__any_sync(0xffffffffu, late || *abort)) {
            __syncwarp();  // the flag comes before what any lane does next
            return false;
        }
    }
}
// The copies of a converged warp, issued by its lane with `lead` (the same holds for their operands).
__device__ __forceinline__ void mbar_expect_if(bool lead, uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}"
        ::"r"(bar), "r"(bytes), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d_if(bool lead, uint32_t dst, const void *tmap, uint32_t bar,
                                               int x, int y) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];\n\t}"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_if(bool lead, uint32_t dst, const void *tmap, uint32_t bar,
                                               int x, int y, int z) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];\n\t}"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar),
          "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void bulk_load_if(bool lead, uint32_t dst, const void *src, uint32_t bytes,
                                             uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void umma_commit_if(bool lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(bar), "r"((uint32_t)lead)
        : "memory");
}

}  // namespace hmd
