// Latent attention, expanded form: the new tokens of prompts, after a cached prefix or none.
//
// A cached token is one row [c (d_c) ; k_r (64)] shared by every head; head h's key is
// [W_uk[h] c ; k_r], its value W_uv[h] c. With many queries per key the expanded form does the
// least arithmetic (2 d + 64 products a (query, key) pair and head, against 2 d_c + 64 absorbed), so
// every key and value is formed once, into a workspace, and attended as usual. It is bound by the
// tensor cores: attention's products, and 4 d d_c flop per (token, head) to expand.
//
// The intermediate keys, values, queries and softmax weights are fp16, not bf16: rounding keys,
// values and weights to bf16 would each add the error of the bf16 output itself (2^-8); fp16's 2^-11
// adds nothing visible. Its range is 65504: larger keys, values or queries are clipped and reported
// (HMD_DEVWARN_RANGE). Downwards it ends at 2^-14, so the values of a head in a tile of 128 positions are
// stored times 2^e, e = 0, 20, 40 or 60, with which the largest of them is at 2^-5 or above (or as near as
// e = 60 brings it): values are held to 2^-11, or to 2^-20 of the largest. Most often e is 0 everywhere, or the
// same; where it is not, the softmax lowers a tile's exponents by e and adds its weights times 2^e to the
// row's sum, so that tiles of any sizes add up (a loop of its own: in the common one this took 2 to 4% of the
// kernel). e goes with the values, in the last bits of three of them (those to 2^-10). Keys and queries need no
// such factor: what they lose below 2^-14, at most 2^-25, moves a score by 2^-25 scale sum |q| (or |k|), with
// the usual scale 4e-7 for 192 dims of size 1 and 0.03 at the end of fp16's range. So that this holds for any
// scale, the power of two in one of 2 or more goes to the queries.
//
// Kernel 1 (rows): appends the new rows to the cache and converts every position's shared part
// k_r to fp16. Kernel 2 (expand): one CTA per (128 positions, a share of the heads):
//     [K_h ; V_h] [128 x 2d] = C [128 x d_c] [W_uk[h] ; W_uv[h]]^T     tcgen05, M = 128, N = 128
// C is the products' A operand and stays in TMEM, so that only the weights stream through shared memory
// (a 128 x 128 product with both operands there reads 128 bytes a cycle, all it has: 74 us for 8192
// positions of 32 heads, 59 us so); two accumulators, so one step's results are stored while the next
// is computed. It is bound by the warp that copies the weights, 256 KB a head and tile from L2 in stages of
// 16 KB: a stage takes 400 cycles, of which its products are 256 (one predicate more in that warp's loop
// made 66 us of 59, the test of a flag 79).
// Kernel 3 (attend): one CTA per (sequence, head, 256 queries): two query tiles of 128 whose
// softmax groups alternate with the tensor core, as in the FA prefill; K tiles are d/64 + 1
// blocks (the last one k_r, shared by the heads), V tiles d/64, all in one ring of blocks. A softmax group
// reads its scores into registers at once, so that one S in TMEM serves both groups and each has
// its own P: a tile's scores are complete before the softmax of the tile before is done (with S and P
// of a group in one place a key tile took 3400 cycles, softmax and products of a group in turn; now
// 2900). d = 128: the products of a key tile alone take 2560, and with the copies they move 340 KB through
// shared memory, 2660 cycles of its 128 bytes. B = 2, T = 4096, 32 heads: 405 us in all (1.02 PFLOP/s), 457
// to 483 in a row under the power limit; B = 3, 1000 after 2801: 237, 241 to 251 in a row. A CTA's start and
// end are about 12000 cycles, a fifth of the kernel at T = 4096.
// If the workspace holds fewer heads than H, kernels 2 and 3 run once per group of heads.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "latent_ring.h"
#include "ptx.cuh"
#include "softmax.cuh"
#include "../../include/hmd.h"

namespace hmd {
namespace {

__device__ unsigned int g_err;

constexpr int kPT = 64;              // tokens per page
constexpr int kDR = 64;              // the rows' part shared as it is by every head's key
constexpr int kTile = 128;           // positions per key tile, queries per query tile
constexpr uint32_t kBlk = kTile * 128;  // one [128 rows][128 B] block, 128-byte swizzle
constexpr float kHalfMax = 65504.f;
// A row's weights are held relative to a base that moves when the largest is above 2^kTop, then to
// 2^kFresh: fp16 holds a weight to 2^-11 down to 2^-23 of the row's largest, and to 2^-34 of that below. (With
// the largest at 1, 100,000 keys of 2^-25.5 each were in the row's sum and not in its output.)
constexpr float kTop = 15.f, kFresh = 9.f;
// A head's values in a tile are stored times 2^e, e = kMaxExp - kExpStep * code, the code in the last bits of
// its first kExpBits values (kMissing: kernel 2 gave up on the tile). The largest e leaves a row's sum, which
// has every weight times 2^e, far from fp32's ends: 2^75 a key, and the 2^-125 at which the softmax clamps a
// masked key's weight is 2^-65.
constexpr int kMaxExp = 60, kExpStep = 20, kExpBits = 3;
constexpr uint32_t kMissing = 7;
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Instruction descriptor of kind::f16 with fp16 A/B and fp32 D: the bf16 one with both type fields 0.
constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
    return idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// The fp16 nearest to x whose last bit is `bit`.
__device__ __forceinline__ uint32_t half_with_last_bit(float x, uint32_t bit) {
    const __half n = __float2half_rn(x);
    const uint32_t h = __half_as_ushort(n);
    if ((h & 1u) == bit) return h;
    return (h & 0x7fffu) == 0 || fabsf(x) > fabsf(__half2float(n)) ? h + 1 : h - 1;
}
// Clips to fp16's range; true if anything was outside it.
__device__ __forceinline__ bool clip_half(float &x) {
    const bool out = fabsf(x) > kHalfMax;
    if (out) x = copysignf(kHalfMax, x);
    return out;
}

// For the products' warp after a wait that gave up: it goes on over what memory holds, with waits that return
// at once, and frees slots whose copies may not have landed. So it first waits (bounded) until the
// copying warp, which sees the flag too, fills no more of them. (Stopping the products instead cost 1 to 2%.)
__device__ __forceinline__ void await_stop(volatile int *copies_end, unsigned long long limit_ns) {
    const unsigned long long t0 = globaltimer_ns();
    while (!__any_sync(0xffffffffu, *copies_end || globaltimer_ns() - t0 > 2 * limit_ns)) {
    }
    __syncwarp();
}

struct PrefillParams {
    const __nv_bfloat16 *q, *c;
    __nv_bfloat16 *pool, *o;
    const int32_t *prefix_lens, *prompt_lens, *page_table;
    int B, T, H, dc, max_prefix, n_pages, max_pages;
    int s_pad;              // positions per sequence in the workspace, whole tiles
    int h0, heads;          // this launch's heads h0 .. h0 + heads - 1
    int splits, per_split;  // kernel 2: shares of the heads
    int n_qb;               // kernel 3: query blocks of 256
    float scale_log2, q_scale;  // scale * log2(e) without the power of two that the queries take
    __half *kr;             // [B][s_pad][64]
    __half *k, *v;          // [B][heads][s_pad][d]
    int skip_cta;                // of the launch: see CopySkip
    unsigned long long wait_ns;
};

// A sequence's cached positions and new tokens; both 0 if the lengths were refused.
struct Seq {
    int prefix, n, total;
    bool ok;
};
__device__ __forceinline__ Seq seq_of(const PrefillParams &p, int b) {
    Seq s;
    s.prefix = p.prefix_lens ? p.prefix_lens[b] : 0;
    s.n = p.prompt_lens ? p.prompt_lens[b] : p.T;
    s.ok = s.prefix >= 0 && s.prefix <= p.max_prefix && s.n >= 0 && s.n <= p.T;
    if (!s.ok) s.prefix = s.n = 0;
    s.total = s.n > 0 ? s.prefix + s.n : 0;  // nothing is attended without new tokens
    return s;
}
__device__ __forceinline__ int page_of(const PrefillParams &p, int b, int pos) {
    const int lp = pos / kPT;
    const int pg = lp < p.max_pages ? p.page_table[(size_t)b * p.max_pages + lp] : -1;
    return pg >= 0 && pg < p.n_pages ? pg : -1;
}

// ---- kernel 1: a warp per position ---------------------------------------------------------------
__global__ void __launch_bounds__(256) latent_rows_kernel(const PrefillParams p, int span) {
    griddep_wait();
    griddep_launch_dependents();  // not before: the next kernel reads W without waiting
    const int lane = threadIdx.x & 31, row_w = p.dc + kDR;
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int b = (int)(i / span), pos = (int)(i - (long long)b * span);
    if (b >= p.B) return;
    const Seq s = seq_of(p, b);
    if (!s.ok && pos == 0 && lane == 0) atomicOr(&g_err, HMD_DEVERR_SEQLEN);
    if (pos >= s.total) return;
    const int pg = page_of(p, b, pos);
    if (pg < 0 && lane == 0) atomicOr(&g_err, HMD_DEVERR_PAGE);
    __nv_bfloat16 *cached = p.pool + ((size_t)max(pg, 0) * kPT + pos % kPT) * row_w;
    const __nv_bfloat16 *src = cached;
    if (pos >= s.prefix) {
        src = p.c + ((size_t)b * p.T + pos - s.prefix) * row_w;
        if (pg >= 0)
            for (int c = lane * 8; c < row_w; c += 256)
                *reinterpret_cast<uint4 *>(cached + c) = *reinterpret_cast<const uint4 *>(src + c);
    }
    uint32_t kr = 0;
    if (pg >= 0 || src != cached) {
        const uint32_t x = *reinterpret_cast<const uint32_t *>(src + p.dc + lane * 2);
        float lo = bf16_lo(x), hi = bf16_hi(x);
        const bool out_lo = clip_half(lo), out_hi = clip_half(hi);
        if (out_lo || out_hi) atomicOr(&g_err, HMD_DEVWARN_RANGE);
        kr = pack_f16x2(lo, hi);
    }
    *reinterpret_cast<uint32_t *>(p.kr + ((size_t)b * p.s_pad + pos) * kDR + lane * 2) = kr;
}

// ---- kernel 2 ------------------------------------------------------------------------------------
constexpr int kExpandThreads = 320;
constexpr int kExpAcc = 2;  // accumulators of 128 columns, behind the latent rows' 256 in TMEM
struct ExpandSmem {
    static constexpr uint32_t W_STAGE = kBlk;  // a step's 128 rows of weights x 64 latent dims
    // The latent rows land in blocks 0-7 and go to TMEM; then all 14 blocks are stages of weights, of
    // which the first six have been loading meanwhile.
    static constexpr int NW = 14, EARLY = 6;
    static constexpr uint32_t OFF_MISC = NW * W_STAGE;
    static constexpr uint32_t BYTES = OFF_MISC + 512 + 1024;
    static constexpr uint32_t ALLOC = BYTES;   // one CTA per SM
    static constexpr int B_A = 0, B_MOVED = 1, B_WFULL = 2, B_WFREE = B_WFULL + NW, B_ACC = B_WFREE + NW,
                         B_READ = B_ACC + kExpAcc, B_END = B_READ + kExpAcc, N_BARS = B_END + 1;
    static constexpr uint32_t OFF_MAX = OFF_MISC + 448;  // [two sets of warps][two steps][four warps]
    static_assert(N_BARS * 8 + 12 <= 448, "barriers");
    __device__ static uint32_t stage(int w) { return (w < EARLY ? w + NW - EARLY : w - EARLY) * W_STAGE; }
};
static_assert(ExpandSmem::ALLOC <= 232448, "shared memory per CTA");

// Four lanes exchange pieces of 32 bytes: lane l's piece t becomes lane t's (of the four) piece l, so that
// with a row per lane a store of four lanes writes a whole line of 128 bytes.
__device__ __forceinline__ void transpose4(uint32_t (&blk)[4][8], int lane) {
#pragma unroll
    for (int bit = 1; bit < 4; bit *= 2) {
        const bool upper = lane & bit;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t & bit) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t &x = blk[t][j], &y = blk[t | bit][j];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x : y, bit);
                if (upper) x = got;
                else y = got;
            }
        }
    }
}
// A barrier of the four warps that store the same steps (set 0 or 1), and an OR over a predicate of theirs.
__device__ __forceinline__ bool bar_set_or(int set, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(1 + set)
        : "memory");
    return r != 0;
}
// 32 bytes to global memory, in one store if `whole` (then dst is 32-byte aligned, else 16)
__device__ __forceinline__ void store_32b(void *dst, const uint32_t (&v)[8], bool whole = true) {
    if (!whole) {
        static_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kExpandThreads, 1)
latent_kv_kernel(const __grid_constant__ CUtensorMap tmc, const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv, const PrefillParams p) {
    using SM = ExpandSmem;
    constexpr int STEPS = D / 64;  // steps of 128 columns a head: K and V of 64 dims at once, of 128 in turn
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(sm), bars = sb + SM::OFF_MISC;
    auto bar = [&](int i) { return bars + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + SM::OFF_MISC + 8 * SM::N_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + SM::OFF_MISC + 8 * SM::N_BARS + 4);
    volatile int *copies_end = abort_flag + 1;  // the copying warp asks for no more
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int tiles = p.s_pad / kTile, tile = blockIdx.x / p.splits;
    const int b = tile / tiles, pos0 = (tile - b * tiles) * kTile;
    const int ha = (blockIdx.x % p.splits) * p.per_split, hb = min(p.heads, ha + p.per_split);
    const int n_kc = p.dc / 64, n_steps = (hb - ha) * STEPS;
    // a CTA's heads, in an order that begins elsewhere for every tile
    auto head_of = [&](int st) { return ha + (st / STEPS + tile) % (hb - ha); };
    const Seq s = seq_of(p, b);
    if (pos0 >= s.total || n_steps <= 0) {
        griddep_wait();
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < SM::N_BARS; ++i)
            mbar_init(bar(i), i >= SM::B_READ && i < SM::B_READ + kExpAcc ? 4 : i == SM::B_MOVED ? 8 : 1);
        // a test may have the first stage wait for bytes that no copy brings
        if ((int)blockIdx.x == p.skip_cta) mbar_expect_tx(bar(SM::B_WFULL), 16);
        fence_barrier_init();
        *abort_flag = 0;
        *copies_end = 0;
    }
    if (warp == 9) {
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    int n_loaded = 0;  // of warp 8: stages of weights

    if (warp == 8) {
        const bool lead = elect_one();
        const int n_all = n_steps * n_kc;
        int n = 0, w = 0, round = 0, st = 0, kc = 0, h = p.h0 + head_of(0);  // (no division per stage)
        auto load_w = [&] {
            const uint32_t dst = sb + SM::stage(w);
            mbar_expect_if(lead, bar(SM::B_WFULL + w), SM::W_STAGE);
            if (STEPS == 1 || st % 2 == 0)
                tma_load_3d_if(lead, dst, &tmk, bar(SM::B_WFULL + w), kc * 64, 0, h);
            if (STEPS == 1 || st % 2 == 1)
                tma_load_3d_if(lead, dst + (STEPS == 1 ? D * 128 : 0), &tmv, bar(SM::B_WFULL + w), kc * 64, 0, h);
            ++n;
            if (++w == SM::NW) {
                w = 0;
                ++round;
            }
            if (++kc == n_kc) {
                kc = 0;
                h = p.h0 + head_of(++st);
            }
        };
        while (n < SM::EARLY && n < n_all) load_w();
        griddep_wait();  // the appended rows are kernel 1's
        griddep_launch_dependents();
        // the tile's two pages of latent rows: blocks of 64 dims (a missing page's rows hold anything;
        // their results are stored as zeros)
        int pg[2];
        uint32_t bytes = 0;
        for (int h = 0; h < 2; ++h) {
            pg[h] = uniform(pos0 + h * kPT < s.total ? page_of(p, b, pos0 + h * kPT) : -1);
            if (pg[h] >= 0) bytes += n_kc * (kBlk / 2);
        }
        mbar_expect_if(lead, bar(SM::B_A), bytes);
        for (int kc = 0; kc < n_kc; ++kc)
            for (int h = 0; h < 2; ++h)
                tma_load_2d_if(lead && pg[h] >= 0, sb + kc * kBlk + h * (kBlk / 2), &tmc,
                               bar(SM::B_A), kc * 64, pg[h] * kPT);
        bool ok = true;
        while (n < n_all) {
            if (round > 0) ok = wait_warp(lead, bar(SM::B_WFREE + w), (round - 1) & 1, abort_flag, p.wait_ns);
            else if (n == SM::EARLY) ok = wait_warp(lead, bar(SM::B_MOVED), 0, abort_flag, p.wait_ns);
            if (!ok) break;
            load_w();
        }
        if (!ok && lead) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
        n_loaded = n;
        *copies_end = 1;
        __syncwarp();
    } else if (warp == 9) {
        const bool lead = elect_one();
        const Desc d_w(smem_desc_sw128(sb, 16, 1024));
        constexpr uint32_t ID = idesc_bf16(128, 128, 0, 0);
        auto wait = [&](int i, uint32_t parity) {
            if (!wait_warp(lead, bar(i), parity, abort_flag, p.wait_ns)) await_stop(copies_end, p.wait_ns);
        };
        griddep_wait();  // what the first wait is for comes after it: the kernel before is not part of its limit
        wait(SM::B_MOVED, 0);
        int w = 0, round = 0;
        for (int st = 0; st < n_steps; ++st) {
            const int acc = st % kExpAcc;
            if (st >= kExpAcc) wait(SM::B_READ + acc, (st / kExpAcc - 1) & 1);
            for (int kc = 0; kc < n_kc; ++kc) {
                wait(SM::B_WFULL + w, round & 1);
                tc_fence_after();
                const Desc wd = d_w.at(SM::stage(w));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_ts_if(lead, tmem + 256 + acc * 128, tmem + kc * 32 + kk * 8, wd.at(kk * 32), ID,
                               (kc > 0 || kk > 0) ? 1u : 0u);
                umma_commit_if(lead, bar(SM::B_WFREE + w));
                if (kc == n_kc - 1) umma_commit_if(lead, bar(SM::B_ACC + acc));
                if (++w == SM::NW) {
                    w = 0;
                    ++round;
                }
            }
        }
        if (lead) {
            if (*abort_flag) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
            umma_commit(bar(SM::B_END));  // every product is done before TMEM goes (bounded)
            (void)mbar_wait_bounded(bar(SM::B_END), 0);
        }
        __syncwarp();
    } else {
        // warps 0-3 store the even steps, 4-7 the odd ones; a lane has a position (its row of TMEM)
        griddep_wait();  // the workspace may still be read by the kernel before
        const int quarter = warp & 3, pos = pos0 + quarter * 32 + lane;
        const bool live = pos < s.total && page_of(p, b, pos) >= 0;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const bool lead = elect_one();
        bool out = false;
        // the latent rows to TMEM as the products' A operand, half of the dims per four warps
        wait_warp(lead, bar(SM::B_A), 0, abort_flag, p.wait_ns);
        if (!uniform(*abort_flag)) {
            const int row = quarter * 32 + lane;
            for (int kc = warp >> 2; kc < n_kc; kc += 2) {
                uint32_t x[32];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(&x[4 * j]) =
                        *reinterpret_cast<const uint4 *>(sm + kc * kBlk + row * 128 + ((j ^ (row & 7)) << 4));
                __syncwarp();
                tmem_st32(tmem + kc * 32 + lanes, x);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SM::B_MOVED));
        }
        for (int st = warp >> 2; st < n_steps; st += 2) {
            const int acc = st % kExpAcc;
            const bool ready = wait_warp(lead, bar(SM::B_ACC + acc), (st / kExpAcc) & 1, abort_flag, p.wait_ns);
            const bool values = STEPS == 1 || st % 2 == 1;  // the same in all steps of a set of warps
            if (!ready && !values) break;  // reported by the products' warp
            tc_fence_after();
            uint32_t r[2][64];  // 128 columns
            tmem_ld64(tmem + 256 + acc * 128 + lanes, r[0]);
            tmem_ld64(tmem + 256 + acc * 128 + 64 + lanes, r[1]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SM::B_READ + acc));  // the accumulator is free
            float big[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int j = 0; j < 64; ++j) big[c] = fmaxf(big[c], fabsf(__uint_as_float(r[c][j])));
                if (!live) big[c] = 0.f;
            }
            int e = 0;
            if (values) {
                // the values' power of two, from the tile's largest one
                volatile uint32_t *s_max = reinterpret_cast<volatile uint32_t *>(sm + SM::OFF_MAX) +
                                           (warp >> 2) * 8 + (st >> 1 & 1) * 4;
                const float mine = STEPS == 1 ? big[1] : fmaxf(big[0], big[1]);
                const uint32_t top_w = __reduce_max_sync(0xffffffffu, __float_as_uint(mine));
                if (lane == 0) s_max[quarter] = top_w;
                if (bar_set_or(warp >> 2, !ready)) break;  // reported by the products' warp; all four leave
                const uint32_t top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
                e = min(kMaxExp, max(0, 127 + 14 - (int)(top >> 23)) / kExpStep * kExpStep);
                const float f = pow2(e);
#pragma unroll
                for (int c = STEPS == 1 ? 1 : 0; c < 2; ++c) {
                    big[c] *= f;
#pragma unroll
                    for (int j = 0; j < 64; ++j) r[c][j] = __float_as_uint(__uint_as_float(r[c][j]) * f);
                }
            }
            uint32_t blk[2][4][8];  // as fp16: pieces of 32 bytes
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (big[c] > kHalfMax) {
                    out = true;
#pragma unroll
                    for (int j = 0; j < 64; ++j) {
                        float x = __uint_as_float(r[c][j]);
                        clip_half(x);
                        r[c][j] = __float_as_uint(x);
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    blk[c][j / 8][j % 8] =
                        live ? pack_f16x2(__uint_as_float(r[c][2 * j]), __uint_as_float(r[c][2 * j + 1])) : 0u;
                if (c == (STEPS == 1 ? 1 : 0) && values && quarter == 0 && lane == 0) {
                    const uint32_t code = (kMaxExp - e) / kExpStep;
                    uint32_t h[kExpBits];
#pragma unroll
                    for (int j = 0; j < kExpBits; ++j)
                        h[j] = half_with_last_bit(live ? __uint_as_float(r[c][j]) : 0.f, code >> j & 1u);
                    blk[c][0][0] = h[0] | h[1] << 16;
                    blk[c][0][1] = h[2] | (blk[c][0][1] & 0xffff0000u);
                }
                __syncwarp();
            }
            const size_t row0 = (((size_t)b * p.heads + head_of(st)) * p.s_pad + pos0 + quarter * 32 + (lane & ~3)) * D;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                transpose4(blk[c], lane);
                const bool key = STEPS == 2 ? st % 2 == 0 : c == 0;
                __half *dst = (key ? p.k : p.v) + row0 + (STEPS == 2 ? c * 64 : 0) + (lane & 3) * 16;
#pragma unroll
                for (int t = 0; t < 4; ++t) store_32b(dst + t * D, blk[c][t]);
            }
        }
        if (out) atomicOr(&g_err, HMD_DEVWARN_RANGE);
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 8 && lane == 0) {
        // the copies in flight land (bounded) before shared memory is released
        (void)mbar_wait_bounded(bar(SM::B_A), 0, p.wait_ns);
        for (int i = max(0, n_loaded - SM::NW); i < n_loaded; ++i)
            (void)mbar_wait_bounded(bar(SM::B_WFULL + i % SM::NW), (i / SM::NW) & 1, p.wait_ns);
    }
    if (*abort_flag && warp < 8) {
        // not all of these heads' keys and values are there: the attention leaves out what needs them
        for (int h = ha + tid; h < hb; h += 256)
            *reinterpret_cast<uint2 *>(p.v + (((size_t)b * p.heads + h) * p.s_pad + pos0) * D) =
                make_uint2(0x00010001u, 0x00000001u);
    }
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- kernel 3 ------------------------------------------------------------------------------------
constexpr int kSoftmax = 256;                  // softmax threads: two groups of four warps
constexpr int kAttThreads = kSoftmax + 64;     // + the MMA warp (8) and the TMA warp (9)
template <int D>
struct AttendSmem {
    static constexpr int KB = RingShape<D>::KB, VB = RingShape<D>::VB, NR = RingShape<D>::NR;
    static constexpr uint32_t Q_TILE = KB * kBlk;
    static constexpr uint32_t OFF_Q = 0, OFF_R = 2 * Q_TILE;
    static constexpr uint32_t OFF_BAR = OFF_R + NR * kBlk;
    static constexpr uint32_t BYTES = OFF_BAR + 256 + 1024;
    static constexpr uint32_t ALLOC = BYTES > 118784 ? BYTES : 118784;  // one CTA per SM
    // B_S, B_P, B_O: S_j complete, P_j written, O_j complete; B_SR: S read. Keys are free once the last
    // query tile's S is complete (all but their last block a little earlier, at B_K: a tile's values
    // take the place of its first keys), values once its O is. B_S, B_O and B_K are kRingPhases each,
    // for the key tiles in turn.
    static constexpr int B_FULL = 0, B_S = NR, B_O = B_S + 2 * kRingPhases, B_K = B_O + 2 * kRingPhases,
                         B_P = B_K + kRingPhases, B_SR = B_P + 2, B_Q = B_SR + 1, B_END = B_Q + 1,
                         N_BARS = B_END + 1;
    static_assert(N_BARS * 8 + 12 <= 256, "barriers");
    __device__ static int s(int j, int i) { return B_S + j * kRingPhases + ring_barrier(i); }
    __device__ static int o(int j, int i) { return B_O + j * kRingPhases + ring_barrier(i); }
    // in TMEM: O_0, O_1, S (both query tiles' in turn), P_0, P_1
    static constexpr uint32_t T_O = 0, T_S = 256, T_P = 384;
};
static_assert(AttendSmem<128>::ALLOC <= 232448, "shared memory per CTA");

template <int D>
__global__ void __launch_bounds__(kAttThreads, 1)
latent_attend_prompt_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                            const __grid_constant__ CUtensorMap tmr, const PrefillParams p) {
    using SM = AttendSmem<D>;
    constexpr int KB = SM::KB, VB = SM::VB, NR = SM::NR, NB = KB + VB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(sm), bars = sb + SM::OFF_BAR;
    auto bar = [&](int i) { return bars + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + SM::OFF_BAR + 8 * SM::N_BARS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + SM::OFF_BAR + 8 * SM::N_BARS + 4);
    volatile int *copies_end = abort_flag + 1;  // the copying warp asks for no more
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    // longest query blocks of all heads first (a wave of CTAs on a few heads' blocks of all lengths,
    // which keeps their keys in L2, ended 8% later)
    const int bh = blockIdx.x % (p.B * p.heads);
    const int qb = p.n_qb - 1 - (int)(blockIdx.x / (p.B * p.heads));
    const int b = bh / p.heads, hl = bh - b * p.heads, h = p.h0 + hl;
    griddep_launch_dependents();
    const Seq s = seq_of(p, b);
    const int t_first = qb * 2 * kTile, t_last = min(s.n, t_first + 2 * kTile) - 1;
    if (t_first >= s.n) {
        griddep_wait();
        return;
    }
    // key tiles of each query tile: up to its last row's position (none without rows)
    const int nt0 = uniform((s.prefix + min(t_last, t_first + kTile - 1)) / kTile + 1);
    const int nt1 = uniform(t_last >= t_first + kTile ? (s.prefix + t_last) / kTile + 1 : 0);
    const int n_tiles = max(nt0, nt1);
    if (tid == 0) {
        for (int i = 0; i < SM::N_BARS; ++i)
            mbar_init(bar(i), i == SM::B_Q ? 8 : (i == SM::B_P || i == SM::B_P + 1 || i == SM::B_SR) ? 4 : 1);
        // a test may have the first block wait for bytes that no copy brings
        if ((int)blockIdx.x == p.skip_cta) mbar_expect_tx(bar(SM::B_FULL), 16);
        fence_barrier_init();
        *abort_flag = 0;
        *copies_end = 0;
    }
    if (warp == 8) {
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    const int qt = (warp >> 2) & 1, row = tid & (kTile - 1);  // of a softmax thread
    const int t_row = t_first + qt * kTile + row;
    const bool row_ok = t_row <= t_last;
    const int pos_row = s.prefix + t_row;  // the row's position: its last key
    if (tid < kSoftmax) {
        // Q -> shared memory as fp16: consecutive threads take consecutive 16-byte chunks, all loads in
        // flight (with a row per thread it took 10 us of a CTA's 40)
        constexpr int CH = (D + kDR) / 8;
        bool out = false;
        uint4 x[CH];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int i = tid + kSoftmax * k, r = i / CH, c = i - r * CH;
            x[k] = t_first + r <= t_last
                       ? *reinterpret_cast<const uint4 *>(
                             p.q + (((size_t)b * p.T + t_first + r) * p.H + h) * (D + kDR) + c * 8)
                       : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int i = tid + kSoftmax * k, r = i / CH, c = i - r * CH;
            const uint32_t in[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo = bf16_lo(in[e]) * p.q_scale, hi = bf16_hi(in[e]) * p.q_scale;
                out |= clip_half(lo);
                out |= clip_half(hi);
                y[e] = pack_f16x2(lo, hi);
            }
            *reinterpret_cast<uint4 *>(sm + SM::OFF_Q + (r >> 7) * SM::Q_TILE + (c >> 3) * kBlk + (r & 127) * 128 +
                                       (((c & 7) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        if (out) atomicOr(&g_err, HMD_DEVWARN_RANGE);
        fence_proxy_async_smem();  // Q is read by the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SM::B_Q));
    }
    griddep_wait();  // keys and values are kernel 2's

    const int last = nt1 > 0;  // the last query tile
    int n_loaded = 0;          // of warp 9: blocks
    if (warp == 9) {
        // ===== copies: the blocks of K_0, K_1, V_0, K_2, V_1, ... in the order of their use, block n into
        // slot n % NR (the warp converged) ========================================================
        const bool lead = elect_one();
        RingPlace<D> at, old;  // the block to load, the one whose slot it takes
        bool ok = true;
        int n = 0, slot = 0;
        for (; n < n_tiles * NB; ++n) {
            if (n >= NR) {
                const int i = old.tile(n_tiles);
                const RingFree by = old.freed_by(n_tiles);
                const int free = by == kFreeOutput ? SM::o(last, i) : by == kFreeKeys ? SM::B_K + ring_barrier(i)
                                                                                      : SM::s(last, i);
                ok = wait_warp(lead, bar(free), ring_parity(i), abort_flag, p.wait_ns);
                if (!ok) break;
                old.next(n_tiles);
            }
            const uint32_t dst = sb + SM::OFF_R + slot * kBlk, fb = bar(SM::B_FULL + slot);
            mbar_expect_if(lead, fb, kBlk);
            const bool key = at.key(n_tiles);
            const int u = at.block(n_tiles), row0 = at.tile(n_tiles) * kTile;
            if (key && u < KB - 1) tma_load_3d_if(lead, dst, &tmk, fb, u * 64, row0, bh);
            else if (key) tma_load_3d_if(lead, dst, &tmr, fb, 0, row0, b);
            else tma_load_3d_if(lead, dst, &tmv, fb, u * 64, row0, bh);
            at.next(n_tiles);
            if (++slot == NR) slot = 0;
        }
        if (!ok && lead) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
        n_loaded = n;
        *copies_end = 1;
        __syncwarp();
    } else if (warp == 8) {
        // ===== products: S_0(i+1), O_0(i), S_1(i+1), O_1(i) (the warp converged). A tile's scores are
        // complete before its softmax is done with the tile before, so both softmax groups and the tensor
        // core always have work; one S serves both, since it is read into registers at once =======
        const bool lead = elect_one();
        const Desc d_q(smem_desc_sw128(sb + SM::OFF_Q, 16, 1024));
        const Desc d_k(smem_desc_sw128(sb + SM::OFF_R, 16, 1024));
        const Desc d_v(smem_desc_sw128(sb + SM::OFF_R, kBlk, 1024));
        constexpr uint32_t ID_S = idesc_f16(128, kTile, 0, 0);
        constexpr uint32_t ID_O = idesc_f16(128, D, 0, 1), ID_O64 = idesc_f16(128, 64, 0, 1);
        int n_s = 0;  // scores issued
        // lanes 0 .. count - 1 wait for blocks n .. n + count - 1 of the stream, lane `count` for barrier i
        // (i < 0: for blocks only)
        auto wait_for = [&](int n, int count, int i, int parity) {
            const int u = n + lane;
            const bool block = lane < count;
            if (!wait_warp(block || (lane == count && i >= 0), bar(block ? SM::B_FULL + u % NR : max(i, 0)),
                           (block ? u / NR : parity) & 1, abort_flag, p.wait_ns))
                await_stop(copies_end, p.wait_ns);
            tc_fence_after();
        };
        auto issue_s = [&](int j, int i) {  // S = Q_j K_i^T
            const int n = ring_key<D>(i);
            wait_for(n, j == 0 || i >= nt0 ? KB : 0, n_s > 0 ? SM::B_SR : -1, n_s - 1);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                const Desc k = d_k.at(((uint32_t)(n + kb) % NR) * kBlk);
                const Desc q = d_q.at(j * SM::Q_TILE + kb * kBlk);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_if(lead, tmem + SM::T_S, q.at(kk * 32), k.at(kk * 32), ID_S, (kb > 0 || kk > 0) ? 1u : 0u);
                if (kb == KB - 2) umma_commit_if(lead && j == last, bar(SM::B_K + ring_barrier(i)));
            }
            umma_commit_if(lead, bar(SM::s(j, i)));
            ++n_s;
        };
        auto issue_o = [&](int j, int i) {  // O_j (+)= P_j V_i, P_j from TMEM
            const int n = ring_value<D>(i, n_tiles);
            wait_for(n, j == 0 || i >= nt0 ? VB : 0, SM::B_P + j, i);
            const uint32_t slot = (uint32_t)n % NR;
            const uint32_t o = tmem + SM::T_O + 128 * j, pj = tmem + SM::T_P + 64 * j;
            const Desc v = d_v.at(slot * kBlk);
            const uint32_t more = i > 0 ? 1u : 0u;
            if (VB == 1 || slot + 1 < NR) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_ts_if(lead, o, pj + 8 * kk, v.at(kk * 2048), ID_O, kk > 0 ? 1u : more);
            } else {  // the tile's second block is at the ring's start: 64 dims at a time
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_ts_if(lead, o, pj + 8 * kk, v.at(kk * 2048), ID_O64, kk > 0 ? 1u : more);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    umma_ts_if(lead, o + 64, pj + 8 * kk, d_v.at(kk * 2048), ID_O64, kk > 0 ? 1u : more);
            }
            umma_commit_if(lead, bar(SM::o(j, i)));
        };
        if (!wait_warp(lead, bar(SM::B_Q), 0, abort_flag, p.wait_ns)) await_stop(copies_end, p.wait_ns);
        for (int i = -1; i < n_tiles; ++i) {
            if (i + 1 < nt0) issue_s(0, i + 1);
            if (i >= 0 && i < nt0) issue_o(0, i);
            if (i + 1 < nt1) issue_s(1, i + 1);
            if (i >= 0 && i < nt1) issue_o(1, i);
        }
        if (lead) {
            if (*abort_flag) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
            umma_commit(bar(SM::B_END));  // every product is done before TMEM goes (bounded)
            (void)mbar_wait_bounded(bar(SM::B_END), 0);
        }
        __syncwarp();
    } else if ((qt ? nt1 : nt0) > 0) {
        // ================= softmax: query tile qt, one thread per row ==========================
        const int nt = qt ? nt1 : nt0;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_col = lane_base + SM::T_S, p_col = lane_base + SM::T_P + 64 * qt,
                       o_col = lane_base + SM::T_O + 128 * qt;
        const bool lead = elect_one();
        float m_base = -INFINITY, l_run = 0.f;
        // The values of the tile at hand are times 2^e: exponents are lower by e and the sum is times 2^-e, so
        // that nothing is to be done while e stays. `mixed`: it does not, and its bits are read a tile
        // ahead, a lane each.
        const __half *v0 = p.v + (size_t)bh * p.s_pad * D;
        auto e_of = [](uint32_t code) { return kMaxExp - kExpStep * (int)code; };
        uint32_t c_min = ~0u, c_max = 0;
#pragma unroll 4
        for (int i = lane; i < nt; i += 32) {
            const uint2 v = *reinterpret_cast<const uint2 *>(v0 + (size_t)i * kTile * D);
            const uint32_t code = (v.x & 1u) | (v.x >> 15 & 2u) | (v.y & 1u) << 2;
            c_min = min(c_min, code);
            c_max = max(c_max, code);
        }
        c_min = __reduce_min_sync(0xffffffffu, c_min);
        c_max = __reduce_max_sync(0xffffffffu, c_max);
        int e = e_of(c_min);
        auto attend = [&](auto mixed) {
            const unsigned short *e_at = reinterpret_cast<const unsigned short *>(v0) + (lane & 3);
            uint32_t e_bit = 0;
            if constexpr (decltype(mixed)::value) e_bit = *e_at;
            for (int i = 0; i < nt; ++i) {
                if constexpr (decltype(mixed)::value) {
                    const int e_i = e_of(__ballot_sync(0xffffffffu, e_bit & 1u) & ((1u << kExpBits) - 1));
                    if (i + 1 < nt) e_bit = e_at[(size_t)(i + 1) * kTile * D];
                    m_base += (float)(e_i - e);
                    l_run *= pow2(e - e_i);
                    e = e_i;
                }
                wait_warp(lead, bar(SM::s(qt, i)), ring_parity(i), abort_flag, p.wait_ns);
                tc_fence_after();
                float x[kTile];
                {
                    uint32_t r[64];
                    tmem_ld64(s_col, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 64; ++j) x[j] = __uint_as_float(r[j]);
                    tmem_ld64(s_col + 64, r);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(SM::B_SR));  // S may be the other query tile's now
#pragma unroll
                    for (int j = 0; j < 64; ++j) x[64 + j] = __uint_as_float(r[j]);
                }
                const int j0 = i * kTile;
                if (!(row_ok && j0 + kTile - 1 <= pos_row)) {
#pragma unroll
                    for (int j = 0; j < kTile; ++j) x[j] = (row_ok && j0 + j <= pos_row) ? x[j] : -INFINITY;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // short chains
#pragma unroll
                for (int j = 0; j < kTile; j += 8) {
                    mx4[0] = max3(mx4[0], x[j], x[j + 1]);
                    mx4[1] = max3(mx4[1], x[j + 2], x[j + 3]);
                    mx4[2] = max3(mx4[2], x[j + 4], x[j + 5]);
                    mx4[3] = max3(mx4[3], x[j + 6], x[j + 7]);
                }
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
                const bool move = mx > m_base + kTop;
                float f = 1.f;  // factor of the row's earlier output and sum
                if (move) {
                    const float to = mx - kFresh;
                    f = exp2f(m_base - to);  // 0 while the row had no key (m_base = -inf)
                    m_base = to;
                    l_run *= f;
                }
                const float mu = (m_base == -INFINITY) ? 0.f : m_base;
                uint32_t pk[kTile / 32][16];  // P, two keys a word
                {
                    const uint64_t sc2 = f2(p.scale_log2, p.scale_log2), nmu2 = f2(-mu, -mu);
                    uint64_t acc[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < kTile / 32; ++c) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            const uint64_t y = f2_fma(f2(x[c * 32 + 2 * u], x[c * 32 + 2 * u + 1]), sc2, nmu2);
                            uint64_t e;
                            if ((u & 3) == 3) {
                                e = exp2_fma_x2(y);
                            } else {
                                float a0, a1;
                                f2_split(y, a0, a1);
                                e = f2(ex2_approx(a0), ex2_approx(a1));
                            }
                            acc[u & 1] = f2_add(acc[u & 1], e);
                            float e0, e1;
                            f2_split(e, e0, e1);
                            pk[c][u] = pack_f16x2(e0, e1);
                        }
                    }
                    float a0, a1, b0, b1;
                    f2_split(acc[0], a0, a1);
                    f2_split(acc[1], b0, b1);
                    l_run += (a0 + a1) + (b0 + b1);
                }
                // the product before has read P and added to O: the row's earlier output to the new base, then P
                if (i > 0) wait_warp(lead, bar(SM::o(qt, i - 1)), ring_parity(i - 1), abort_flag, p.wait_ns);
                tc_fence_after();
                __syncwarp();  // the row-dependent branches above rejoin before the TMEM accesses
                if (__any_sync(0xffffffffu, move) && i > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t r[32];
                        tmem_ld32(o_col + 32 * c, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f);
                        tmem_st32(o_col + 32 * c, r);
                    }
                }
#pragma unroll
                for (int c = 0; c < kTile / 32; ++c) tmem_st16(p_col + 16 * c, pk[c]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(SM::B_P + qt));
            }
        };
        // (kernel 2 gave up on a tile: this CTA does too. Kept in a register of the loop, for the query tile
        // alone, it was 1% of the kernel.)
        if (c_max == kMissing) *abort_flag = 1;
        if (c_min == c_max) attend(std::false_type());
        else attend(std::true_type());
        wait_warp(lead, bar(SM::o(qt, nt - 1)), ring_parity(nt - 1), abort_flag, p.wait_ns);
        const bool ok = __all_sync(0xffffffffu, *abort_flag == 0);
        if (ok) {
            tc_fence_after();
            const float inv = l_run > 0.f ? pow2(-e) / l_run : 0.f;
            const int t0 = t_first + qt * kTile + (row & ~3);
            const bool whole = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0;
            __nv_bfloat16 *dst = p.o + (((size_t)b * p.T + t0) * p.H + h) * D + (lane & 3) * 16;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                __syncwarp();  // converged for the TMEM loads after the row-dependent stores
                uint32_t blk[4][8];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t r[32];
                    tmem_ld32(o_col + 64 * c + 32 * half, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        blk[half * 2 + j / 8][j % 8] = pack_bf16x2(__uint_as_float(r[2 * j]) * inv,
                                                                   __uint_as_float(r[2 * j + 1]) * inv);
                }
                transpose4(blk, lane);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t0 + t <= t_last) store_32b(dst + (size_t)t * p.H * D + 64 * c, blk[t], whole);
            }
        } else if (lane == 0) {
            atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 9 && lane == 0) {
        // the copies in flight land (bounded) before shared memory is released
        for (int i = max(0, n_loaded - NR); i < n_loaded; ++i)
            (void)mbar_wait_bounded(bar(SM::B_FULL + i % NR), (i / NR) & 1, p.wait_ns);
    }
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- host side -----------------------------------------------------------------------------------
size_t padded(int T, int max_prefix) {
    return ((size_t)T + max_prefix + kTile - 1) / kTile * kTile;
}

template <int D>
cudaError_t launch_d(const LatentPrefillArgs &a, cudaStream_t s) {
    const cudaError_t attr_err = once_per_device([] {
        cudaError_t e = cudaFuncSetAttribute(latent_kv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)ExpandSmem::ALLOC);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(latent_attend_prompt_kernel<D>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AttendSmem<D>::ALLOC);
        return e;
    });
    if (attr_err != cudaSuccess) return attr_err;
    PrefillParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.c = static_cast<const __nv_bfloat16 *>(a.c);
    p.pool = static_cast<__nv_bfloat16 *>(a.pool);
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.prefix_lens = a.prefix_lens; p.prompt_lens = a.prompt_lens; p.page_table = a.page_table;
    p.B = a.B; p.T = a.T; p.H = a.H; p.dc = a.d_c;
    p.max_prefix = a.prefix_lens ? a.max_prefix : 0;
    p.n_pages = a.n_pages; p.max_pages = a.max_pages;
    const size_t s_pad = padded(a.T, p.max_prefix);
    p.s_pad = (int)s_pad;
    p.n_qb = (a.T + 2 * kTile - 1) / (2 * kTile);
    p.q_scale = a.scale >= 2.f ? exp2f((float)std::ilogb(a.scale)) : 1.f;
    p.scale_log2 = a.scale / p.q_scale * 1.4426950408889634f;
    // the workspace: k_r of every position, then K and V of as many heads as fit
    const size_t kr_bytes = (size_t)a.B * s_pad * kDR * 2, head_bytes = (size_t)a.B * s_pad * D * 2 * 2;
    const int fit = (int)std::min<size_t>((size_t)a.H, (a.ws_bytes - kr_bytes) / head_bytes);
    const int n_groups = (a.H + fit - 1) / fit, group = (a.H + n_groups - 1) / n_groups;
    p.kr = static_cast<__half *>(a.workspace);
    p.k = p.kr + kr_bytes / 2;
    CUtensorMap tmc, tmuk, tmuv, tmr;
    if (!make_tmap_pool_sw128(&tmc, a.pool, a.n_pages, 1, a.d_c + kDR) ||
        !make_tmap_blocks_sw128(&tmuk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w_uk, a.H, a.w_uk_head, D, a.d_c, D) ||
        !make_tmap_blocks_sw128(&tmuv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w_uv, a.H, a.w_uv_head, D, a.d_c, D) ||
        !make_tmap_blocks_sw128(&tmr, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.kr, a.B, (long long)s_pad * kDR,
                                (long long)s_pad, kDR, kTile))
        return cudaErrorInvalidValue;
    const int span = a.T + p.max_prefix;
    cudaError_t e = launch_pdl(latent_rows_kernel, dim3((unsigned)(((long long)a.B * span + 7) / 8)), dim3(256),
                               0, s, p, span);
    for (int h0 = 0; h0 < a.H && e == cudaSuccess; h0 += group) {
        p.h0 = h0;
        p.heads = std::min(group, a.H - h0);
        p.v = p.k + (size_t)a.B * p.heads * s_pad * D;
        const CopySkip none;
        const CopySkip &skip_kv = h0 == 0 ? a.skip_kv : none, &skip_prompt = h0 == 0 ? a.skip_prompt : none;
        p.skip_cta = skip_kv.cta; p.wait_ns = skip_kv.wait_ns;
        // shares of the heads per position tile: the fewest rounds of CTAs, each costing its heads
        // and about one more for loading the tile's latent rows
        const long long tiles = (long long)a.B * (s_pad / kTile), sms = sm_count();
        long long best = -1;
        for (int n = 1; n <= p.heads; ++n) {
            const int per = (p.heads + n - 1) / n;
            const long long cost = (tiles * n + sms - 1) / sms * (per + 1);
            if (best < 0 || cost < best) {
                best = cost;
                p.splits = n;
                p.per_split = per;
            }
        }
        CUtensorMap tmk, tmv;
        const long long bh = (long long)a.B * p.heads;
        if (!make_tmap_blocks_sw128(&tmk, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.k, bh, (long long)s_pad * D,
                                    (long long)s_pad, D, kTile) ||
            !make_tmap_blocks_sw128(&tmv, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.v, bh, (long long)s_pad * D,
                                    (long long)s_pad, D, kTile))
            return cudaErrorInvalidValue;
        e = launch_pdl(latent_kv_kernel<D>, dim3((unsigned)(tiles * p.splits)), dim3(kExpandThreads),
                       ExpandSmem::ALLOC, s, tmc, tmuk, tmuv, p);
        if (e != cudaSuccess) break;
        p.skip_cta = skip_prompt.cta; p.wait_ns = skip_prompt.wait_ns;
        e = launch_pdl(latent_attend_prompt_kernel<D>, dim3((unsigned)(p.n_qb * bh)), dim3(kAttThreads),
                       AttendSmem<D>::ALLOC, s, tmk, tmv, tmr, p);
    }
    return e;
}

}  // namespace

size_t latent_prefill_ws_bytes(int B, int T, int heads, int d, int max_prefix) {
    return (size_t)B * padded(T, max_prefix) * (kDR + 2 * (size_t)d * heads) * 2;
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs &a, cudaStream_t s) {
    return a.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

uint32_t latent_prefill_read_errors(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_err, sizeof v) != cudaSuccess) return 0;
    if (clear && v) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_err, &z, sizeof z);
    }
    return v;
}

}  // namespace hmd
