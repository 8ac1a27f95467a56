// Latent attention, absorbed form: n_q new tokens per sequence against a paged cache of latent
// rows.
//
// A cached token is one row [c (d_c) ; k_r (64)] shared by every head. Head h's key is
// [W_uk[h] c ; k_r], its value W_uv[h] c. Since (W_uk[h] c) . q = c . (W_uk[h]^T q), the query is
// brought to the latent space once and the cache is read as it is:
//   q~ = W_uk[h]^T q_nope,  s_j = scale (q~ . c_j + q_r . k_rj),  o = W_uv[h] sum_j p_j c_j.
// Every row (token i, head h) of a sequence attends the same latent rows, so the step is bound by
// reading the cache once: (d_c + 64) * 2 bytes a token for all heads.
//
// Kernel 1 (absorb): q~ = W_uk^T q on mma.sync (16 rows of tokens at a time: at most a few hundred
// MFLOP, bound by reading W_uk once), scaled by scale * log2(e), split into a bf16 pair
// q~ = hi + lo and stored as the image kernel 2 wants. Rounding q~ to one bf16 would put an error of
// up to 2^-8 |s| on every score; the pair leaves 2^-16, and its second half rides along in lanes of the
// tensor core that would be idle. It also appends the new latent rows to the cache and lays out the
// schedule (running page counts of the batch). 8 us for 32 heads, d = 128, d_c = 512, 32 or 48 tokens.
// Kernel 2 (attention): the batch's pages, laid end to end, are cut into equal ranges, one per
// SM (times the row groups of 32 rows), whatever the lengths are; a CTA's range may end one
// sequence and begin another. Per page of 64 keys:
//     S   [32 hi, 32 lo rows x 64 keys] = [q~hi ; q~lo] C^T   tcgen05, M = 128, N = 64, q~ in TMEM
//     O^T [d_c x 32 rows] += C^T [d_c x 64 keys] P^T          tcgen05, M = 128, N = 32
// both from the same shared-memory tile of C (K-major, then MN-major). The few rows are the N of the
// second product, so that its accumulator fits TMEM beside the queries, and only pages are left in
// shared memory: three of 72 KiB are in flight or in use, which is what covers HBM's latency (two, with
// the queries in shared memory as well, reached 4.5 TB/s). Warp-specialised: warp 4 streams pages
// by TMA (units of 128 dims, each freed as soon as its product is done), warps 5 and 6 issue the two
// products, warps 0-3 are the softmax. O^T accumulates at an exponent base per row that moves only when the
// row's scores exceed it by more than 2^8 (then O^T is rescaled in TMEM). B = 32, 32 heads, 4096 to
// 8192 keys: 48 us, 226 MB, 4.7 TB/s (its start and the wait for kernel 1 are 7 us; in the 41 after them
// 5.5 TB/s, where the FA decode reaches 6.5). With 96 rows a sequence (three groups, B = 16, 2048 to 4097 keys) 34 us,
// bound by the tensor core: a page costs 36 products of 48 cycles (N = 64) and 16 of 40 for 32 rows.
// Kernel 3 (merge and expand), one CTA per (head, 16 or 32 tokens): joins the ranges' partial sums
// while W_uv[h] is copied to shared memory (asked for while kernel 2 ends: 69.6 -> 67.8 us for the batch
// above), and multiplies by it (mma.sync, the latent output as a bf16 pair). Bound by latency: one
// pass over the partial sums, one over W_uv; about 11 us.
#include <cuda.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "softmax.cuh"
#include "../../include/hmd.h"

namespace hmd {
namespace {

__device__ unsigned int g_err;

constexpr int kPT = 64;        // tokens per page = keys per tile
constexpr int kDR = 64;        // the rows' part shared as it is by every head's key
constexpr int kRows = 32;      // query rows (token, head) per group
constexpr uint32_t kBlk = 8192;  // one [64 rows][128 B] block, 128-byte swizzle
constexpr float kLazy = 8.f;   // log2 headroom before a row's exponent base moves

// byte offset of the 16-byte chunk holding (row, col..col+7) of a [64 rows][64 cols] bf16 block
__device__ __forceinline__ uint32_t blk_off(int row, int col) {
    return (uint32_t)(row * 128 + (((col >> 3) ^ (row & 7)) << 4));
}

struct LatentParams {
    const __nv_bfloat16 *q, *new_c, *w_uk, *w_uv;
    __nv_bfloat16 *pool, *o;
    long long w_uk_head, w_uv_head;  // elements from one head's weights to the next
    const int32_t *page_table, *seq_lens;
    int B, nq, H, d, dc, n_pages, max_pages, max_seq_len;
    int n_groups, n_ranges;
    float scale_log2;
    uint8_t *q_img;  // [B][n_groups][dc / 64 + 1 blocks] of 64 rows: 32 hi, 32 lo
    float *part_o;   // [n_ranges + B][n_groups][32][dc], see part_index
    float *part_ml;  // [n_ranges + B][n_groups][32][2]: exponent base, sum (-1: range gave up)
    int32_t *cum;    // [B + 1] pages before each sequence (kernel 1's own, for large batches)
    int4 *start;     // [n_ranges + 1]: a range's first page, its sequence, that sequence's first page
                     // and its length
    int2 *ranges;    // [B]: a sequence's ranges [x, y)
    int skip_cta;    // of kernel 2: see CopySkip
    unsigned long long wait_ns;
};

// Pages of a sequence: none for an unused row or a length that is refused.
__device__ __forceinline__ int pages_of(const LatentParams &p, int L) {
    return L >= p.nq && L <= p.max_seq_len ? (L + kPT - 1) / kPT : 0;
}

// Range i < n covers the flat pages [i P / n, (i + 1) P / n), n = min(n_ranges, P), so none is
// empty. Ranges and sequences both grow along the pages, so (range + sequence) is different for
// every piece of a sequence in a range.
__device__ __forceinline__ int range_begin(int i, int P, int n) {
    return (int)((long long)i * P / n);
}
__device__ __forceinline__ int range_of(int page, int P, int n) {
    return (int)((((long long)page + 1) * n - 1) / P);  // P > 0
}
__device__ __forceinline__ size_t part_index(const LatentParams &p, int range, int b, int group) {
    return (size_t)(range + b) * p.n_groups + group;
}

// ---- kernel 1 ----------------------------------------------------------------------------------
constexpr int kAbsThreads = 128;
constexpr int kAbsTok = 32;  // tokens (b, i) per CTA
template <int D>
struct AbsSmem {
    static constexpr int QP = D + 8, WP = 128 + 8;  // pitches (elements) without bank conflicts
    __nv_bfloat16 q[kAbsTok][QP];
    __nv_bfloat16 w[D][WP];
};

// The last block: lengths to running page counts, the ranges' first pages and the sequences' ranges.
// s_cum: room for kCumShared counts in shared memory, where the search reads them (a larger batch's
// are read from global memory).
constexpr int kCumShared = 4096;
__device__ void schedule_block(const LatentParams &p, int32_t *s_cum) {
    __shared__ int warp_sum[kAbsThreads / 32];
    const bool in_shared = p.B < kCumShared;
    int32_t *cum = in_shared ? s_cum : p.cum;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int base = 0;
    if (tid == 0) cum[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAbsThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < p.B) {
            const int L = p.seq_lens[b];
            n = pages_of(p, L);
            if (n == 0 && L != 0) atomicOr(&g_err, HMD_DEVERR_SEQLEN);
        }
        int sum = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += up;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        for (int v = 0; v < warp; ++v) sum += warp_sum[v];
        if (b < p.B) cum[b + 1] = base + sum;
        for (int v = 0; v < kAbsThreads / 32; ++v) base += warp_sum[v];
        __syncthreads();
    }
    const int P = base, n_live = min(p.n_ranges, P);
    for (int i = tid; i <= p.n_ranges; i += kAbsThreads) {
        int4 st = make_int4(P, 0, 0, 0);
        if (i < n_live) {
            // the last sequence whose pages start at or before the range's first page
            st.x = range_begin(i, P, n_live);
            int lo = 0, hi = p.B;  // cum[lo] <= st.x < cum[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (cum[mid] <= st.x) lo = mid;
                else hi = mid;
            }
            st = make_int4(st.x, lo, cum[lo], p.seq_lens[lo]);
        }
        p.start[i] = st;
    }
    for (int b = tid; b < p.B; b += kAbsThreads) {
        const int c0 = cum[b], c1 = cum[b + 1];
        p.ranges[b] = c1 > c0 ? make_int2(range_of(c0, P, n_live), range_of(c1 - 1, P, n_live) + 1)
                              : make_int2(0, 0);
    }
}

static_assert(sizeof(AbsSmem<64>) >= kCumShared * sizeof(int32_t), "the schedule's counts fit");
template <int D>
__global__ void __launch_bounds__(kAbsThreads) latent_absorb_kernel(const LatentParams p) {
    extern __shared__ __align__(16) uint8_t abs_smem[];
    AbsSmem<D> &sm = *reinterpret_cast<AbsSmem<D> *>(abs_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int n_tok = p.B * p.nq, dq = D + kDR, row_w = p.dc + kDR;
    if (blockIdx.x == gridDim.x - 1) {
        schedule_block(p, reinterpret_cast<int32_t *>(abs_smem));
        return;
    }
    const int n_app = (n_tok + kAbsThreads / 32 - 1) / (kAbsThreads / 32);
    if (blockIdx.x >= gridDim.x - 1 - n_app) {
        // append: a warp copies the row of token (b, i) to position L - nq + i
        const int tok = (blockIdx.x - (gridDim.x - 1 - n_app)) * (kAbsThreads / 32) + warp;
        if (tok >= n_tok) return;
        const int b = tok / p.nq, L = p.seq_lens[b];
        if (L < p.nq || L > p.max_seq_len) return;
        const int pos = L - p.nq + (tok - b * p.nq);
        const int pg = p.page_table[(size_t)b * p.max_pages + pos / kPT];
        if (pg < 0 || pg >= p.n_pages) {
            if (lane == 0) atomicOr(&g_err, HMD_DEVERR_PAGE);
            return;
        }
        __nv_bfloat16 *dst = p.pool + ((size_t)pg * kPT + pos % kPT) * row_w;
        for (int c = lane * 8; c < row_w; c += 256)
            *reinterpret_cast<uint4 *>(dst + c) =
                *reinterpret_cast<const uint4 *>(p.new_c + (size_t)tok * row_w + c);
        return;
    }
    const int n_cols = p.dc / 128;
    const int cc = blockIdx.x % n_cols, h = (blockIdx.x / n_cols) % p.H;
    const int tok0 = blockIdx.x / (n_cols * p.H) * kAbsTok;
    const int rows = min(kAbsTok, n_tok - tok0);
    // operands to shared memory, all copies in flight at once
    const __nv_bfloat16 *w = p.w_uk + h * p.w_uk_head + cc * 128;
    for (int idx = tid; idx < D * 16; idx += kAbsThreads) {
        const int n = idx >> 4, c = (idx & 15) * 8;
        cp_async16(smem_u32(&sm.w[n][c]), w + (size_t)n * p.dc + c);
    }
    for (int idx = tid; idx < kAbsTok * (D / 8); idx += kAbsThreads) {
        const int r = idx / (D / 8), c = idx % (D / 8) * 8;
        if (r < rows) cp_async16(smem_u32(&sm.q[r][c]), p.q + ((size_t)(tok0 + r) * p.H + h) * dq + c);
        else *reinterpret_cast<uint4 *>(&sm.q[r][c]) = make_uint4(0, 0, 0, 0);
    }
    const size_t img_bytes = (size_t)(p.dc / 64 + 1) * kBlk;
    // image address of (token, head) row r of group r / 32, in the block of dims col..
    auto img = [&](int tok, int hh, int col, bool lo) {
        const int b = tok / p.nq, r = (tok - b * p.nq) * p.H + hh;
        return p.q_img + ((size_t)b * p.n_groups + r / kRows) * img_bytes + (size_t)(col >> 6) * kBlk +
               blk_off(r % kRows + (lo ? kRows : 0), col & 63) + (col & 7) * 2;
    };
    if (cc == 0) {
        // the queries' shared part, 8 dims a thread
        for (int idx = tid; idx < rows * (kDR / 8); idx += kAbsThreads) {
            const int tok = tok0 + idx / (kDR / 8), c = idx % (kDR / 8) * 8;
            const uint4 in = *reinterpret_cast<const uint4 *>(p.q + ((size_t)tok * p.H + h) * dq + D + c);
            const uint32_t x[4] = {in.x, in.y, in.z, in.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x0 = bf16_lo(x[e]) * p.scale_log2, x1 = bf16_hi(x[e]) * p.scale_log2;
                hi[e] = pack_bf16x2(x0, x1);
                lo[e] = pack_bf16x2(x0 - bf16_lo(hi[e]), x1 - bf16_hi(hi[e]));
            }
            *reinterpret_cast<uint4 *>(img(tok, h, p.dc + c, false)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(img(tok, h, p.dc + c, true)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    cp_async_wait_all();
    __syncthreads();
    // 32 tokens x 128 latent dims: a warp takes 32 of the dims
    float acc[2][4][4] = {};
    const int mi = lane >> 3;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t a[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
            ldmatrix_x4(smem_u32(&sm.q[m * 16 + (lane & 15)][kk * 16 + (lane >> 4) * 8]), a[m][0],
                        a[m][1], a[m][2], a[m][3]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint32_t b0, b1, b2, b3;
            ldmatrix_x4_trans(smem_u32(&sm.w[kk * 16 + ((mi & 1) << 3) + (lane & 7)]
                                           [warp * 32 + n * 16 + ((mi >> 1) << 3)]),
                              b0, b1, b2, b3);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                mma_bf16_16816(acc[m][2 * n], a[m], b0, b1);
                mma_bf16_16816(acc[m][2 * n + 1], a[m], b2, b3);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = m * 16 + (lane >> 2) + 8 * e;
                if (r >= rows) continue;
                const int col = cc * 128 + warp * 32 + n * 8 + (lane & 3) * 2;
                const float x0 = acc[m][n][2 * e] * p.scale_log2, x1 = acc[m][n][2 * e + 1] * p.scale_log2;
                const uint32_t hi = pack_bf16x2(x0, x1);
                *reinterpret_cast<uint32_t *>(img(tok0 + r, h, col, false)) = hi;
                *reinterpret_cast<uint32_t *>(img(tok0 + r, h, col, true)) =
                    pack_bf16x2(x0 - bf16_lo(hi), x1 - bf16_hi(hi));
            }
        }
    }
}

// ---- kernel 2 ----------------------------------------------------------------------------------
constexpr int kAttThreads = 224;  // softmax (warps 0-3), copies (4), scores (5), outputs (6)
// Shared memory for d_c = 128 * NP: a ring of page slots, P, barriers. A page is NP units of 128 dims
// (two blocks) and one of the shared part (one block); a sequence's queries pass through a slot too.
template <int NP>
struct AttSmem {
    static constexpr uint32_t PAGE = (2 * NP + 1) * kBlk;
    static constexpr int NS = NP >= 3 ? 3 : NP == 2 ? 5 : 6;  // slots: what 227 KiB hold
    static constexpr uint32_t OFF_P = NS * PAGE;               // [32 rows][64 keys] bf16
    static constexpr uint32_t OFF_HI = OFF_P + kRows * 128;    // [keys 32-63][32 rows] fp32: high scores
    static constexpr uint32_t OFF_LO = OFF_HI + 32 * kRows * 4;  // [key pairs 0-15][32 rows]: low scores
    static constexpr uint32_t OFF_MISC = OFF_LO + 16 * kRows * 4;
    static constexpr uint32_t BYTES = OFF_MISC + 1024;
    static constexpr uint32_t ALLOC = BYTES > 118784 ? BYTES : 118784;  // one CTA per SM
    // barriers
    static constexpr int B_FULL = 0;                      // [NS][NP + 1] unit landed (TMA)
    static constexpr int B_FREE = B_FULL + NS * (NP + 1);  // [NS][NP + 1] unit's readers done
    static constexpr int B_Q = B_FREE + NS * (NP + 1);     // queries in TMEM (two warps)
    static constexpr int B_S = B_Q + 1;    // scores computed
    static constexpr int B_SR = B_S + 1;   // scores read (two warps)
    static constexpr int B_P = B_SR + 1;   // weights written (four warps)
    static constexpr int B_O = B_P + 1;    // the page's output product done
    static constexpr int B_END = B_O + 1;  // everything issued is done (teardown), one per issuing warp
    static constexpr int N_BARS = B_END + 2;
    static_assert(N_BARS * 8 <= 512, "barriers");
};
static_assert(AttSmem<4>::ALLOC <= 232448, "shared memory per CTA");
// TMEM columns: scores [64 rows, then unused lanes][64 keys], O^T of every unit [128 dims][32 rows],
// the queries as packed bf16 pairs [32 hi, 32 lo rows][(d_c + 64) / 2]
constexpr uint32_t kTmemS = 0, kTmemO = 64, kTmemQ = 192, kTmemCols = 512;

// Barriers of the four softmax warps, of the two that read scores, and an OR over a predicate.
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void bar_scores() { asm volatile("bar.sync 2, 64;" ::: "memory"); }
__device__ __forceinline__ bool bar_softmax_or(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred)
        : "memory");
    return r != 0;
}

// A CTA's walk over its flat pages: the sequence of page `at`, and that sequence's last page in the
// range. The next sequence's length is read when a sequence begins: a load that something waits
// for takes microseconds while pages fill the SM's way to L2.
struct Walk {
    int b, at, page0, seg_begin, seg_end;  // page0: the sequence's first page
    int L, next_L;
    __device__ __forceinline__ void enter(const LatentParams &p, int end, int length) {
        L = length;
        seg_begin = at;
        seg_end = min(end, page0 + pages_of(p, L));
        next_L = b + 1 < p.B ? p.seq_lens[b + 1] : 0;
    }
    __device__ __forceinline__ void seek(const LatentParams &p, int end) {  // at == seg_end < end
        int length = uniform(next_L);
        ++b;
        while (pages_of(p, length) == 0) length = uniform(p.seq_lens[++b]);  // there is one: at < end
        page0 = at;
        enter(p, end, length);
    }
};

template <int NP>
__global__ void __launch_bounds__(kAttThreads, 1)
latent_attend_kernel(const __grid_constant__ CUtensorMap tmc, const __grid_constant__ CUtensorMap tmr,
                     const LatentParams p) {
    using SM = AttSmem<NP>;
    constexpr int NS = SM::NS, NU = NP + 1;
    constexpr uint32_t PAGE = SM::PAGE;
    extern __shared__ __align__(1024) uint8_t sm[];  // no byte is left to align it by hand
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + SM::OFF_MISC;
    auto bar = [&](int i) { return bars + 8 * i; };
    auto full = [&](int st, int u) { return bars + 8 * (SM::B_FULL + st * NU + u); };
    auto free_ = [&](int st, int u) { return bars + 8 * (SM::B_FREE + st * NU + u); };
    uint8_t *misc = sm + SM::OFF_MISC + 512;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 4);
    volatile int *page_ok = reinterpret_cast<volatile int *>(misc + 16);  // [NS]
    float *s_f = reinterpret_cast<float *>(misc + 64);                    // [32] rescaling factors
    float(*s_mx)[kRows] = reinterpret_cast<float(*)[kRows]>(misc + 192);  // [2] maxima, then sums
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int group = blockIdx.x % p.n_groups, range = blockIdx.x / p.n_groups;

    if (tid == 0) {
        for (int i = 0; i < SM::N_BARS; ++i)
            mbar_init(bar(i), i == SM::B_P ? 4 : (i == SM::B_Q || i == SM::B_SR) ? 2 : 1);
        // a test may have the first unit wait for bytes that no copy brings
        if ((int)blockIdx.x == p.skip_cta) mbar_expect_tx(full(0, 0), 16);
        fence_barrier_init();
        *abort_flag = (sb & 1023u) ? 1 : 0;  // (the swizzle needs 1024; else every wait gives up)
        prefetch_tmap(&tmc);
        prefetch_tmap(&tmr);
    }
    if (warp == 5) {
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    griddep_wait();  // the image, the appended rows and the schedule are kernel 1's
    griddep_launch_dependents();  // not before: kernel 3 reads W_uv, which then is complete, without waiting
    const int4 st0 = p.start[range], st1 = p.start[range + 1];
    const int begin = uniform(st0.x), end = uniform(st1.x), n_pages = end - begin;
    Walk w;
    w.b = uniform(st0.y);
    w.at = begin;
    w.page0 = uniform(st0.z);
    w.enter(p, end, uniform(st0.w));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);

    int n_issued = 0;  // of warp 4: units of the ring
    if (warp == 4) {
        // ===== copies into the ring: each sequence's queries, then its pages (the warp converged) ===
        const bool lead = elect_one();
        bool ok = true;
        int k = 0, issued = 0;  // items; units, in order
        // item k; src: the queries' image, or NULL for page pg. The item's units go out in the order in
        // which their slots come free, as many at a time as are free (lane v asks for the v-th)
        auto issue = [&](const uint8_t *src, int pg) {
            const int st = k % NS;
            const bool good = src || (pg >= 0 && pg < p.n_pages);
            int v = 0;
            unsigned long long t0 = 0;
            while (v < NU) {
                uint32_t is_free = ~0u;
                if (k >= NS)
                    is_free = __ballot_sync(0xffffffffu, mbar_test_if(lane < NU, free_(st, (lane + NP) % NU),
                                                                      ((k / NS) - 1) & 1) || lane >= NU);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < NU; ++e) {
                    const int u = e == 0 ? NP : e - 1;  // the shared part's slot is free first
                    if (e != v || !((is_free >> e) & 1u)) continue;
                    const uint32_t dst = sb + st * PAGE + u * 2 * kBlk, bytes = u == NP ? kBlk : 2 * kBlk;
                    if (u == 0) page_ok[st] = good;  // read by whoever waits for unit 0
                    __syncwarp();
                    mbar_expect_if(lead, full(st, u), good ? bytes : 0);
                    if (src) bulk_load_if(lead, dst, src + (size_t)u * 2 * kBlk, bytes, full(st, u));
                    else if (u < NP) tma_load_3d_if(lead && good, dst, &tmc, full(st, u), 0, pg * kPT, u * 2);
                    else tma_load_2d_if(lead && good, dst, &tmr, full(st, u), NP * 128, pg * kPT);
                    ++v;
                    ++issued;
                    t0 = 0;
                }
                if (v < NU) {
                    const unsigned long long now = globaltimer_ns();
                    if (t0 == 0) t0 = now;
                    const bool late = now - t0 > p.wait_ns;
                    if (late) *abort_flag = 1;
                    ok = !__any_sync(0xffffffffu, late || *abort_flag);
                    if (!ok) return;
                }
            }
            if (!good && lead) atomicOr(&g_err, HMD_DEVERR_PAGE);
        };
        while (ok && w.at < end) {
            const uint8_t *q = p.q_img + ((size_t)w.b * p.n_groups + group) * PAGE;
            issue(q, 0);
            ++k;
            const int32_t *table = p.page_table + (size_t)w.b * p.max_pages - w.page0;
            int next = table[w.at];
            for (; w.at < w.seg_end && ok; ++w.at, ++k) {
                const int pg = uniform(next);
                if (w.at + 1 < w.seg_end) next = table[w.at + 1];
                issue(nullptr, pg);
            }
            if (ok && w.at < end) w.seek(p, end);
        }
        if (!ok && lead) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
        n_issued = issued;
        __syncwarp();
    } else if (warp == 5) {
        // ================= scores (the warp converged) =========================================
        const bool lead = elect_one();
        const Desc d_k(smem_desc_sw128(sb, 16, 1024));  // keys x dims
        constexpr uint32_t ID_S = idesc_bf16(128, kPT, 0, 0);
        Walk ws = w;
        int ks = 1, seg = 0;  // items in the ring: the queries come before a sequence's pages
        bool ok = true;
        for (int s = 0; s < n_pages; ++s) {
            // S = [q~hi ; q~lo] C^T once the page has landed (lane u asks for unit u), the scores before
            // have been read and, for a new sequence, its queries are in place
            const int st = ks % NS;
            const bool first = ws.at == ws.seg_begin;
            const bool asks = lane < NU || (lane == NU && s > 0) || (lane == NU + 1 && first);
            const uint32_t b = lane < NU ? full(st, lane) : lane == NU ? bar(SM::B_SR) : bar(SM::B_Q);
            const uint32_t parity = lane < NU ? (ks / NS) & 1 : lane == NU ? (s - 1) & 1 : seg & 1;
            ok = wait_warp(asks, b, parity, abort_flag, p.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const Desc kd = d_k.at(st * PAGE);
#pragma unroll
            for (int v = 0; v < NU; ++v) {
                const int u = v == 0 ? NP : v - 1;  // the shared part's slot is free first
#pragma unroll
                for (int kk = 0; kk < (u == NP ? 4 : 8); ++kk)
                    umma_ts_if(lead, tmem + kTmemS, tmem + kTmemQ + u * 64 + kk * 8,
                               kd.at(u * 2 * kBlk + (kk >> 2) * kBlk + (kk & 3) * 32), ID_S,
                               (v > 0 || kk > 0) ? 1u : 0u);
                if (u == NP) umma_commit_if(lead, free_(st, NP));
            }
            umma_commit_if(lead, bar(SM::B_S));
            ++ks;
            if (__all_sync(0xffffffffu, ++ws.at == ws.seg_end && ws.at < end)) {
                ws.seek(p, end);
                ++ks;
                ++seg;
            }
        }
        if (lead) {
            if (!ok) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
            // every product is done before TMEM and shared memory go (bounded)
            umma_commit(bar(SM::B_END));
            (void)mbar_wait_bounded(bar(SM::B_END), 0);
        }
        __syncwarp();
    } else if (warp == 6) {
        // ===== outputs (the warp converged), issued beside the scores: 52 products and 7 commits a page
        // are more than one warp issues in the tensor core's time =================================
        const bool lead = elect_one();
        const Desc d_v(smem_desc_sw128(sb, kBlk, 1024));  // dims x keys
        const Desc d_p(smem_desc_sw128(sb + SM::OFF_P, 16, 1024));
        constexpr uint32_t ID_O = idesc_bf16(128, kRows, 1, 0);
        Walk wp = w;
        int kp = 1;
        bool ok = true;
        for (int pv = 0; pv < n_pages; ++pv) {
            ok = wait_warp(lead, bar(SM::B_P), pv & 1, abort_flag, p.wait_ns);
            if (!ok) break;
            // O^T += C^T P^T, unit by unit; each unit's slot is free after it
            tc_fence_after();
            const int st = kp % NS;
            const bool fresh = __all_sync(0xffffffffu, wp.at == wp.seg_begin);
            const Desc v = d_v.at(st * PAGE);
#pragma unroll
            for (int u = 0; u < NP; ++u) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_if(lead, tmem + kTmemO + u * kRows, v.at(u * 2 * kBlk + kk * 2048),
                            d_p.at(kk * 32), ID_O, (fresh && kk == 0) ? 0u : 1u);
                umma_commit_if(lead, free_(st, u));
            }
            umma_commit_if(lead, bar(SM::B_O));
            ++kp;
            if (__all_sync(0xffffffffu, ++wp.at == wp.seg_end && wp.at < end)) {
                wp.seek(p, end);
                ++kp;
            }
        }
        if (lead) {
            if (!ok) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
            umma_commit(bar(SM::B_END + 1));
            (void)mbar_wait_bounded(bar(SM::B_END + 1), 0);
        }
        __syncwarp();
    } else {
        // ================= softmax and the partial results =====================================
        // Warp 0 receives the rows' scores of q~hi (lane = row), warp 1 those of q~lo. They swap halves
        // and each does the softmax of 32 of the page's keys; all four warps hold O^T (lane = latent
        // dim of a unit).
        const bool lead = elect_one();
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        float *hi_x = reinterpret_cast<float *>(sm + SM::OFF_HI) + lane;        // [key - 32][row]
        uint32_t *lo_x = reinterpret_cast<uint32_t *>(sm + SM::OFF_LO) + lane;  // [key pair][row]
        bool ok = true;
        int item = 0, k = 0;  // ring items, pages
        while (ok && w.at < end) {
            const int b = w.b, L = w.L, page0 = w.page0;
            if (warp < 2) {
                // this sequence's queries to TMEM: lane = row of the image (32 hi, then 32 lo). The
                // scores of the sequence before are complete, so its queries are not read any more
                const int st = item % NS;
                ok &= wait_warp(lane < NU, full(st, min(lane, NP)), (item / NS) & 1, abort_flag, p.wait_ns);
                const uint8_t *row = sm + st * PAGE + (warp * 32 + lane) * 128;
                const bool none = group * kRows + lane >= p.nq * p.H;  // no such query: its row is not written
#pragma unroll 1
                for (int c = 0; c < 2 * NP + 1; ++c) {
                    uint32_t r[32];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(row + c * kBlk + ((e ^ (lane & 7)) << 4));
                        r[4 * e] = none ? 0u : x.x;
                        r[4 * e + 1] = none ? 0u : x.y;
                        r[4 * e + 2] = none ? 0u : x.z;
                        r[4 * e + 3] = none ? 0u : x.w;
                    }
                    tmem_st32(tmem + kTmemQ + c * 32 + lanes, r);
                }
                tmem_wait_st();
                tc_fence_before();
                fence_proxy_async_smem();  // the slot's next filling comes after these reads
                bar_scores();
                // (not after a wait that gave up: the slot's copy may not have landed)
                if (ok && warp == 0 && lane < NU) mbar_arrive(free_(st, lane));
                if (ok && lane == 0) mbar_arrive(bar(SM::B_Q));
            }
            ++item;
            // the last position this row sees (-1: no such row)
            const int r_row = group * kRows + lane;
            const int last = r_row < p.nq * p.H ? L - p.nq + r_row / p.H : -1;
            float base = -INFINITY, l = 0.f;
            for (; w.at < w.seg_end; ++w.at, ++k, ++item) {
                const int st = item % NS, pos0 = (w.at - page0) * kPT;
                float x[32], mx = -INFINITY;
                bool grew = false;
                if (warp < 2) {
                    // the scores and, for page_ok, the page
                    ok &= wait_warp(lane < 2, lane ? full(st, 0) : bar(SM::B_S),
                                    (lane ? item / NS : k) & 1, abort_flag, p.wait_ns);
                    tc_fence_after();
                    {
                        uint32_t r[64];
                        tmem_ld64(tmem + kTmemS + lanes, r);
                        tmem_wait_ld();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(SM::B_SR));
                        if (warp == 0) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                hi_x[j * kRows] = __uint_as_float(r[32 + j]);
                                x[j] = __uint_as_float(r[j]);
                            }
                        } else {
                            // a low score is below 2^-8 of its row's: bf16 keeps it to 2^-17 of that
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                lo_x[j * kRows] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(r[32 + j]);
                        }
                    }
                    bar_scores();
                    if (warp == 0) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint32_t v = lo_x[j * kRows];
                            x[2 * j] += bf16_lo(v);
                            x[2 * j + 1] += bf16_hi(v);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] += hi_x[j * kRows];
                    }
                    const bool good = page_ok[st] != 0;
                    if (!good || pos0 + kPT > L - p.nq + 1 || (group + 1) * kRows > p.nq * p.H) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!good || pos0 + 32 * warp + j > last) x[j] = -INFINITY;
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        m4[0] = max3(m4[0], x[j], x[j + 1]);
                        m4[1] = max3(m4[1], x[j + 2], x[j + 3]);
                        m4[2] = max3(m4[2], x[j + 4], x[j + 5]);
                        m4[3] = max3(m4[3], x[j + 6], x[j + 7]);
                    }
                    mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    grew = mx > base + kLazy;
                    s_mx[warp][lane] = mx;
                }
                if (bar_softmax_or(grew || !ok)) {
                    ok = !bar_softmax_or(!ok);
                    if (!ok) break;
                    if (warp < 2) {
                        // a row that outgrew its base moves it to the maximum of both halves
                        mx = fmaxf(mx, s_mx[warp ^ 1][lane]);
                        float f = 1.f;
                        if (mx > base + kLazy) {
                            f = exp2f(base - mx);
                            base = mx;
                            l *= f;
                        }
                        if (warp == 0) s_f[lane] = f;
                    }
                    bar_softmax();
                    if (w.at > w.seg_begin) {
                        // the earlier output to the new bases, once the product into it is done
                        ok = wait_warp(lead, bar(SM::B_O), (k - 1) & 1, abort_flag, p.wait_ns);
                        tc_fence_after();
#pragma unroll 1
                        for (int u = 0; u < NP; ++u) {
                            uint32_t r[32];
                            tmem_ld32(tmem + kTmemO + u * kRows + lanes, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                r[c] = __float_as_uint(__uint_as_float(r[c]) * s_f[c]);
                            tmem_st32(tmem + kTmemO + u * kRows + lanes, r);
                        }
                        tmem_wait_st();
                    }
                    bar_softmax();  // s_f and s_mx are free again
                }
                if (warp < 2) {
                    const float m = base == -INFINITY ? 0.f : base;
                    uint32_t pk[16];
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float p0 = ex2_approx(x[2 * j] - m), p1 = ex2_approx(x[2 * j + 1] - m);
                        sum[(2 * j) & 3] += p0;
                        sum[(2 * j + 1) & 3] += p1;
                        pk[j] = pack_bf16x2(p0, p1);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    // P [32 rows][64 keys], rows of 128 bytes, 128-byte swizzle, once the product
                    // before has read it. bf16 as the latent rows, the one type a product can have beside them:
                    // 2^-8 of a weight at random signs, as in the FA decode; the sum has them in full
                    if (k > 0) ok &= wait_warp(lead, bar(SM::B_O), (k - 1) & 1, abort_flag, p.wait_ns);
                    uint8_t *row = sm + SM::OFF_P + lane * 128;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4 *>(row + (((4 * warp + e) ^ (lane & 7)) << 4)) =
                            make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                }
                if (!page_ok[st] || pos0 + kPT > L) {
                    // rows behind the sequence (or of a page that was not copied) hold anything: as
                    // values they are zeroed before the output product reads them
                    const int n_ok = page_ok[st] ? L - pos0 : 0;
                    for (int idx = tid; idx < (kPT - n_ok) * NP * 16; idx += 128) {
                        const int row = n_ok + idx / (NP * 16), ch = idx % (NP * 16);
                        *reinterpret_cast<uint4 *>(sm + st * PAGE + (ch >> 3) * kBlk +
                                                   blk_off(row, (ch & 7) * 8)) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(SM::B_P));
            }
            const size_t piece = part_index(p, range, b, group);
            if (ok) ok = wait_warp(lead, bar(SM::B_O), (k - 1) & 1, abort_flag, p.wait_ns);
            ok = !bar_softmax_or(!ok);
            if (!ok) {
                // this piece and the range's later ones are marked as missing
                while (true) {
                    if (tid < kRows) p.part_ml[(part_index(p, range, w.b, group) * kRows + tid) * 2 + 1] = -1.f;
                    w.at = w.seg_end;
                    if (w.at >= end) break;
                    w.seek(p, end);
                }
                break;
            }
            tc_fence_after();
            float *dst = p.part_o + piece * kRows * p.dc + tid;  // lane = latent dim of the unit
#pragma unroll 1
            for (int u = 0; u < NP; ++u) {
                uint32_t r[32];
                tmem_ld32(tmem + kTmemO + u * kRows + lanes, r);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) dst[(size_t)c * p.dc + u * 128] = __uint_as_float(r[c]);
            }
            tc_fence_before();
            if (warp == 1) s_mx[1][lane] = l;
            bar_softmax();
            if (warp == 0)
                *reinterpret_cast<float2 *>(p.part_ml + (piece * kRows + lane) * 2) =
                    make_float2(base, l + s_mx[1][lane]);
            bar_softmax();
            if (w.at < end) w.seek(p, end);
        }
        if (!ok && tid == 0) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 4 && lane == 0) {
        // the copies in flight land (bounded) before shared memory is released
        for (int i = max(0, n_issued - NS * NU); i < n_issued; ++i) {
            const int ki = i / NU, v = i % NU;
            (void)mbar_wait_bounded(full(ki % NS, v == 0 ? NP : v - 1), (ki / NS) & 1, p.wait_ns);
        }
    }
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- kernel 3 ----------------------------------------------------------------------------------
constexpr int kExpThreads = 512;
constexpr int kExpWarps = kExpThreads / 32;
// Up to TOK tokens (b, i) of one head per CTA, d_c = 128 * NP latent dims.
template <int D, int NP, int TOK>
struct ExpSmem {
    static constexpr int WP = NP * 128 + 8;  // pitch (elements) without bank conflicts
    __nv_bfloat16 w[D][WP];                  // W_uv[h]
    __nv_bfloat16 hi[TOK][WP], lo[TOK][WP];  // the merged latent output as a bf16 pair
    float den[kExpWarps];
    uint64_t bar;
    uint32_t missing;                        // tokens of which a range gave up
    // A token's sums, per warp that shares it: over hi and lo, which are written after them (warps
    // share a token only where all tokens are merged at once).
    static_assert(2 * TOK * WP * 2 >= kExpWarps * NP * 128 * 4, "the sums fit");
    __device__ float (*red())[NP * 128] { return reinterpret_cast<float(*)[NP * 128]>(&hi[0][0]); }
};
static_assert(sizeof(ExpSmem<128, 4, 32>) <= 232448, "shared memory per CTA");

template <int D, int NP, int TOK>
__global__ void __launch_bounds__(kExpThreads, 1) latent_expand_kernel(const LatentParams p, int tokens) {
    using SM = ExpSmem<D, NP, TOK>;
    constexpr int DC = NP * 128, kFlight = NP > 2 ? 3 : 4;
    extern __shared__ __align__(16) uint8_t exp_smem[];
    SM &sm = *reinterpret_cast<SM *>(exp_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x, tok0 = blockIdx.y * tokens, rows = min(tokens, p.B * p.nq - tok0);
    const uint32_t bar = smem_u32(&sm.bar);
    if (warp == kExpWarps - 1) {
        // W_uv[h] lands during kernel 2's end and the merge, a bulk copy per row
        if (lane == 0) {
            mbar_init(bar, 1);
            fence_barrier_init();
            mbar_arrive_expect_tx(bar, D * DC * 2);
            sm.missing = 0;
        }
        __syncwarp();
        const __nv_bfloat16 *w = p.w_uv + h * p.w_uv_head;
        for (int v = lane; v < D; v += 32) bulk_load(smem_u32(&sm.w[v][0]), w + (size_t)v * DC, DC * 2, bar);
    }
    griddep_launch_dependents();
    griddep_wait();
    __syncthreads();
    // merge the ranges: `wpr` warps share a token's ranges, a lane has 4 dims of every 128
    const int wpr = rows > 8 ? 1 : rows > 4 ? 2 : rows > 2 ? 4 : rows > 1 ? 8 : 16;
    for (int r0 = 0; r0 < rows; r0 += kExpWarps / wpr) {
        const int r = r0 + warp / wpr, part = warp % wpr;
        float4 acc[NP];
#pragma unroll
        for (int u = 0; u < NP; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
        if (r < rows) {
            const int tok = tok0 + r, b = tok / p.nq, row = (tok - b * p.nq) * p.H + h;
            const int2 range = p.ranges[b];
            const int i0 = range.x, i1 = range.y, g = row / kRows, c = row % kRows;
            float M = -INFINITY;
            bool lost = false;
            for (int i = i0 + lane; i < i1; i += 32) {
                const float2 v = *reinterpret_cast<const float2 *>(
                    p.part_ml + (part_index(p, i, b, g) * kRows + c) * 2);
                M = fmaxf(M, v.x);
                lost |= v.y < 0.f;
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            lost = __any_sync(0xffffffffu, lost);
            if (lost && lane == 0) atomicOr(&sm.missing, 1u << r);
            if (M != -INFINITY) {
                for (int i = i0 + part; i < i1; i += kFlight * wpr) {  // kFlight ranges' loads in flight
                    float2 v[kFlight];
                    float4 x[kFlight][NP];
#pragma unroll
                    for (int e = 0; e < kFlight; ++e) {
                        const int ie = i + e * wpr;
                        if (ie < i1) {
                            const size_t at = part_index(p, ie, b, g) * kRows + c;
                            v[e] = *reinterpret_cast<const float2 *>(p.part_ml + at * 2);
#pragma unroll
                            for (int u = 0; u < NP; ++u)
                                x[e][u] = *reinterpret_cast<const float4 *>(p.part_o + at * DC + u * 128 + lane * 4);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < kFlight; ++e) {
                        if (i + e * wpr < i1) {
                            const float f = exp2f(v[e].x - M);
                            den += f * v[e].y;
#pragma unroll
                            for (int u = 0; u < NP; ++u) {
                                acc[u].x += f * x[e][u].x; acc[u].y += f * x[e][u].y;
                                acc[u].z += f * x[e][u].z; acc[u].w += f * x[e][u].w;
                            }
                        }
                    }
                }
            }
        }
        if (wpr > 1) {
#pragma unroll
            for (int u = 0; u < NP; ++u) *reinterpret_cast<float4 *>(&sm.red()[warp][u * 128 + lane * 4]) = acc[u];
            if (lane == 0) sm.den[warp] = den;
            __syncthreads();
            if (part == 0)
                for (int v = 1; v < wpr; ++v) {
#pragma unroll
                    for (int u = 0; u < NP; ++u) {
                        const float4 x = *reinterpret_cast<const float4 *>(&sm.red()[warp + v][u * 128 + lane * 4]);
                        acc[u].x += x.x; acc[u].y += x.y; acc[u].z += x.z; acc[u].w += x.w;
                    }
                    den += sm.den[warp + v];
                }
            __syncthreads();
        }
        if (part == 0 && r < rows) {
            const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
            for (int u = 0; u < NP; ++u) {
                const float x[4] = {acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv};
                const uint32_t h0 = pack_bf16x2(x[0], x[1]), h1 = pack_bf16x2(x[2], x[3]);
                *reinterpret_cast<uint2 *>(&sm.hi[r][u * 128 + lane * 4]) = make_uint2(h0, h1);
                *reinterpret_cast<uint2 *>(&sm.lo[r][u * 128 + lane * 4]) =
                    make_uint2(pack_bf16x2(x[0] - bf16_lo(h0), x[1] - bf16_hi(h0)),
                               pack_bf16x2(x[2] - bf16_lo(h1), x[3] - bf16_hi(h1)));
            }
        }
    }
    for (int r = rows + warp; r < TOK; r += kExpWarps) {  // rows without a token
#pragma unroll
        for (int u = 0; u < NP; ++u) {
            *reinterpret_cast<uint2 *>(&sm.hi[r][u * 128 + lane * 4]) = make_uint2(0u, 0u);
            *reinterpret_cast<uint2 *>(&sm.lo[r][u * 128 + lane * 4]) = make_uint2(0u, 0u);
        }
    }
    const bool ok = mbar_wait_bounded(bar, 0);
    if (__syncthreads_or(!ok)) {
        if (tid == 0) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
        return;
    }
    // out[TOK][D] = latent output x W_uv^T: a warp has 8 columns and 16 tokens, or (D = 64, 16 tokens)
    // half of the warps do
    constexpr int CT = D / 8, RT = TOK / 16;  // column and row tiles
    for (int t = warp; t < CT * RT; t += kExpWarps) {
        const int ct = t % CT, rt = t / CT;
        float a0[4] = {}, a1[4] = {};
#pragma unroll 8
        for (int kk = 0; kk < DC / 16; ++kk) {
            uint32_t ah[4], al[4];
            ldmatrix_x4(smem_u32(&sm.hi[rt * 16 + (lane & 15)][kk * 16 + (lane >> 4) * 8]), ah[0], ah[1], ah[2], ah[3]);
            ldmatrix_x4(smem_u32(&sm.lo[rt * 16 + (lane & 15)][kk * 16 + (lane >> 4) * 8]), al[0], al[1], al[2], al[3]);
            const __nv_bfloat16 *wr = &sm.w[ct * 8 + (lane >> 2)][kk * 16 + (lane & 3) * 2];
            const uint32_t b0 = *reinterpret_cast<const uint32_t *>(wr);
            const uint32_t b1 = *reinterpret_cast<const uint32_t *>(wr + 8);
            mma_bf16_16816(a0, ah, b0, b1);
            mma_bf16_16816(a1, al, b0, b1);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = rt * 16 + (lane >> 2) + 8 * e;
            if (r < rows && !((sm.missing >> r) & 1u))  // else o stays as it was
                *reinterpret_cast<uint32_t *>(p.o + ((size_t)(tok0 + r) * p.H + h) * D + ct * 8 + (lane & 3) * 2) =
                    pack_bf16x2(a0[2 * e] + a1[2 * e], a0[2 * e + 1] + a1[2 * e + 1]);
        }
    }
}

// ---- host side ---------------------------------------------------------------------------------
struct Plan {
    int n_groups, n_ranges;
    size_t off_o, off_ml, off_start, off_ranges, off_cum, bytes;
};
Plan make_plan(int nq, int B, int H, int dc, int max_seq_len) {
    Plan pl;
    pl.n_groups = (int)(((long long)nq * H + kRows - 1) / kRows);
    const long long pages = (long long)B * (((long long)max_seq_len + kPT - 1) / kPT);
    // one CTA per SM: the groups of one range run side by side and share its pages through L2
    pl.n_ranges = (int)std::min<long long>(std::max(1, sm_count() / pl.n_groups), pages);
    const size_t pieces = (size_t)(pl.n_ranges + B) * pl.n_groups;
    pl.off_o = (size_t)B * pl.n_groups * (dc / 64 + 1) * kBlk;
    pl.off_ml = pl.off_o + pieces * kRows * dc * sizeof(float);
    pl.off_start = pl.off_ml + pieces * kRows * 2 * sizeof(float);
    pl.off_ranges = pl.off_start + ((size_t)pl.n_ranges + 1) * sizeof(int4);
    pl.off_cum = pl.off_ranges + (size_t)B * sizeof(int2);
    pl.bytes = pl.off_cum + (((size_t)B + 1) * sizeof(int32_t) + 15) / 16 * 16;
    return pl;
}

template <int NP>
cudaError_t launch_attend(const CUtensorMap &tmc, const CUtensorMap &tmr, const LatentParams &p,
                          cudaStream_t s) {
    constexpr int smem = (int)AttSmem<NP>::ALLOC;
    const cudaError_t e = once_per_device([] {
        return cudaFuncSetAttribute(latent_attend_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)AttSmem<NP>::ALLOC);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_attend_kernel<NP>, dim3((unsigned)(p.n_ranges * p.n_groups)),
                      dim3(kAttThreads), smem, s, tmc, tmr, p);
}

template <int D>
cudaError_t launch_absorb(const LatentParams &p, cudaStream_t s) {
    const cudaError_t e = once_per_device([] {
        return cudaFuncSetAttribute(latent_absorb_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(AbsSmem<D>));
    });
    if (e != cudaSuccess) return e;
    const int blocks = (p.B * p.nq + kAbsTok - 1) / kAbsTok;
    const int n_app = (p.B * p.nq + kAbsThreads / 32 - 1) / (kAbsThreads / 32);
    return launch_pdl(latent_absorb_kernel<D>, dim3((unsigned)(p.dc / 128 * p.H * blocks + n_app + 1)),
                      dim3(kAbsThreads), sizeof(AbsSmem<D>), s, p);
}

template <int D, int NP, int TOK>
cudaError_t launch_expand_t(const LatentParams &p, int tokens, cudaStream_t s) {
    const cudaError_t e = once_per_device([] {
        return cudaFuncSetAttribute(latent_expand_kernel<D, NP, TOK>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(ExpSmem<D, NP, TOK>));
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_expand_kernel<D, NP, TOK>,
                      dim3((unsigned)p.H, (unsigned)((p.B * p.nq + tokens - 1) / tokens)),
                      dim3(kExpThreads), sizeof(ExpSmem<D, NP, TOK>), s, p, tokens);
}
// The fewest tokens a CTA (each reads all of W_uv[h]) with which the grid has at most one CTA per SM.
template <int D, int NP>
cudaError_t launch_expand_np(const LatentParams &p, cudaStream_t s) {
    int tokens = 4;
    while (tokens < 32 && (long long)p.H * ((p.B * p.nq + tokens - 1) / tokens) > sm_count()) tokens *= 2;
    return tokens > 16 ? launch_expand_t<D, NP, 32>(p, tokens, s) : launch_expand_t<D, NP, 16>(p, tokens, s);
}
template <int D>
cudaError_t launch_expand(const LatentParams &p, cudaStream_t s) {
    switch (p.dc / 128) {
        case 1: return launch_expand_np<D, 1>(p, s);
        case 2: return launch_expand_np<D, 2>(p, s);
        case 3: return launch_expand_np<D, 3>(p, s);
        default: return launch_expand_np<D, 4>(p, s);
    }
}

}  // namespace

bool latent_supported(int d, int d_c, int d_r, int page_tokens) {
    return (d == 64 || d == 128) && d_c >= 128 && d_c <= 512 && d_c % 128 == 0 && d_r == kDR &&
           page_tokens == kPT;
}

size_t latent_decode_ws_bytes(int nq, int B, int H, int d_c, int max_seq_len) {
    return make_plan(nq, B, H, d_c, max_seq_len).bytes;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t s) {
    const Plan pl = make_plan(a.nq, a.B, a.H, a.d_c, a.max_seq_len);
    // c in units of 128 dims, two column blocks a box, and the shared part
    CUtensorMap tmc, tmr;
    if (!make_tmap_colblocks_sw128(&tmc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.pool, (long long)a.n_pages * kPT,
                                   a.d_c + kDR, a.d_c / 64, kPT, 2) ||
        !make_tmap_pool_sw128(&tmr, a.pool, a.n_pages, 1, a.d_c + kDR))
        return cudaErrorInvalidValue;
    LatentParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.new_c = static_cast<const __nv_bfloat16 *>(a.new_c);
    p.w_uk = static_cast<const __nv_bfloat16 *>(a.w_uk);
    p.w_uv = static_cast<const __nv_bfloat16 *>(a.w_uv);
    p.w_uk_head = a.w_uk_head; p.w_uv_head = a.w_uv_head;
    p.pool = static_cast<__nv_bfloat16 *>(a.pool);
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.page_table = a.page_table; p.seq_lens = a.seq_lens;
    p.B = a.B; p.nq = a.nq; p.H = a.H; p.d = a.d; p.dc = a.d_c; p.n_pages = a.n_pages;
    p.max_pages = a.max_pages; p.max_seq_len = a.max_seq_len;
    p.n_groups = pl.n_groups; p.n_ranges = pl.n_ranges;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.q_img = ws;
    p.part_o = reinterpret_cast<float *>(ws + pl.off_o);
    p.part_ml = reinterpret_cast<float *>(ws + pl.off_ml);
    p.start = reinterpret_cast<int4 *>(ws + pl.off_start);
    p.ranges = reinterpret_cast<int2 *>(ws + pl.off_ranges);
    p.cum = reinterpret_cast<int32_t *>(ws + pl.off_cum);
    p.skip_cta = a.skip.cta; p.wait_ns = a.skip.wait_ns;
    cudaError_t e = a.d == 128 ? launch_absorb<128>(p, s) : launch_absorb<64>(p, s);
    if (e != cudaSuccess) return e;
    switch (a.d_c / 128) {
        case 1: e = launch_attend<1>(tmc, tmr, p, s); break;
        case 2: e = launch_attend<2>(tmc, tmr, p, s); break;
        case 3: e = launch_attend<3>(tmc, tmr, p, s); break;
        default: e = launch_attend<4>(tmc, tmr, p, s); break;
    }
    if (e != cudaSuccess) return e;
    return a.d == 128 ? launch_expand<128>(p, s) : launch_expand<64>(p, s);
}

uint32_t latent_decode_read_errors(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_err, sizeof v) != cudaSuccess) return 0;
    if (clear && v) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_err, &z, sizeof z);
    }
    return v;
}

}  // namespace hmd
