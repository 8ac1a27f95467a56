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
// q~ = hi + lo and stored as the shared-memory image kernel 2 wants. Rounding q~ to one bf16 would
// put an error of 2^-9 |s| on every score; the pair leaves 2^-17, and its second half rides
// along in the tensor core's N dimension. It also appends the new latent rows to the cache and
// lays out the schedule (running page counts of the batch).
// Kernel 2 (attention): the batch's pages, laid end to end, are cut into equal ranges, one per
// SM (times the row groups of 32 rows), whatever the lengths are; a CTA's range may end one
// sequence and begin another. Per page of 64 keys, with keys and latent dims as the M of the
// products (the few query rows as N, so nothing is padded to 128 rows):
//     S^T [64 keys x 64] = C [64 x (d_c + 64)] [q~hi ; q~lo]^T     tcgen05, M = 64, N = 64
//     O^T [d_c x 32]    += C^T [d_c x 64 keys] P^T                 tcgen05, M = 128, N = 32
// both from the same shared-memory tile of C (K-major, then MN-major). Warp-specialised: warp 4
// streams pages by TMA (units of 128 dims, each freed as soon as its product is done), warp 5
// issues the products, warps 0-3 are the softmax. O^T accumulates at an exponent base per row
// that moves only when the row's scores exceed it by more than 2^8 (then O^T is rescaled in
// TMEM), so the common page needs one vote and no exchange of maxima.
// Kernel 3 (merge and expand), one cluster per (head, 16 tokens) with a CTA per 128 latent dims:
// joins the ranges' partial sums, multiplies by its dims' part of W_uv[h] (mma.sync, the latent
// output as a bf16 pair) and adds up over the cluster in rank order.
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
    int32_t *cum;    // [B + 1] pages before each sequence
    int4 *start;     // [n_ranges + 1]: a range's first page, its sequence, that sequence's first page
                     // and the page after its last
    int2 *ranges;    // [B]: a sequence's ranges [x, y)
};

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
__device__ void schedule_block(const LatentParams &p) {
    __shared__ int warp_sum[kAbsThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int base = 0;
    if (tid == 0) p.cum[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAbsThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < p.B) {
            const int L = p.seq_lens[b];
            if (L >= p.nq && L <= p.max_seq_len) n = (L + kPT - 1) / kPT;
            else if (L != 0) atomicOr(&g_err, HMD_DEVERR_SEQLEN);
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
        if (b < p.B) p.cum[b + 1] = base + sum;
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
                if (p.cum[mid] <= st.x) lo = mid;
                else hi = mid;
            }
            st = make_int4(st.x, lo, p.cum[lo], p.cum[lo + 1]);
        }
        p.start[i] = st;
    }
    for (int b = tid; b < p.B; b += kAbsThreads) {
        const int c0 = p.cum[b], c1 = p.cum[b + 1];
        p.ranges[b] = c1 > c0 ? make_int2(range_of(c0, P, n_live), range_of(c1 - 1, P, n_live) + 1)
                              : make_int2(0, 0);
    }
}

template <int D>
__global__ void __launch_bounds__(kAbsThreads) latent_absorb_kernel(const LatentParams p) {
    extern __shared__ __align__(16) uint8_t abs_smem[];
    AbsSmem<D> &sm = *reinterpret_cast<AbsSmem<D> *>(abs_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int n_tok = p.B * p.nq, dq = D + kDR, row_w = p.dc + kDR;
    if (blockIdx.x == gridDim.x - 1) {
        schedule_block(p);
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
    if (h == 0 && cc == n_cols - 1) {
        // rows of the last group that belong to no query: zero (16-byte chunks of every block)
        const int pad0 = p.nq * p.H, n_pad = p.n_groups * kRows - pad0, chunks = (p.dc / 64 + 1) * 8;
        for (int r = 0; r < rows && n_pad; ++r) {
            const int tok = tok0 + r, b = tok / p.nq;
            if (tok != b * p.nq) continue;
            uint8_t *base = p.q_img + ((size_t)b * p.n_groups + p.n_groups - 1) * img_bytes;
            for (int idx = tid; idx < n_pad * 2 * chunks; idx += kAbsThreads) {
                const int ch = idx % chunks, rr = idx / chunks;
                const int row = kRows - n_pad + rr % n_pad + (rr >= n_pad ? kRows : 0);
                *reinterpret_cast<uint4 *>(base + (size_t)(ch >> 3) * kBlk + blk_off(row, (ch & 7) * 8)) =
                    make_uint4(0, 0, 0, 0);
            }
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
constexpr int kAttThreads = 192;
// Shared memory for d_c = 128 * NP: the queries' image, page stages, P, barriers. A page is NP
// units of 128 dims (two blocks) and one of the shared part (one block).
template <int NP>
struct AttSmem {
    static constexpr uint32_t PAGE = (2 * NP + 1) * kBlk;
    static constexpr int NS = NP >= 3 ? 2 : 4;  // page stages: what 227 KiB hold
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_C = PAGE;
    static constexpr uint32_t OFF_P = OFF_C + NS * PAGE;       // two tiles [32 rows][64 keys]
    static constexpr uint32_t OFF_MISC = OFF_P + 2 * kRows * 128;
    static constexpr uint32_t BYTES = OFF_MISC + 2048;
    static constexpr uint32_t ALLOC = BYTES > 118784 ? BYTES : 118784;  // one CTA per SM
    // barriers
    static constexpr int B_FULL = 0;                      // [NS][NP + 1] unit landed (TMA)
    static constexpr int B_FREE = B_FULL + NS * (NP + 1);  // [NS][NP + 1] unit's products done
    static constexpr int B_QFULL = B_FREE + NS * (NP + 1);
    static constexpr int B_QFREE = B_QFULL + 1;
    static constexpr int B_S = B_QFREE + 1;  // [2] scores computed
    static constexpr int B_P = B_S + 2;      // [2] weights written (four warps)
    static constexpr int B_O = B_P + 2;      // [2] the page's output product done
    static constexpr int B_END = B_O + 2;    // everything issued is done (teardown)
    static constexpr int N_BARS = B_END + 1;
    static_assert(N_BARS * 8 <= 512, "barriers");
};
static_assert(AttSmem<4>::ALLOC + 1024 <= 232448, "shared memory per CTA");
// TMEM: scores of even and odd pages, then O^T of every unit
constexpr uint32_t kTmemS = 0, kTmemO = 128, kTmemCols = 256;

// 16 lanes x 64 columns of TMEM words: register 4j + e of thread t holds lane (base + t / 4 +
// 8 (e / 2)), column 8j + 2 (t % 4) + e % 2.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// Four 8x8 b16 matrices to shared memory, transposed: lane l gives the address of row l % 8 of
// matrix l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1,
                                                  uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
                 "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}
// The softmax warps' own barrier, and the same with an OR over a predicate.
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
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

// A CTA's walk over its flat pages: the sequence of page `at`, and that sequence's last page in
// the range.
struct Walk {
    int b, at, page0, seg_begin, seg_end;  // page0: the sequence's first page
    __device__ __forceinline__ void seek(const LatentParams &p, int end) {  // at == seg_end < end
        do {
            ++b;
            seg_end = uniform(p.cum[b + 1]);
        } while (seg_end <= at);  // skips sequences without pages; ends: cum[B] >= end > at
        page0 = seg_begin = at;
        seg_end = min(end, seg_end);
    }
};

template <int NP>
__global__ void __launch_bounds__(kAttThreads, 1)
latent_attend_kernel(const __grid_constant__ CUtensorMap tmc, const LatentParams p) {
    using SM = AttSmem<NP>;
    constexpr int NS = SM::NS, NU = NP + 1;
    constexpr uint32_t PAGE = SM::PAGE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(sm);
    const uint32_t bars = sb + SM::OFF_MISC;
    auto bar = [&](int i) { return bars + 8 * i; };
    auto full = [&](int st, int u) { return bars + 8 * (SM::B_FULL + st * NU + u); };
    auto free_ = [&](int st, int u) { return bars + 8 * (SM::B_FREE + st * NU + u); };
    uint8_t *misc = sm + SM::OFF_MISC + 512;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 4);
    volatile int *page_ok = reinterpret_cast<volatile int *>(misc + 16);  // [NS]
    float(*s_red)[kRows] = reinterpret_cast<float(*)[kRows]>(misc + 64);  // [4][32]
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int group = blockIdx.x % p.n_groups, range = blockIdx.x / p.n_groups;

    if (tid == 0) {
        for (int i = 0; i < SM::N_BARS; ++i)
            mbar_init(bar(i), (i == SM::B_P || i == SM::B_P + 1) ? 4 : 1);
        fence_barrier_init();
        *abort_flag = 0;
        prefetch_tmap(&tmc);
    }
    if (warp == 5) {
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    griddep_launch_dependents();
    griddep_wait();  // the image, the appended rows and the schedule are kernel 1's
    const int4 st0 = p.start[range], st1 = p.start[range + 1];
    const int begin = uniform(st0.x), end = uniform(st1.x), n_pages = end - begin;
    Walk w;
    w.b = uniform(st0.y);
    w.at = w.seg_begin = begin;
    w.page0 = uniform(st0.z);
    w.seg_end = min(end, uniform(st0.w));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);

    if (warp == 4) {
        // ================= copies: the queries of each sequence, and its pages ==============
        bool ok = true;
        int k = 0, seg = 0, issued = 0, q_issued = 0;  // issued: units, in order (lane 0)
        while (ok && w.at < end) {
            const int b = w.b, first = w.at - w.page0, n = w.seg_end - w.at;
            if (seg > 0) ok = wait_or_abort(bar(SM::B_QFREE), (seg - 1) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(SM::B_QFULL), PAGE);
                ++q_issued;
                const uint8_t *src = p.q_img + ((size_t)b * p.n_groups + group) * PAGE;
#pragma unroll
                for (int i = 0; i < 2 * NP + 1; ++i)
                    bulk_load(sb + SM::OFF_Q + i * kBlk, src + (size_t)i * kBlk, kBlk, bar(SM::B_QFULL));
            }
            int entry = -1;
            for (int t = 0; t < n && ok; ++t, ++k) {
                if ((t & 31) == 0)
                    entry = t + lane < n ? p.page_table[(size_t)b * p.max_pages + first + t + lane] : -1;
                const int pg = __shfl_sync(0xffffffffu, entry, t & 31);
                const int st = k % NS;
                const bool good = pg >= 0 && pg < p.n_pages;
                if (lane == 0) {
                    if (!good) atomicOr(&g_err, HMD_DEVERR_PAGE);
#pragma unroll
                    for (int v = 0; v < NU; ++v) {
                        const int u = v == 0 ? NP : v - 1;  // the shared part is free first
                        if (k >= NS) ok = wait_or_abort(free_(st, u), ((k / NS) - 1) & 1, abort_flag);
                        if (!ok) break;
                        if (u == 0) page_ok[st] = good;  // read by whoever waits for unit 0
                        const uint32_t bytes = u == NP ? kBlk : 2 * kBlk;
                        mbar_arrive_expect_tx(full(st, u), good ? bytes : 0);
                        ++issued;
                        if (!good) continue;
                        const uint32_t dst = sb + SM::OFF_C + st * PAGE + u * 2 * kBlk;
                        tma_load_2d(dst, &tmc, full(st, u), u * 128, pg * kPT);
                        if (u < NP) tma_load_2d(dst + kBlk, &tmc, full(st, u), u * 128 + 64, pg * kPT);
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
            }
            w.at = w.seg_end;
            ++seg;
            if (w.at < end) w.seek(p, end);
        }
        if (!ok && lane == 0) {
            // the copies in flight land (bounded) before shared memory is released
            atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
            for (int i = max(0, issued - NS * NU); i < issued; ++i) {
                const int pk = i / NU, v = i % NU;
                (void)mbar_wait_bounded(full(pk % NS, v == 0 ? NP : v - 1), (pk / NS) & 1);
            }
            if (q_issued > 0) (void)mbar_wait_bounded(bar(SM::B_QFULL), (q_issued - 1) & 1);
        }
    } else if (warp == 5) {
        // ================= products, whichever is ready first (the warp converged) ===========
        const bool lead = elect_one();
        const Desc d_q(smem_desc_sw128(sb + SM::OFF_Q, 16, 1024));
        const Desc d_k(smem_desc_sw128(sb + SM::OFF_C, 16, 1024));    // keys x dims
        const Desc d_v(smem_desc_sw128(sb + SM::OFF_C, kBlk, 1024));  // dims x keys
        const Desc d_p(smem_desc_sw128(sb + SM::OFF_P, 16, 1024));
        constexpr uint32_t ID_S = idesc_bf16(64, 2 * kRows, 0, 0);
        constexpr uint32_t ID_O = idesc_bf16(128, kRows, 1, 0);
        int s = 0, pv = 0, seg = 0;
        Walk ws = w, wp = w;  // the sequences of the next scores and of the next output product
        bool ok = true;
        unsigned long long t0 = 0;
        while (pv < n_pages) {
            bool moved = false;
            if (pv < s && mbar_test_warp(lead, bar(SM::B_P + (pv & 1)), (pv >> 1) & 1)) {
                // O^T += C^T P^T, unit by unit; each unit's page slot is free after it
                tc_fence_after();
                if (wp.at == wp.seg_end) wp.seek(p, end);
                const int st = pv % NS;
                const bool fresh = __all_sync(0xffffffffu, wp.at == wp.seg_begin);
                const Desc v = d_v.at(st * PAGE), pt = d_p.at((pv & 1) * kRows * 128);
#pragma unroll
                for (int u = 0; u < NP; ++u) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_if(lead, tmem + kTmemO + u * kRows, v.at(u * 2 * kBlk + kk * 2048),
                                pt.at(kk * 32), ID_O, (fresh && kk == 0) ? 0u : 1u);
                    umma_commit_if(lead, free_(st, u));
                }
                umma_commit_if(lead, bar(SM::B_O + (pv & 1)));
                ++wp.at;
                ++pv;
                moved = true;
            } else if (s < n_pages && s <= pv + 1) {
                // S^T = C [q~hi ; q~lo]^T once the page (and a new sequence's queries) landed: lane u
                // asks for unit u. The scores before last have been read: their output product is
                // issued. (Unit by unit as they land, the questions cost more than the products.)
                if (ws.at == ws.seg_end) ws.seek(p, end);
                const int st = s % NS;
                const bool asks = lane < NU || (lane == NU && ws.at == ws.seg_begin);
                if (mbar_test_warp(asks, lane < NU ? full(st, lane) : bar(SM::B_QFULL),
                                   (lane < NU ? s / NS : seg) & 1)) {
                    tc_fence_after();
                    const uint32_t d = tmem + kTmemS + (s & 1) * 64;
                    const Desc kd = d_k.at(st * PAGE);
#pragma unroll
                    for (int v = 0; v < NU; ++v) {
                        const int u = v == 0 ? NP : v - 1;  // the shared part's slot is free first
#pragma unroll
                        for (int kk = 0; kk < (u == NP ? 4 : 8); ++kk) {
                            const uint32_t off = u * 2 * kBlk + (kk >> 2) * kBlk + (kk & 3) * 32;
                            umma_if(lead, d, kd.at(off), d_q.at(off), ID_S, (v > 0 || kk > 0) ? 1u : 0u);
                        }
                        if (u == NP) umma_commit_if(lead, free_(st, NP));
                    }
                    umma_commit_if(lead, bar(SM::B_S + (s & 1)));
                    ++s;
                    if (__all_sync(0xffffffffu, ++ws.at == ws.seg_end)) {
                        umma_commit_if(lead, bar(SM::B_QFREE));
                        ++seg;
                    }
                    moved = true;
                }
            }
            if (moved) {
                t0 = 0;
            } else {
                const unsigned long long now = globaltimer_ns();
                if (t0 == 0) t0 = now;
                const bool late = now - t0 > kWaitLimitNs;
                if (late) *abort_flag = 1;
                if (__any_sync(0xffffffffu, late || *abort_flag)) {
                    ok = false;
                    break;
                }
            }
        }
        if (lead) {
            if (!ok) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
            // every product is done before TMEM and shared memory go (bounded)
            umma_commit(bar(SM::B_END));
            (void)mbar_wait_bounded(bar(SM::B_END), 0);
        }
        __syncwarp();
    } else {
        // ================= softmax and the partial results =====================================
        const bool lead = elect_one();
        const int c0 = (lane & 3) * 2;  // this thread's columns: 8j + c0, 8j + c0 + 1, j < 4
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        bool ok = true;
        int k = 0;
        while (ok && w.at < end) {
            const int b = w.b, L = p.seq_lens[b], page0 = w.page0;
            // the last position each of this thread's rows sees (-1: no such row)
            int last[8];
            float base[8], l[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = group * kRows + (j >> 1) * 8 + c0 + (j & 1);
                last[j] = r < p.nq * p.H ? L - p.nq + r / p.H : -1;
                base[j] = -INFINITY;
                l[j] = 0.f;
            }
            for (; w.at < w.seg_end; ++w.at, ++k) {
                const int st = k % NS, pos0 = (w.at - page0) * kPT;
                // the scores (their completion implies the earlier products', so P's tile of two
                // pages ago has been read) and, for page_ok, the page
                ok = wait_warp(lane < 2, lane ? full(st, 0) : bar(SM::B_S + (k & 1)),
                                        (lane ? k / NS : k >> 1) & 1, abort_flag);
                tc_fence_after();
                float s[16];  // [j][e]: column 8j + c0 + e % 2, key 16 warp + lane / 4 + 8 (e / 2)
                {
                    uint32_t r[32];
                    tmem_ld_16x256b_x8(tmem + kTmemS + (k & 1) * 64 + lanes, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[4 * j + e] = __uint_as_float(r[4 * j + e]) + __uint_as_float(r[16 + 4 * j + e]);
                }
                const bool good = page_ok[st] != 0;
                const int key0 = pos0 + warp * 16 + (lane >> 2);
                bool grew = false;
                if (!good || pos0 + kPT > L - p.nq + 1 || (group + 1) * kRows > p.nq * p.H) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!good || key0 + 8 * (e >> 1) > last[2 * j + (e & 1)]) s[4 * j + e] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) grew |= s[4 * j + e] > base[2 * j + (e & 1)] + kLazy;
                if (bar_softmax_or(grew || !ok)) {
                    ok = !bar_softmax_or(!ok);
                    if (!ok) break;
                    // some row outgrew its base: every row's new base is the maximum so far
                    float mx[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        mx[j] = fmaxf(s[4 * (j >> 1) + (j & 1)], s[4 * (j >> 1) + (j & 1) + 2]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], off));
                        if (lane < 4) s_red[warp][(j >> 1) * 8 + c0 + (j & 1)] = mx[j];
                    }
                    bar_softmax();
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = (j >> 1) * 8 + c0 + (j & 1);
                        const float m = fmaxf(fmaxf(fmaxf(s_red[0][c], s_red[1][c]),
                                                    fmaxf(s_red[2][c], s_red[3][c])), base[j]);
                        f[j] = m == -INFINITY ? 1.f : exp2f(base[j] - m);
                        base[j] = m;
                        l[j] *= f[j];
                    }
                    if (w.at > w.seg_begin) {
                        bar_softmax();  // the maxima have been read: their place takes the factors
                        if (warp == 0 && lane < 4)
#pragma unroll
                            for (int j = 0; j < 8; ++j) s_red[0][(j >> 1) * 8 + c0 + (j & 1)] = f[j];
                        bar_softmax();
                        ok = wait_warp(lead, bar(SM::B_O + ((k - 1) & 1)), ((k - 1) >> 1) & 1, abort_flag);
                        ok = !bar_softmax_or(!ok);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int u = 0; u < NP; ++u) {
                            uint32_t r[32];
                            tmem_ld32(tmem + kTmemO + u * kRows + lanes, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                r[c] = __float_as_uint(__uint_as_float(r[c]) * s_red[0][c]);
                            tmem_st32(tmem + kTmemO + u * kRows + lanes, r);
                        }
                        tmem_wait_st();
                    }
                    bar_softmax();  // s_red is free again
                }
                uint32_t pk[8];  // [j][key half]: two columns of one key
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float m0 = base[2 * j] == -INFINITY ? 0.f : base[2 * j];
                    const float m1 = base[2 * j + 1] == -INFINITY ? 0.f : base[2 * j + 1];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = ex2_approx(s[4 * j + 2 * e] - m0);
                        const float p1 = ex2_approx(s[4 * j + 2 * e + 1] - m1);
                        l[2 * j] += p0;
                        l[2 * j + 1] += p1;
                        pk[2 * j + e] = pack_bf16x2(p0, p1);
                    }
                }
                // P^T [32 rows][64 keys], rows of 128 bytes, 128-byte swizzle
                const uint32_t pt = sb + SM::OFF_P + (k & 1) * kRows * 128;
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    const int row = 8 * (2 * jj + (lane >> 4)) + (lane & 7);
                    stmatrix_x4_trans(pt + blk_off(row, (2 * warp + ((lane >> 3) & 1)) * 8), pk[4 * jj],
                                      pk[4 * jj + 1], pk[4 * jj + 2], pk[4 * jj + 3]);
                }
                if (!good || pos0 + kPT > L) {
                    // rows behind the sequence (or of a page that was not copied) hold anything: as
                    // values they are zeroed before the output product reads them
                    const int n_ok = good ? L - pos0 : 0;
                    for (int idx = tid; idx < (kPT - n_ok) * NP * 16; idx += 128) {
                        const int row = n_ok + idx / (NP * 16), ch = idx % (NP * 16);
                        *reinterpret_cast<uint4 *>(sm + SM::OFF_C + st * PAGE + (ch >> 3) * kBlk +
                                                   blk_off(row, (ch & 7) * 8)) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(SM::B_P + (k & 1)));
            }
            const size_t piece = part_index(p, range, b, group);
            float *ml = p.part_ml + piece * kRows * 2;
            if (ok) ok = wait_warp(lead, bar(SM::B_O + ((k - 1) & 1)), ((k - 1) >> 1) & 1, abort_flag);
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
            // sums of the keys over the lanes that share a column, then over the warps
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);
                if (lane < 4) s_red[warp][(j >> 1) * 8 + c0 + (j & 1)] = l[j];
            }
            bar_softmax();
            if (warp == 0 && lane < 4) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = (j >> 1) * 8 + c0 + (j & 1);
                    ml[2 * c] = base[j];
                    ml[2 * c + 1] = (s_red[0][c] + s_red[1][c]) + (s_red[2][c] + s_red[3][c]);
                }
            }
            bar_softmax();
            if (w.at < end) w.seek(p, end);
        }
        if (!ok && tid == 0) atomicOr(&g_err, HMD_DEVERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- kernel 3 ----------------------------------------------------------------------------------
constexpr int kExpThreads = 512;
constexpr int kExpWarps = kExpThreads / 32;
constexpr int kExpTok = 16;  // tokens (b, i) per cluster
template <int D>
struct ExpSmem {
    static constexpr int WP = 128 + 8;  // pitch (elements) without bank conflicts
    __nv_bfloat16 w[D][WP];             // W_uv[h][v][this CTA's 128 dims]
    __nv_bfloat16 hi[kExpTok][WP], lo[kExpTok][WP];
    float red[kExpWarps][128];          // a row's partial sums, per warp
    float out[kExpTok][D];              // this CTA's part of the output
    float den[kExpWarps];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

// Grid (d_c / 128, H, token blocks), clusters along x.
template <int D>
__global__ void __launch_bounds__(kExpThreads) latent_expand_kernel(const LatentParams p) {
    extern __shared__ __align__(16) uint8_t exp_smem[];
    ExpSmem<D> &sm = *reinterpret_cast<ExpSmem<D> *>(exp_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cc = blockIdx.x, h = blockIdx.y, tok0 = blockIdx.z * kExpTok;
    const int n_cols = p.dc / 128, rows = min(kExpTok, p.B * p.nq - tok0);
    griddep_launch_dependents();
    griddep_wait();
    const __nv_bfloat16 *wv = p.w_uv + h * p.w_uv_head + cc * 128;
    for (int idx = tid; idx < D * 16; idx += kExpThreads) {
        const int v = idx >> 4, c = (idx & 15) * 8;
        cp_async16(smem_u32(&sm.w[v][c]), wv + (size_t)v * p.dc + c);  // lands during the merge
    }
    // merge the ranges: `wpr` warps share a token's ranges, lanes its 128 dims (4 each)
    const int wpr = rows > 8 ? 1 : rows > 4 ? 2 : rows > 2 ? 4 : rows > 1 ? 8 : 16;
    uint32_t missing = 0;  // tokens of which a range gave up
    for (int r0 = 0; r0 < rows; r0 += kExpWarps / wpr) {
        const int r = r0 + warp / wpr, part = warp % wpr;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float M = -INFINITY, den = 0.f;
        bool lost = false;
        if (r < rows) {
            const int tok = tok0 + r, b = tok / p.nq, row = (tok - b * p.nq) * p.H + h;
            const int2 range = p.ranges[b];
            const int i0 = range.x, i1 = range.y;
            const int g = row / kRows, c = row % kRows;
            for (int i = i0 + lane; i < i1; i += 32) {
                const float2 v = *reinterpret_cast<const float2 *>(
                    p.part_ml + (part_index(p, i, b, g) * kRows + c) * 2);
                M = fmaxf(M, v.x);
                lost |= v.y < 0.f;
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            lost = __any_sync(0xffffffffu, lost);
            if (!lost && M != -INFINITY) {
#pragma unroll 8
                for (int i = i0 + part; i < i1; i += wpr) {
                    const size_t at = part_index(p, i, b, g) * kRows + c;
                    const float2 v = *reinterpret_cast<const float2 *>(p.part_ml + at * 2);
                    const float4 x = *reinterpret_cast<const float4 *>(p.part_o + at * p.dc + cc * 128 + lane * 4);
                    const float f = exp2f(v.x - M);
                    den += f * v.y;
                    acc.x += f * x.x; acc.y += f * x.y; acc.z += f * x.z; acc.w += f * x.w;
                }
            }
        }
        if (wpr > 1) {
            *reinterpret_cast<float4 *>(&sm.red[warp][lane * 4]) = acc;
            if (lane == 0) sm.den[warp] = den;
            __syncthreads();
            if (part == 0)
                for (int v = 1; v < wpr; ++v) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.red[warp + v][lane * 4]);
                    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
                    den += sm.den[warp + v];
                }
            __syncthreads();
        }
        if (part == 0 && r < rows) {
            const float inv = den > 0.f ? 1.f / den : 0.f;
            const float x[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
            const uint32_t h0 = pack_bf16x2(x[0], x[1]), h1 = pack_bf16x2(x[2], x[3]);
            *reinterpret_cast<uint2 *>(&sm.hi[r][lane * 4]) = make_uint2(h0, h1);
            *reinterpret_cast<uint2 *>(&sm.lo[r][lane * 4]) =
                make_uint2(pack_bf16x2(x[0] - bf16_lo(h0), x[1] - bf16_hi(h0)),
                           pack_bf16x2(x[2] - bf16_lo(h1), x[3] - bf16_hi(h1)));
        }
        if (r < rows && lost) missing |= 1u << r;
    }
    for (int r = rows + warp; r < kExpTok; r += kExpWarps) {  // rows without a token
        *reinterpret_cast<uint2 *>(&sm.hi[r][lane * 4]) = make_uint2(0u, 0u);
        *reinterpret_cast<uint2 *>(&sm.lo[r][lane * 4]) = make_uint2(0u, 0u);
    }
    // a warp knows the losses of the tokens it merged; the output needs all of them
    __shared__ uint32_t s_missing;
    if (tid == 0) s_missing = 0;
    cp_async_wait_all();
    __syncthreads();
    if (lane == 0 && missing) atomicOr(&s_missing, missing);
    // out[16 tokens][D] = latent output x W_uv^T over this CTA's dims; a warp takes 8 columns
    if (warp < D / 8) {
        float acc[4] = {};
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            uint32_t ah[4], al[4];
            ldmatrix_x4(smem_u32(&sm.hi[lane & 15][kk * 16 + (lane >> 4) * 8]), ah[0], ah[1], ah[2], ah[3]);
            ldmatrix_x4(smem_u32(&sm.lo[lane & 15][kk * 16 + (lane >> 4) * 8]), al[0], al[1], al[2], al[3]);
            const __nv_bfloat16 *wr = &sm.w[warp * 8 + (lane >> 2)][kk * 16 + (lane & 3) * 2];
            const uint32_t b0 = *reinterpret_cast<const uint32_t *>(wr);
            const uint32_t b1 = *reinterpret_cast<const uint32_t *>(wr + 8);
            mma_bf16_16816(acc, ah, b0, b1);
            mma_bf16_16816(acc, al, b0, b1);
        }
        const int v = warp * 8 + (lane & 3) * 2;
        *reinterpret_cast<float2 *>(&sm.out[lane >> 2][v]) = make_float2(acc[0], acc[1]);
        *reinterpret_cast<float2 *>(&sm.out[(lane >> 2) + 8][v]) = make_float2(acc[2], acc[3]);
    }
    cluster_sync_all();
    // every CTA of the cluster finishes a share of the elements, adding the parts in rank order
    const uint32_t me = cluster_rank();
    for (int idx = (int)me * kExpThreads + tid; idx < rows * (D / 2); idx += n_cols * kExpThreads) {
        const int r = idx / (D / 2), v = idx % (D / 2) * 2;
        if ((s_missing >> r) & 1u) continue;  // o stays as it was
        float y[4][2];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            y[c][0] = c < n_cols ? ld_cluster_f32(smem_u32(&sm.out[r][v]), c) : 0.f;
            y[c][1] = c < n_cols ? ld_cluster_f32(smem_u32(&sm.out[r][v + 1]), c) : 0.f;
        }
        const float x0 = ((y[0][0] + y[1][0]) + y[2][0]) + y[3][0];
        const float x1 = ((y[0][1] + y[1][1]) + y[2][1]) + y[3][1];
        *reinterpret_cast<uint32_t *>(p.o + ((size_t)(tok0 + r) * p.H + h) * D + v) = pack_bf16x2(x0, x1);
    }
    cluster_sync_all();  // nobody leaves while its part is still read
}

// ---- host side ---------------------------------------------------------------------------------
int device_sms() {
    return once_per_device([] {
        int dev = 0, v = 0;
        if (cudaGetDevice(&dev) == cudaSuccess &&
            cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
            return v;
        cudaGetLastError();
        return 148;
    });
}

struct Plan {
    int n_groups, n_ranges;
    size_t off_o, off_ml, off_start, off_ranges, off_cum, bytes;
};
Plan make_plan(int nq, int B, int H, int dc, int max_seq_len) {
    Plan pl;
    pl.n_groups = (int)(((long long)nq * H + kRows - 1) / kRows);
    const long long pages = (long long)B * ((max_seq_len + kPT - 1) / kPT);
    // one CTA per SM: the groups of one range run side by side and share its pages through L2
    pl.n_ranges = (int)std::min<long long>(std::max(1, device_sms() / pl.n_groups), pages);
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
cudaError_t launch_attend(const CUtensorMap &tm, const LatentParams &p, cudaStream_t s) {
    constexpr int smem = (int)AttSmem<NP>::ALLOC + 1024;
    const cudaError_t e = once_per_device([] {
        return cudaFuncSetAttribute(latent_attend_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)AttSmem<NP>::ALLOC + 1024);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(latent_attend_kernel<NP>, dim3((unsigned)(p.n_ranges * p.n_groups)),
                      dim3(kAttThreads), smem, s, tm, p);
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

template <int D>
cudaError_t launch_expand(const LatentParams &p, cudaStream_t s) {
    const cudaError_t e = once_per_device([] {
        return cudaFuncSetAttribute(latent_expand_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(ExpSmem<D>));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.dc / 128), (unsigned)p.H,
                       (unsigned)((p.B * p.nq + kExpTok - 1) / kExpTok));
    cfg.blockDim = dim3(kExpThreads);
    cfg.dynamicSmemBytes = sizeof(ExpSmem<D>);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)(p.dc / 128);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, latent_expand_kernel<D>, p);
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
    CUtensorMap tm;
    if (!make_tmap_pool_sw128(&tm, a.pool, a.n_pages, 1, a.d_c + kDR)) return cudaErrorInvalidValue;
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
    cudaError_t e = a.d == 128 ? launch_absorb<128>(p, s) : launch_absorb<64>(p, s);
    if (e != cudaSuccess) return e;
    switch (a.d_c / 128) {
        case 1: e = launch_attend<1>(tm, p, s); break;
        case 2: e = launch_attend<2>(tm, p, s); break;
        case 3: e = launch_attend<3>(tm, p, s); break;
        default: e = launch_attend<4>(tm, p, s); break;
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
