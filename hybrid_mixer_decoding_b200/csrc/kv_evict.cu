// Eviction from a paged KV cache by accumulated attention weight.
//
// Of a sequence's L entries, each kv-head keeps the `recent` latest and, of the n = L - recent
// others, those with the largest accumulated weight, `budget` in all, and packs them in their
// order: kept[0] < kept[1] < ..., entry kept[i] moves to position i. Attention over a set of keys
// does not depend on their order, so the packed cache decodes as the same set of keys.
//
// Kernel 1 (choose), one cluster of 1 to 8 CTAs per (sequence, kv-head): the m-th largest of n weights
// is found digit by digit (11, 11 and 10 bits of the weight's order-preserving integer, a
// histogram in shared memory per digit, added up over the cluster). Then each warp counts and,
// after one scan over the warps and CTAs, writes the entries of its own contiguous stretch: above
// the threshold, or equal to it while equal ones are still wanted, lowest index first. The
// weights are read once, into shared memory, unless a CTA's share is above kCacheKeys.
// Kernel 2 (move): rows of K and V and the weights go to their places. Into other pages, every
// row is independent. Within the same pages, kept[i] >= i means that a destination is a source
// of earlier rows only: one CTA owns one 64-byte column of the rows of a (sequence, kv-head) and
// walks them in order, a barrier between a block's loads and its stores.
// Kernel 2 is bound by memory: it reads and writes each kept row once (B = 32, Hkv = 8, d = 128, half of
// up to 8192 entries into other pages: 178 us at 6.0 TB/s read and written). Kernel 1 reads each weight
// once but is bound by latency: three digits, each a pass, a barrier over the cluster and a scan (14 us
// there; 24 us for 16 heads of 100,000 entries on 8 CTAs each; on one CTA each the whole call took 155 us
// instead of 55). A digit that settles the choice ends the search.
#include <cuda_bf16.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "../../include/hmd.h"

namespace hmd {
namespace {

__device__ unsigned int g_err;

constexpr int kPT = 64;               // tokens per page
constexpr int kChooseThreads = 1024;
constexpr int kWarps = kChooseThreads / 32;
constexpr int kBins = 2048;           // 11 bits a digit
constexpr int kCacheKeys = 49152;     // weights held in shared memory: 192 KiB
constexpr int kMaxRanks = 8;          // CTAs of a cluster (of 16, few fit at once: 58 us instead of 24)
constexpr int kShare = 4096;          // a CTA of a cluster has at least this many entries
constexpr int kMoveThreads = 256;
constexpr int kRowsPerBlock = 64;     // rows moved by one CTA into other pages

// Order-preserving integer of a weight; -0 is 0, and NaN comes above everything.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Row {
    int L, slot, n_keep, n_old, m;  // n_old: entries before the recent ones, m of them are kept
    bool ok;
};
__device__ __forceinline__ Row row_of(const EvictArgs &a, int b) {
    Row r;
    r.L = a.seq_lens[b];
    r.slot = a.slots ? a.slots[b] : b;
    r.ok = r.L >= 0 && r.L <= a.max_seq_len && r.slot >= 0 && r.slot < a.n_slots;
    if (!r.ok) r.L = 0;
    r.n_keep = min(r.L, a.budget);
    const int recent = min(r.L, a.recent);
    r.n_old = r.L - recent;
    r.m = r.n_keep - recent;
    return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint2 ld_cluster_u2(const void *at, uint32_t rank) {
    uint32_t remote;
    uint2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(at)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(remote) : "memory");
    return v;
}

// Grid (sequence, kv-head) x cluster size, clusters along x: CTA `rank` holds the entries
// [rank * share, (rank + 1) * share) of the n_old ones.
// CACHED: the share's order keys are held in shared memory; else they are formed again per digit.
template <bool CACHED>
__global__ void __launch_bounds__(kChooseThreads, 2) evict_choose_kernel(const EvictArgs a, int n_ranks) {
    extern __shared__ uint32_t keys[];
    __shared__ __align__(8) uint32_t hist[3][kBins];  // one per digit: a slower CTA may still read
    __shared__ uint32_t warp_gt[kWarps], warp_eq[kWarps];
    __shared__ __align__(8) uint32_t s_count[2];      // this CTA's keys above and at the threshold
    __shared__ uint32_t s_digit, s_left, s_whole;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = n_ranks > 1 ? (int)cluster_rank() : 0, bg = blockIdx.x / n_ranks;
    const int b = bg / a.Hkv, g = bg - b * a.Hkv;
    for (int i = tid; i < 3 * kBins; i += kChooseThreads) hist[0][i] = 0;
    griddep_launch_dependents();
    griddep_wait();  // the weights and lengths come from the steps before
    const Row r = row_of(a, b);
    if (!r.ok && tid == 0 && g == 0 && rank == 0) {
        const int L = a.seq_lens[b];
        atomicOr(&g_err, (L < 0 || L > a.max_seq_len) ? HMD_DEVERR_SEQLEN : HMD_DEVERR_SLOT);
    }
    int32_t *kept = a.kept + (size_t)bg * a.budget;
    const int t_all = rank * kChooseThreads + tid, n_all = n_ranks * kChooseThreads;
    for (int i = r.n_keep + t_all; i < a.budget; i += n_all) kept[i] = -1;
    for (int i = r.m + t_all; i < r.n_keep; i += n_all) kept[i] = r.n_old + (i - r.m);
    if (r.m == r.n_old) {  // nothing to evict
        for (int i = t_all; i < r.m; i += n_all) kept[i] = i;
        return;
    }
    if (r.m == 0) return;  // the recent ones alone
    // this CTA's entries: whole 32-entry groups
    const int share = ((r.n_old + 31) / 32 + n_ranks - 1) / n_ranks * 32;
    const int e0 = min(r.n_old, rank * share), n = min(r.n_old, e0 + share) - e0;
    const float *w = a.weights + ((size_t)r.slot * a.Hkv + g) * a.w_len + e0;
    auto key_at = [&](int i) { return CACHED ? keys[i] : order_key(w[i]); };
    __syncthreads();  // the histograms are zero
    for (int i0 = tid; i0 < n; i0 += 8 * kChooseThreads) {
        float x[8];  // eight loads in flight: none waits for a histogram's atomics
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + u * kChooseThreads < n) x[u] = __ldg(w + i0 + u * kChooseThreads);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * kChooseThreads;
            if (i >= n) break;
            const uint32_t k = order_key(x[u]);
            if (CACHED) keys[i] = k;
            atomicAdd(&hist[0][k >> 21], 1u);
        }
    }
    // the m-th largest key: `left` of the keys that share the digits found so far are wanted
    uint32_t prefix = 0, mask = 0, left = (uint32_t)r.m;
#pragma unroll 1
    for (int digit = 0; digit < 3; ++digit) {
        const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
        const uint32_t bits = digit == 2 ? 0x3ffu : 0x7ffu;
        if (digit > 0) {
#pragma unroll 8
            for (int i = tid; i < n; i += kChooseThreads) {
                const uint32_t k = key_at(i);
                if ((k & mask) == prefix) atomicAdd(&hist[digit][(k >> shift) & bits], 1u);
            }
        }
        if (n_ranks > 1) cluster_sync_all();
        else __syncthreads();
        // counts from the largest digit down: thread t holds digits 2047 - 2t and 2046 - 2t
        const uint32_t *at = &hist[digit][kBins - 2 - 2 * tid];
        uint2 v = *reinterpret_cast<const uint2 *>(at);
        uint32_t c0 = v.y, c1 = v.x;
        if (n_ranks > 1) {
            uint2 x[kMaxRanks];  // all ranks' counts in flight at once
#pragma unroll
            for (int q = 0; q < kMaxRanks; ++q)
                x[q] = q < n_ranks && q != rank ? ld_cluster_u2(at, q) : make_uint2(0, 0);
#pragma unroll
            for (int q = 0; q < kMaxRanks; ++q) {
                c0 += x[q].y;
                c1 += x[q].x;
            }
        }
        uint32_t sum = c0 + c1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += up;
        }
        if (lane == 31) warp_gt[warp] = sum;
        __syncthreads();
        // keys with a larger digit
        const uint32_t before = sum - c0 - c1 + __reduce_add_sync(0xffffffffu, lane < warp ? warp_gt[lane] : 0u);
        if (before < left && left <= before + c0) {
            s_digit = kBins - 1 - 2 * tid;
            s_left = left - before;
            s_whole = left == before + c0;
        } else if (before + c0 < left && left <= before + c0 + c1) {
            s_digit = kBins - 2 - 2 * tid;
            s_left = left - before - c0;
            s_whole = left == before + c0 + c1;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= bits << shift;
        left = s_left;
        if (s_whole) {  // every key that shares these digits is wanted: no further digit decides
            prefix -= 1;  // not 0: less than all keys are wanted
            left = 0;
            break;
        }
    }
    // each warp's stretch of whole 32-entry groups: count, scan over the warps and CTAs, write
    const int per_warp = ((n + 31) / 32 + kWarps - 1) / kWarps * 32;
    const int i0 = min(n, warp * per_warp), i1 = min(n, i0 + per_warp);
    uint32_t n_gt = 0, n_eq = 0;
#pragma unroll 8
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t k = key_at(i);
        n_gt += k > prefix;
        n_eq += k == prefix;
    }
    n_gt = __reduce_add_sync(0xffffffffu, n_gt);
    n_eq = __reduce_add_sync(0xffffffffu, n_eq);
    if (lane == 0) {
        warp_gt[warp] = n_gt;
        warp_eq[warp] = n_eq;
    }
    __syncthreads();
    uint32_t gt = 0, eq = 0;  // keys above and at the threshold before this stretch
    if (n_ranks > 1) {
        if (warp == 0) {
            const uint32_t g_all = __reduce_add_sync(0xffffffffu, warp_gt[lane]);
            const uint32_t e_all = __reduce_add_sync(0xffffffffu, warp_eq[lane]);
            if (lane == 0) {
                s_count[0] = g_all;
                s_count[1] = e_all;
            }
        }
        cluster_sync_all();
        uint2 x[kMaxRanks];
#pragma unroll
        for (int q = 0; q < kMaxRanks; ++q) x[q] = q < rank ? ld_cluster_u2(s_count, q) : make_uint2(0, 0);
#pragma unroll
        for (int q = 0; q < kMaxRanks; ++q) {
            gt += x[q].x;
            eq += x[q].y;
        }
    }
    gt += __reduce_add_sync(0xffffffffu, lane < warp ? warp_gt[lane] : 0u);
    eq += __reduce_add_sync(0xffffffffu, lane < warp ? warp_eq[lane] : 0u);
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? key_at(i + lane) : 0u;
        const uint32_t is_gt = __ballot_sync(0xffffffffu, i + lane < i1 && k > prefix);
        const uint32_t is_eq = __ballot_sync(0xffffffffu, i + lane < i1 && k == prefix);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t my_gt = gt + __popc(is_gt & below), my_eq = eq + __popc(is_eq & below);
        const bool take = ((is_gt >> lane) & 1u) || (((is_eq >> lane) & 1u) && my_eq < left);
        if (take) kept[my_gt + min(my_eq, left)] = e0 + i + lane;
        gt += __popc(is_gt);
        eq += __popc(is_eq);
    }
    if (n_ranks > 1) cluster_sync_all();  // nobody leaves while its counts are still read
}

// Row address of position i under a table (nullptr and an error for a page outside the pool).
__device__ __forceinline__ size_t row_index(const EvictArgs &a, const int32_t *table, int max_pages,
                                            int b, int g, int i, bool &ok) {
    const int lp = i / kPT;
    const int pg = lp < max_pages ? table[(size_t)b * max_pages + lp] : -1;
    ok = pg >= 0 && pg < a.n_pages;
    if (!ok) atomicOr(&g_err, HMD_DEVERR_PAGE);
    return ((size_t)pg * a.Hkv + g) * kPT + i % kPT;
}

// Into other pages: one CTA per (sequence, kv-head, 64 rows); d / 8 lanes carry a row of K and
// the same row of V, 16 bytes each.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int n_chunks,
                                                                  bool move_weights) {
    griddep_launch_dependents();
    griddep_wait();  // kept is the choosing kernel's output
    const int tid = threadIdx.x, bg = blockIdx.x / n_chunks, chunk = blockIdx.x - bg * n_chunks;
    const int b = bg / a.Hkv, g = bg - b * a.Hkv;
    const int32_t *kept = a.kept + (size_t)bg * a.budget;
    if (g == 0 && chunk == 0 && tid == 0) a.new_lens[b] = row_of(a, b).n_keep;
    const int row0 = chunk * kRowsPerBlock, lpr = a.d / 8, rows_at_once = kMoveThreads / lpr;
    const int c = (tid % lpr) * 8;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k_pool);
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_pool);
#pragma unroll 4
    for (int i = row0 + tid / lpr; i < min(row0 + kRowsPerBlock, a.budget); i += rows_at_once) {
        const int j = kept[i];
        if (j < 0) break;
        bool ok_s, ok_d;
        const size_t src = row_index(a, a.page_table, a.max_pages, b, g, j, ok_s) * a.d + c;
        const size_t dst = row_index(a, a.dst_table, a.dst_max_pages, b, g, i, ok_d) * a.d + c;
        if (!ok_s || !ok_d) continue;
        const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(k + src));
        const uint4 y = __ldcs(reinterpret_cast<const uint4 *>(v + src));
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.k_pool) + dst) = x;
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.v_pool) + dst) = y;
    }
    if (move_weights && tid < kRowsPerBlock && row0 + tid < a.budget) {
        const int j = kept[row0 + tid];
        const int slot = a.slots ? a.slots[b] : b;
        if (j >= 0)
            a.weights_out[((size_t)slot * a.Hkv + g) * a.w_out_len + row0 + tid] =
                a.weights[((size_t)slot * a.Hkv + g) * a.w_len + j];
    }
}

// Within the same pages: CTA (sequence, kv-head, column). Columns 0 .. d/32-1 are 64-byte
// columns of K, the next d/32 of V, the last one the weights (if they are packed in place).
__global__ void __launch_bounds__(kMoveThreads) evict_pack_kernel(const EvictArgs a, int n_cols,
                                                                  bool pack_rows) {
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, bg = blockIdx.x / n_cols, col = blockIdx.x - bg * n_cols;
    const int b = bg / a.Hkv, g = bg - b * a.Hkv;
    const int32_t *kept = a.kept + (size_t)bg * a.budget;
    const int n = min(a.budget, a.max_seq_len);  // -1 from there on
    if (pack_rows && bg % a.Hkv == 0 && col == 0 && tid == 0) a.new_lens[b] = row_of(a, b).n_keep;
    if (!pack_rows || col == a.d / 16) {  // the weights: 4-byte rows
        const int slot = a.slots ? a.slots[b] : b;
        if (slot < 0 || slot >= a.n_slots) return;  // reported by the choosing kernel
        const float *w = a.weights + ((size_t)slot * a.Hkv + g) * a.w_len;
        float *out = a.weights_out + ((size_t)slot * a.Hkv + g) * a.w_out_len;
        for (int i0 = 0; i0 < n; i0 += 4 * kMoveThreads) {
            float x[4];
            int j[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * kMoveThreads + tid;
                j[u] = i < n ? kept[i] : -1;
                x[u] = j[u] >= 0 ? w[j[u]] : 0.f;
            }
            __syncthreads();  // every load of this block before any store into its sources
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (j[u] >= 0) out[i0 + u * kMoveThreads + tid] = x[u];
        }
        return;
    }
    const int cols = a.d / 32;
    __nv_bfloat16 *pool = static_cast<__nv_bfloat16 *>(col < cols ? a.k_pool : a.v_pool);
    const int c = (col % cols) * 32 + (tid & 3) * 8;
    constexpr int kRows = kMoveThreads / 4, kUnroll = 8;
    for (int i0 = 0; i0 < n; i0 += kUnroll * kRows) {
        uint4 x[kUnroll];
        int j[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kRows + tid / 4;
            j[u] = i < n ? kept[i] : -1;
            if (j[u] == i) j[u] = -1;  // already there
            if (j[u] >= 0) {
                bool ok;
                const size_t src = row_index(a, a.page_table, a.max_pages, b, g, j[u], ok);
                if (ok) x[u] = *reinterpret_cast<const uint4 *>(pool + src * a.d + c);
                else j[u] = -1;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (j[u] < 0) continue;
            bool ok;
            const size_t dst = row_index(a, a.page_table, a.max_pages, b, g,
                                         i0 + u * kRows + tid / 4, ok);
            if (ok) *reinterpret_cast<uint4 *>(pool + dst * a.d + c) = x[u];
        }
    }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs &a, cudaStream_t s) {
    const cudaError_t attr_err = once_per_device([] {
        return cudaFuncSetAttribute(evict_choose_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kCacheKeys * 4);
    });
    if (attr_err != cudaSuccess) return attr_err;
    const int heads = a.B * a.Hkv;
    // Split an entry list over a cluster while every CTA keeps at least kShare entries and the
    // clusters of all heads fit the GPU at once (two CTAs per SM, which shared memory allows up to about
    // 22,000 cached entries a CTA; longer shares run in two rounds).
    int n_ranks = 1;
    while (n_ranks < kMaxRanks && a.max_seq_len / (2 * n_ranks) >= kShare && heads * n_ranks <= sm_count()) n_ranks *= 2;
    const int share = ((a.max_seq_len + 31) / 32 + n_ranks - 1) / n_ranks * 32;
    const bool cached = share <= kCacheKeys;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(heads * n_ranks));
    cfg.blockDim = dim3(kChooseThreads);
    cfg.dynamicSmemBytes = cached ? (size_t)share * 4 : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)n_ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = n_ranks > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, cached ? evict_choose_kernel<true> : evict_choose_kernel<false>, a, n_ranks);
    if (e != cudaSuccess) return e;
    const bool same_pages = a.dst_table == a.page_table, same_weights = a.weights_out == a.weights;
    if (!same_pages) {
        const int keep = std::min(a.budget, a.max_seq_len);
        const int n_chunks = (keep + kRowsPerBlock - 1) / kRowsPerBlock;
        e = launch_pdl(evict_move_kernel, dim3((unsigned)(heads * n_chunks)), dim3(kMoveThreads), 0,
                       s, a, n_chunks, !same_weights);
        if (e != cudaSuccess || !same_weights) return e;
        return launch_pdl(evict_pack_kernel, dim3((unsigned)heads), dim3(kMoveThreads), 0, s, a, 1,
                          false);
    }
    // packing the weights in order is right whether or not weights_out is another buffer
    const int n_cols = a.d / 16 + 1;
    return launch_pdl(evict_pack_kernel, dim3((unsigned)(heads * n_cols)), dim3(kMoveThreads), 0, s,
                      a, n_cols, true);
}

uint32_t kv_evict_read_errors(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_err, sizeof v) != cudaSuccess) return 0;
    if (clear && v) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_err, &z, sizeof z);
    }
    return v;
}

}  // namespace hmd
