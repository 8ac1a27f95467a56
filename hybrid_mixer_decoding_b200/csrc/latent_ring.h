// The order in which the prompt attention of the latent expanded form streams keys and values through
// its ring of shared-memory blocks, and which product frees each block. Plain C++, so that the host
// can walk the same schedule.
#pragma once

#ifdef __CUDACC__
#define HMD_RING_FN __host__ __device__ constexpr
#else
#define HMD_RING_FN constexpr
#endif

namespace hmd {

// A key tile has KB blocks, a value tile VB; block n of the stream goes to slot n % NR.
template <int D>
struct RingShape {
    static constexpr int KB = D / 64 + 1, VB = D / 64, NB = KB + VB;
    static constexpr int NR = D == 128 ? 8 : 5;  // what shared memory holds beside the queries
};

// Each kind of product has kRingPhases barriers, the tiles in turn, so that a barrier's phase completes
// only every second tile. A waiter can tell a phase from the one after it and no further; the copies
// ask for a tile's product when the next tile's may be complete (its blocks are in the ring before),
// but that of the tile after next never is: its last block is the one to be loaded or a later one.
constexpr int kRingPhases = 2;
HMD_RING_FN int ring_barrier(int tile) { return (int)((unsigned)tile % kRingPhases); }
HMD_RING_FN int ring_parity(int tile) { return (int)((unsigned)tile / kRingPhases) & 1; }

// What frees a block: the last query tile's scores (all but a key tile's last block a little earlier,
// by the products up to it) or its output.
enum RingFree { kFreeKeys, kFreeScores, kFreeOutput };

// A block of the stream K_0, K_1, V_0, K_2, V_1, ..., V_(n_tiles - 1): block u of K_g and V_(g-1).
template <int D>
struct RingPlace {
    using S = RingShape<D>;
    int g = 0, u = 0;
    HMD_RING_FN void next(int n_tiles) {
        if (++u == (g == 0 ? S::KB : g < n_tiles ? S::NB : S::VB)) {
            u = 0;
            ++g;
        }
    }
    HMD_RING_FN bool key(int n_tiles) const { return g < n_tiles && u < S::KB; }
    HMD_RING_FN int tile(int n_tiles) const { return key(n_tiles) ? g : g - 1; }
    // block of its key or value tile
    HMD_RING_FN int block(int n_tiles) const { return key(n_tiles) || g == n_tiles ? u : u - S::KB; }
    HMD_RING_FN RingFree freed_by(int n_tiles) const {
        return !key(n_tiles) ? kFreeOutput : u < S::KB - 1 ? kFreeKeys : kFreeScores;
    }
};

// First blocks of K_i and V_i in the stream.
template <int D>
HMD_RING_FN int ring_key(int i) {
    return i == 0 ? 0 : i * RingShape<D>::NB - RingShape<D>::VB;
}
template <int D>
HMD_RING_FN int ring_value(int i, int n_tiles) {
    return (i + 1) * RingShape<D>::NB - RingShape<D>::VB + (i + 1 < n_tiles ? RingShape<D>::KB : 0);
}

}  // namespace hmd
