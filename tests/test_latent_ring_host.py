"""The ring of key and value blocks in the prompt attention of the latent expanded form: no wait of
the copies for a product can be overtaken.

The copy warp asks a barrier whether phase k is complete by its parity, so it can tell phase k from
k + 1 and no further: once k + 1 is complete too, the answer is "not yet" until k + 2. This walks the
kernel's own schedule (csrc/latent_ring.h, compiled for the host) with product warps that are as fast as
the blocks in the ring allow, and checks that never happens, whatever the timing.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include "hybrid_mixer_decoding_b200/csrc/latent_ring.h"
using namespace hmd;
template <int D> void walk(int n_tiles) {
    using S = RingShape<D>;
    RingPlace<D> at;
    for (int n = 0; n < n_tiles * S::NB; ++n, at.next(n_tiles)) {
        const int i = at.tile(n_tiles), key = at.key(n_tiles);
        std::printf("%d %d %d %d %d %d %d %d %d %d\n", D, n_tiles, n, i, key, at.block(n_tiles),
                    (int)at.freed_by(n_tiles), ring_barrier(i), ring_parity(i),
                    key ? ring_key<D>(i) : ring_value<D>(i, n_tiles));
    }
}
int main() {
    std::printf("%d %d\n", RingShape<128>::NR, RingShape<64>::NR);
    for (int n = 1; n <= 40; ++n) { walk<128>(n); walk<64>(n); }
}
"""
KEYS, SCORES, OUTPUT = 0, 1, 2


@pytest.fixture(scope="module")
def schedule(tmp_path_factory):
    gxx = shutil.which("g++") or shutil.which("c++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-I", ROOT, str(d / "ring.cpp"), "-o", str(d / "ring")], check=True)
    lines = subprocess.run([str(d / "ring")], check=True, capture_output=True, text=True).stdout.splitlines()
    slots = dict(zip((128, 64), map(int, lines[0].split())))
    walks = {}
    for line in lines[1:]:
        head, n_tiles, *rest = map(int, line.split())
        walks.setdefault((head, n_tiles), []).append(rest)
    return slots, walks


def phases_done(walk, loaded):
    """Completed products of each kind, in tiles, once `loaded` blocks of the stream are in the ring (or
    have been): the last query tile's scores of the tiles whose keys, outputs whose values are there."""
    done = {}
    for kind in (KEYS, SCORES, OUTPUT):
        n, tiles = 0, 1 + max(i for _, i, *_ in walk)
        for i in range(tiles):
            need = [r[0] for r in walk if r[1] == i and r[4] == kind or
                    (kind == SCORES and r[1] == i and r[4] == KEYS)]
            if max(need) >= loaded:
                break
            n = i + 1
        done[kind] = n
    return done


@pytest.mark.parametrize("d", [128, 64])
def test_blocks_come_in_the_order_the_products_expect(schedule, d):
    slots, walks = schedule
    for n_tiles in range(1, 41):
        walk = walks[d, n_tiles]
        kb, vb = d // 64 + 1, d // 64
        assert [r[0] for r in walk] == list(range(n_tiles * (kb + vb)))
        for key, count in ((1, kb), (0, vb)):
            for i in range(n_tiles):
                at = [r for r in walk if r[1] == i and r[2] == key]
                assert [r[3] for r in at] == list(range(count))
                assert [r[0] for r in at] == list(range(at[0][7], at[0][7] + count))


@pytest.mark.parametrize("d", [128, 64])
def test_no_wait_of_the_copies_is_overtaken(schedule, d):
    slots, walks = schedule
    for n_tiles in range(1, 41):
        walk = walks[d, n_tiles]
        for n in range(slots[d], len(walk)):
            _, i, _, _, kind, barrier, parity, _ = walk[n - slots[d]]
            done = phases_done(walk, n)[kind]
            assert done > i  # what it waits for can complete with the blocks that are there
            # phases of that barrier: the tiles that share it
            same = [j for j in range(n_tiles) if walk_barrier(walk, j) == barrier]
            phase = same.index(i)
            assert parity == phase % 2
            complete = sum(j < done for j in same)
            assert complete <= phase + 1, (d, n_tiles, n, i, kind)


def walk_barrier(walk, tile):
    return next(r[5] for r in walk if r[1] == tile)
