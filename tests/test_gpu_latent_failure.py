"""A copy that never lands, in the latent kernels and the scored step: the CTA gives up within its limit,
reports HMD_DEVERR_TIMEOUT and leaves what depends on it as it was; every other output, and the next call,
equals an undisturbed run bit for bit. See test_gpu_failure.py for the hook."""
import pytest
import torch

import hybrid_mixer_decoding_b200 as hmd
from hybrid_mixer_decoding_b200 import _lib
from test_gpu_evict import Cache, new_tokens, scored
from test_gpu_latent import Latent, prefill

pytestmark = pytest.mark.gpu
WAIT_NS = 1_000_000  # 1 ms
KEPT = 9.0  # what the outputs hold before


def run_thrice(call, kernel, cta, pool):
    """(outputs of an undisturbed call, of one with a missing copy); checks errors and a third call."""
    before = pool.clone()
    assert hmd.hmd_device_errors(clear=True) == 0
    want = call()
    torch.cuda.synchronize()
    assert hmd.hmd_device_errors(clear=True) == 0
    appended = pool.clone()
    pool.copy_(before)
    hmd.hmd_test_arm_copy_skip(kernel, cta, WAIT_NS)
    got = call()
    torch.cuda.synchronize()
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_TIMEOUT
    assert torch.equal(pool.view(torch.int16), appended.view(torch.int16))
    assert torch.equal(call(), want)
    assert hmd.hmd_device_errors(clear=True) == 0
    return want, got


def check_kept(want, got, kept):
    assert (got[kept] == KEPT).all()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[kept] = False
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("cta,sequence", [(0, 0), (2, 0), (3, 1), (8, 2)])
def test_absorbed_attention(cta, sequence):
    """One page per range: CTAs 0-2 have the pages of sequence 0, 3-7 of 1, 8 of 2."""
    c = Latent([130, 300, 64], 16, 128, 512, seed=1)
    q, new_c = c.new(1)
    want, got = run_thrice(lambda: c.decode(q, new_c), _lib.TEST_LATENT_ATTEND, cta, c.pool)
    check_kept(want, got, (sequence,))


@pytest.mark.parametrize("d,d_c", [(128, 512), (64, 128)])
def test_absorbed_attention_of_several_pages_and_row_groups(d, d_c):
    """256 rows (token, head) in eight groups, ranges of several pages: group 1 of the first range has the
    second half of the heads of token 0."""
    c = Latent([5000], 64, d, d_c, seed=2)
    q, new_c = c.new(4)
    want, got = run_thrice(lambda: c.decode(q, new_c), _lib.TEST_LATENT_ATTEND, 1, c.pool)
    check_kept(want, got, (0, 0, slice(32, 64)))


@pytest.mark.parametrize("d,d_c", [(128, 512), (64, 256)])
@pytest.mark.parametrize("T", [600, 1500])
def test_prompt_attention(d, d_c, T):
    """CTA 1 has the last query block of head 1 of sequence 0."""
    c = Latent([T, T], 2, d, d_c, seed=3)
    q, new_c = c.randn(2, T, 2, d + 64), c.randn(2, T, d_c + 64)
    want, got = run_thrice(lambda: prefill(c, q, new_c), _lib.TEST_LATENT_PROMPT, 1, c.pool)
    check_kept(want, got, (0, slice((T - 1) // 256 * 256, T), 1))


def check_expansion(want, got, b, h, tile):
    block = got[b, tile // 2 * 256:tile * 128, h]
    assert ((block == KEPT) | (block == want[b, tile // 2 * 256:tile * 128, h])).all()
    block.copy_(torch.full_like(block, KEPT))
    check_kept(want, got, (b, slice(tile // 2 * 256, got.shape[1]), h))


@pytest.mark.parametrize("d,d_c", [(128, 512), (64, 256)])
@pytest.mark.parametrize("cta", [0, 2, 4, 7])
def test_expansion(d, d_c, cta):
    """One head: CTA t expands tile t % 5 of sequence t // 5. The queries from its positions on keep their
    outputs, those before it in the same block of 256 may, and all others are as ever."""
    c = Latent([600, 600], 1, d, d_c, seed=4)
    q, new_c = c.randn(2, 600, 1, d + 64), c.randn(2, 600, d_c + 64)
    want, got = run_thrice(lambda: prefill(c, q, new_c), _lib.TEST_LATENT_KV, cta, c.pool)
    check_expansion(want, got, cta // 5, 0, cta % 5)


def test_expansion_of_one_group_of_heads():
    """A workspace for one head at a time, filled by each: the first head's group gives up on tile 1."""
    c = Latent([600], 3, 128, 512, seed=5)
    q, new_c = c.randn(1, 600, 3, 192), c.randn(1, 600, 576)
    want, got = run_thrice(lambda: prefill(c, q, new_c, heads_in_ws=1), _lib.TEST_LATENT_KV, 1, c.pool)
    check_expansion(want, got, 0, 0, 1)


@pytest.mark.parametrize("nq", [1, 3])
def test_scored_step(nq):
    """CTA 0 has the first keys of kv-head 0 of sequence 0: its heads' outputs and all of its weights stay."""
    Hq, Hkv, d, G = 8, 2, 128, 4
    c = Cache([300, 270], Hkv, d, seed=6)
    q, nk, nv = new_tokens(c, nq, Hq, Hkv, d)
    k0, v0, w0 = c.k.clone(), c.v.clone(), c.w.clone()

    def step():
        c.k.copy_(k0), c.v.copy_(v0), c.w.copy_(w0)
        o = scored(c, q, nk, nv, torch.full_like(q, KEPT))
        torch.cuda.synchronize()
        return o, c.w.clone(), c.k.clone(), c.v.clone()

    want = step()
    assert hmd.hmd_device_errors(clear=True) == 0
    hmd.hmd_test_arm_copy_skip(_lib.TEST_ATTN_SPLIT, 0, WAIT_NS)
    got = step()
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_TIMEOUT
    check_kept(want[0], got[0], (0, slice(None), slice(0, G)))
    assert torch.equal(got[1][0, 0], w0[0, 0])
    assert torch.equal(got[1][0, 1], want[1][0, 1]) and torch.equal(got[1][1], want[1][1])
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
    again = step()
    assert hmd.hmd_device_errors(clear=True) == 0
    assert all(torch.equal(a, b) for a, b in zip(again, want))
