"""Calls of the smaller-cache operators at the ends of what they accept: large batches and row counts, weight
rows of odd length, every combination of packing in place, sliced weights, empty batches."""
import pytest
import torch

import hybrid_mixer_decoding_b200 as hmd
from test_gpu_evict import Cache, check_scored, new_tokens, scored, want_kept
from test_gpu_latent import BF, DR, Latent, check_decode, check_prefill, prefill

pytestmark = pytest.mark.gpu


def test_absorbed_batch_beyond_the_schedules_shared_memory():
    """5000 sequences, most of them unused rows: their page counts do not fit shared memory."""
    g = torch.Generator().manual_seed(1)
    lens = [0 if n < 0.7 else int(n * 300) for n in torch.rand(5000, generator=g).tolist()]
    c = Latent(lens, 3, 64, 128, seed=1)
    q, new_c = c.new(1)
    o = c.decode(q, new_c)
    assert hmd.hmd_device_errors(clear=True) == 0
    live = torch.tensor([n > 0 for n in lens], device="cuda")
    assert (o[~live] == 0).all()
    some = [b for b, n in enumerate(lens) if n][::40]  # the definition of all of them takes a while
    for b in some:
        one = Latent.__new__(Latent)
        one.__dict__.update(c.__dict__, table=c.table[b:b + 1], lens_list=[lens[b]])
        check_decode(one, q[b:b + 1], new_c[b:b + 1], o[b:b + 1])


def test_absorbed_more_row_groups_than_sms():
    """40 tokens of 128 heads are 160 groups of 32 rows."""
    c = Latent([41, 100], 128, 64, 128, seed=2)
    q, new_c = c.new(40)
    check_decode(c, q, new_c, c.decode(q, new_c))
    assert hmd.hmd_device_errors(clear=True) == 0


def test_expanded_batch_of_very_short_prompts():
    c = Latent([2] * 700, 3, 64, 128, seed=3)
    q, new_c = c.randn(700, 2, 3, 128), c.randn(700, 2, 192)
    prompt = [b % 3 for b in range(700)]
    o = prefill(c, q, new_c, prompt=prompt)
    some = [b for b in range(700) if b % 35 < 3]
    for b in some:
        one = Latent.__new__(Latent)
        one.__dict__.update(c.__dict__, table=c.table[b:b + 1], lens_list=[2])
        check_prefill(one, q[b:b + 1], new_c[b:b + 1], o[b:b + 1], [0], prompt[b:b + 1])
    assert hmd.hmd_device_errors(clear=True) == 0


@pytest.mark.parametrize("d,d_c", [(128, 384), (64, 256)])
def test_expanded_weights_as_slices_of_one_projection(d, d_c):
    c = Latent([260], 5, d, d_c, seed=4, joint=True)
    q, new_c = c.randn(1, 260, 5, d + DR), c.randn(1, 260, d_c + DR)
    o = prefill(c, q, new_c)
    check_prefill(c, q, new_c, o, [0], [260])
    assert torch.equal(prefill(c, q, new_c, heads_in_ws=2), o)
    assert hmd.hmd_device_errors(clear=True) == 0


@pytest.mark.parametrize("w_len", [1301, 1302, 1303])
def test_scored_weight_rows_of_odd_length(w_len):
    c = Cache([1300, 65, 700], 3, 64, seed=5, n_slots=4, slots=[2, 0, 3])
    c.w = torch.rand(4, 3, w_len, generator=c.g, device="cuda")
    q, nk, nv = new_tokens(c, 2, 6, 3, 64)
    w0 = c.w.clone()
    check_scored(c, q, nk, nv, scored(c, q, nk, nv), w0)
    assert torch.equal(c.w[1], w0[1])  # nobody's row
    assert hmd.hmd_device_errors(clear=True) == 0


@pytest.mark.parametrize("rows_in_place", [False, True])
@pytest.mark.parametrize("weights_in_place", [False, True])
@pytest.mark.parametrize("lens_in_place", [False, True])
def test_evict_each_part_in_place_or_not(rows_in_place, weights_in_place, lens_in_place):
    lens, budget, recent = [300, 64, 7, 0, 513], 130, 20
    c = Cache(lens, 2, 64, seed=6, extra=5 * 3)
    c.w = c.w[:, :, :575].contiguous()  # rows of odd length
    k0, v0, w0 = c.k.clone(), c.v.clone(), c.w.clone()
    dst = c.table if rows_in_place else c.rest.view(5, 3).contiguous()
    w_out = c.w if weights_in_place else torch.full((5, 2, 131), -7.0, device="cuda")
    new_lens = c.lens if lens_in_place else torch.full_like(c.lens, -9)
    kept = torch.empty(5, 2, budget, dtype=torch.int32, device="cuda")
    hmd.kv_cache_evict(budget, recent, c.k, c.v, c.table, c.lens, c.max_len, c.w, dst, w_out, kept, new_lens)
    assert hmd.hmd_device_errors(clear=True) == 0
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    assert c.lens.tolist() == (new_lens.tolist() if lens_in_place else lens)
    for b, L in enumerate(lens):
        n = min(L, budget)
        for g in range(2):
            at = want_kept(w0[b, g].cpu().numpy(), L, budget, recent)
            assert kept[b, g].tolist() == at.tolist() + [-1] * (budget - n)
            idx = torch.from_numpy(at).cuda()
            assert torch.equal(w_out[b, g, :n], w0[b, g, idx])
            assert torch.equal(c.rows(b, c.k, n, dst)[g], c.rows(b, k0, L)[g, idx])
            assert torch.equal(c.rows(b, c.v, n, dst)[g], c.rows(b, v0, L)[g, idx])
    if not rows_in_place:  # the source pages are as they were
        src = c.table.long().flatten()
        assert torch.equal(c.k[src], k0[src]) and torch.equal(c.v[src], v0[src])
    if not weights_in_place:
        assert torch.equal(c.w, w0)


def test_empty_batches():
    z = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    i = lambda *s: z(*s, dt=torch.int32)  # noqa: E731
    ws, w = z(64, dt=torch.uint8), z(4, 64, 128)
    hmd.attn_latent_decode(z(0, 1, 4, 128), z(0, 1, 192), w, w, z(2, 64, 192), i(0, 2), i(0), 128, z(0, 1, 4, 64), ws)
    hmd.attn_latent_prefill(z(0, 5, 4, 128), z(0, 5, 192), w, w, z(2, 64, 192), i(0, 2), z(0, 5, 4, 64), ws)
    hmd.attn_latent_prefill(z(1, 0, 4, 128), z(1, 0, 192), w, w, z(2, 64, 192), i(1, 2), z(1, 0, 4, 64), ws)
    pool, weights = z(2, 2, 64, 64), z(1, 2, 128, dt=torch.float32)
    hmd.attn_verify_scored(z(0, 1, 4, 64), z(0, 1, 2, 64), z(0, 1, 2, 64), pool, pool, weights, i(0, 2), i(0), 128,
                           z(0, 1, 4, 64), ws)
    hmd.kv_cache_evict(8, 2, pool, pool, i(0, 2), i(0), 128, weights, i(0, 1), weights, i(0, 2, 8), i(0))
    torch.cuda.synchronize()
    assert hmd.hmd_device_errors(clear=True) == 0
