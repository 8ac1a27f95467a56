"""attn_verify_scored and kv_cache_evict on the GPU, against 64-bit definitions.

Tolerances, derived: o is rounded once to bf16 (half a step, 2^-8 of the value) and its softmax
weights are rounded to bf16 before the product with V (2^-8 of sum_j p_j |v_j|); the fp32
arithmetic around it stays below 2^-12 of that sum. A weight is exp of a d-term fp32 dot product:
its relative error is at most twice the error of the score, d * 2^-23 * sum|q_i k_i| / sqrt(d),
plus 2^-16 for the exponential, the sum over the keys and the merge; fp32 sums with the old weight
add 2^-22 of the total. What is moved or chosen has to be equal.
"""
import numpy as np
import pytest
import torch

import hybrid_mixer_decoding_b200 as hmd

pytestmark = pytest.mark.gpu
PT = 64
BF = torch.bfloat16


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Cache:
    """A batch's paged cache in random order, `extra` unused pages, weights with ties."""

    def __init__(self, lens, Hkv, d, seed, extra=0, max_len=None, n_slots=None, slots=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        B, self.max_len = len(lens), max_len or max(1, max(lens))
        per = -(-self.max_len // PT)
        order = torch.randperm(B * per + extra, generator=g, device="cuda").to(torch.int32)
        self.table, self.rest = order[:B * per].view(B, per).contiguous(), order[B * per:]
        n = B * per + extra
        self.k = torch.randn(n, Hkv, PT, d, generator=g, device="cuda").to(BF)
        self.v = torch.randn(n, Hkv, PT, d, generator=g, device="cuda").to(BF)
        self.w = torch.rand(n_slots or B, Hkv, per * PT, generator=g, device="cuda") ** 3
        self.w[torch.rand(self.w.shape, generator=g, device="cuda") < 0.2] = 0.125  # ties
        self.lens, self.slots, self.g = i32(lens), (None if slots is None else i32(slots)), g

    def rows(self, b, pool, L, table=None):
        t = (self.table if table is None else table)[b].long()
        x = pool[t]
        return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :L]


def scored(c, q, nk, nv, o=None):
    B, nq, Hq, d = q.shape
    ws = torch.empty(hmd.attn_verify_scored_workspace_size(nq, B, Hq, c.k.shape[1], d, PT, c.max_len),
                     dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q) if o is None else o
    hmd.attn_verify_scored(q, nk, nv, c.k, c.v, c.w, c.table, c.lens, c.max_len, o, ws, slots=c.slots)
    return o


def new_tokens(c, nq, Hq, Hkv, d, scale=1.0):
    B = len(c.lens)
    r = lambda *s: torch.randn(*s, generator=c.g, device="cuda").to(BF)  # noqa: E731
    return (r(B, nq, Hq, d).float() * scale).to(BF), r(B, nq, Hkv, d), r(B, nq, Hkv, d)


def check_scored(c, q, nk, nv, o, w0):
    B, nq, Hq, d = q.shape
    Hkv = c.k.shape[1]
    G = Hq // Hkv
    for b, L in enumerate(c.lens.tolist()):
        slot = b if c.slots is None else int(c.slots[b])
        K, V = c.rows(b, c.k, L).double(), c.rows(b, c.v, L).double()
        assert torch.equal(K[:, L - nq:], nk[b].transpose(0, 1).double())  # the append
        assert torch.equal(V[:, L - nq:], nv[b].transpose(0, 1).double())
        want = w0[slot].double().clone()
        want[:, L - nq:L] = 0
        bound = torch.zeros(Hkv, device="cuda", dtype=torch.float64)
        for g in range(Hkv):
            Q = q[b, :, g * G:(g + 1) * G].double()  # [nq, G, d]
            x = Q @ K[g].T / d ** 0.5
            hidden = torch.arange(L, device="cuda") > (L - nq + torch.arange(nq, device="cuda"))[:, None]
            p = torch.softmax(x.masked_fill(hidden[:, None], -torch.inf), -1)
            ref = p @ V[g]
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * (p @ V[g].abs())
            assert ((o[b, :, g * G:(g + 1) * G].double() - ref).abs() <= tol).all()
            want[g, :L] += p.sum((0, 1))
            bound[g] = 2 * d * 2.0 ** -23 * (Q.abs() @ K[g].abs().T / d ** 0.5).max() + 2.0 ** -16
        got = c.w[slot].double()
        add = want - w0[slot].double()
        add[:, L - nq:L] = want[:, L - nq:L]
        assert ((got - want).abs() <= bound[:, None] * add.abs() + 2.0 ** -22 * want.abs()).all()
        assert torch.equal(got[:, L:], w0[slot].double()[:, L:])  # behind the sequence: as it was


@pytest.mark.parametrize("d,Hq,Hkv,nq", [(128, 8, 2, 1), (64, 4, 4, 4), (128, 16, 1, 1), (64, 10, 2, 3),
                                         (128, 6, 3, 2)])
def test_scored_ragged(d, Hq, Hkv, nq):
    lens = [max(nq, n) for n in (1, 63, 64, 65, 150, 511, 512, 513, 1300)]
    c = Cache(lens, Hkv, d, seed=d + nq, max_len=1400)
    q, nk, nv = new_tokens(c, nq, Hq, Hkv, d)
    w0 = c.w.clone()
    k2, v2 = c.k.clone(), c.v.clone()
    o = scored(c, q, nk, nv)
    check_scored(c, q, nk, nv, o, w0)
    # the output and the append are attn_verify's, bit for bit
    ws = torch.empty(hmd.attn_verify_workspace_size(hmd.FA, 0, nq, len(lens), Hq, Hkv, d, PT, 1400),
                     dtype=torch.uint8, device="cuda")
    o2 = torch.empty_like(o)
    hmd.attn_verify(hmd.FA, 0, 0, q, nk, nv, k2, v2, c.table, c.lens, 1400, o2, ws)
    assert torch.equal(o, o2) and torch.equal(c.k, k2) and torch.equal(c.v, v2)
    assert hmd.hmd_device_errors(clear=True) == 0


def test_scored_many_splits_and_steep_softmax():
    c = Cache([30001], 2, 128, seed=3)
    q, nk, nv = new_tokens(c, 2, 4, 2, 128, scale=6.0)
    w0 = c.w.clone()
    check_scored(c, q, nk, nv, scored(c, q, nk, nv), w0)


def test_scored_uses_slots_and_reports_a_bad_one():
    c = Cache([70, 5, 200], 2, 64, seed=4, n_slots=6, slots=[4, 9, 0])
    q, nk, nv = new_tokens(c, 1, 4, 2, 64)
    w0 = c.w.clone()
    scored(c, q, nk, nv)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_SLOT
    changed = [(c.w[s] != w0[s]).any().item() for s in range(6)]
    assert changed == [True, False, False, False, True, False]


def test_scored_bad_page_gives_its_keys_no_weight():
    c = Cache([200], 1, 64, seed=5)
    c.table[0, 1] = 10_000
    q, nk, nv = new_tokens(c, 1, 2, 1, 64)
    w0 = c.w.clone()
    scored(c, q, nk, nv)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_PAGE
    assert torch.equal(c.w[0, 0, 64:128], w0[0, 0, 64:128])
    added = (c.w - w0)[0, 0, :199].double().sum() + c.w[0, 0, 199].double()
    assert abs(added.item() - 2.0) < 1e-4  # each head's weights still add up to one


def want_kept(w, L, budget, recent):
    """Kept positions of one (sequence, kv-head) from its weights, by sorting."""
    first = L - min(L, recent)
    m = min(L, budget) - (L - first)
    u = np.where(np.isnan(w[:first]), np.inf, w[:first])
    nan_first = np.where(np.isnan(w[:first]), 0, 1)
    order = np.lexsort((np.arange(first), nan_first, -u))
    return np.concatenate([np.sort(order[:m]), np.arange(first, L)])


def run_evict(c, budget, recent, in_place):
    B, Hkv = len(c.lens), c.k.shape[1]
    keep = -(-min(budget, c.max_len) // PT)
    dst = c.table if in_place else c.rest[:B * keep].view(B, keep).contiguous()
    w_out = c.w if in_place else torch.full((c.w.shape[0], Hkv, keep * PT), -7.0, device="cuda")
    kept = torch.full((B, Hkv, budget), -9, dtype=torch.int32, device="cuda")
    new_lens = c.lens if in_place else torch.full((B,), -9, dtype=torch.int32, device="cuda")
    hmd.kv_cache_evict(budget, recent, c.k, c.v, c.table, c.lens, c.max_len, c.w, dst, w_out, kept,
                       new_lens, slots=c.slots)
    return dst, w_out, kept, new_lens


def check_evict(c, budget, recent, in_place):
    k0, v0, w0, lens = c.k.clone(), c.v.clone(), c.w.clone(), c.lens.tolist()
    src_k = [c.rows(b, k0, L) for b, L in enumerate(lens)]
    src_v = [c.rows(b, v0, L) for b, L in enumerate(lens)]
    dst, w_out, kept, new_lens = run_evict(c, budget, recent, in_place)
    assert hmd.hmd_device_errors(clear=True) == 0
    assert new_lens.tolist() == [min(L, budget) for L in lens]
    touched_k, touched_v = k0.clone(), v0.clone()
    for b, L in enumerate(lens):
        n, slot = min(L, budget), b if c.slots is None else int(c.slots[b])
        for g in range(c.k.shape[1]):
            at = want_kept(w0[slot, g].cpu().numpy(), L, budget, recent)
            assert kept[b, g, :n].tolist() == at.tolist()
            assert (kept[b, g, n:] == -1).all()
            idx = torch.from_numpy(at).cuda()
            assert torch.equal(w_out[slot, g, :n].view(torch.int32), w0[slot, g, idx].view(torch.int32))
            tail = w0[slot, g, n:] if in_place else torch.full_like(w_out[slot, g, n:], -7.0)
            assert torch.equal(w_out[slot, g, n:].view(torch.int32), tail.view(torch.int32))
            i = torch.arange(n, device="cuda")
            page = dst[b].long()[i // PT]
            touched_k[page, g, i % PT] = src_k[b][g, idx]
            touched_v[page, g, i % PT] = src_v[b][g, idx]
    # the packed rows, and nothing else of the pools changed
    assert torch.equal(c.k, touched_k) and torch.equal(c.v, touched_v)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 64), (65, 10), (130, 0), (300, 77),
                                           (511, 511), (2000, 100)])
def test_evict_ragged(budget, recent, in_place):
    lens = [0, 1, 2, 63, 64, 65, 130, 131, 300, 513, 1111]
    c = Cache(lens, 3, 128 if budget % 2 else 64, seed=budget, extra=11 * 20)
    check_evict(c, budget, recent, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_slots_and_odd_values(in_place):
    c = Cache([900, 500], 2, 128, seed=6, extra=20, n_slots=5, slots=[3, 1])
    c.w[3, 0, 100:140] = torch.inf
    c.w[3, 0, 141] = torch.nan
    c.w[3, 1, :] = 0.0
    c.w[3, 1, 50:200] = -0.0  # equal to 0: a tie
    c.w[1, 0, :] = torch.arange(c.w.shape[2], device="cuda") * -1.0
    c.w[1, 1, :] = torch.finfo(torch.float32).tiny / 4  # subnormal
    c.w[1, 1, 77] = torch.finfo(torch.float32).tiny
    check_evict(c, 333, 30, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_longer_than_shared_memory(in_place):
    c = Cache([70001, 49153 + 64, 3000], 1, 64, seed=7, extra=3 * 800)
    check_evict(c, 40000, 64, in_place)


def test_evict_reports_bad_lengths_slots_and_pages():
    c = Cache([100, 100, 100], 1, 64, seed=8, extra=10, slots=[0, 1, 2])
    c.lens[0] = 1000
    k0 = c.k.clone()
    _, _, kept, new_lens = run_evict(c, 50, 5, False)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_SEQLEN
    assert new_lens.tolist() == [0, 50, 50] and (kept[0] == -1).all()
    c.lens[0], c.slots[1] = 100, 3
    _, _, kept, new_lens = run_evict(c, 50, 5, True)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_SLOT
    assert new_lens.tolist() == [50, 0, 50] and (kept[1] == -1).all()
    for in_place in (False, True):
        c = Cache([100], 1, 64, seed=9, extra=2)
        c.table[0, 1] = -3
        k0 = c.k.clone()
        dst, _, kept, _ = run_evict(c, 90, 40, in_place)
        assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_PAGE
        good = (kept[0, 0] < 64).nonzero()[:, 0]
        good = good[good < 64]
        page = int(dst[0, 0])
        assert torch.equal(c.k[page, 0, good], k0[int(c.table[0, 0]), 0, kept[0, 0, good].long()])


def test_decode_evict_decode():
    """As they are used: decode steps that count weights, an eviction in place, further steps on
    the packed cache; each step's output against the keys that are left."""
    B, Hq, Hkv, d, steps = 3, 8, 2, 128, 5
    c = Cache([400, 333, 64], Hkv, d, seed=10, max_len=512)
    c.w.zero_()
    for round_ in range(2):
        for _ in range(steps):
            q, nk, nv = new_tokens(c, 1, Hq, Hkv, d)
            c.lens += 1
            w0 = c.w.clone()
            check_scored(c, q, nk, nv, scored(c, q, nk, nv), w0)
        check_evict(c, 128, 16, True)
    assert c.lens.tolist() == [128, 128, 74]


def test_captured_and_replayed_on_another_stream():
    c = Cache([700, 300], 2, 64, seed=11, extra=20, max_len=704)
    q, nk, nv = new_tokens(c, 1, 4, 2, 64)
    ws = torch.empty(hmd.attn_verify_scored_workspace_size(1, 2, 4, 2, 64, PT, c.max_len),
                     dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q)
    dst = c.rest[:10].view(2, 5).contiguous()
    w_out = torch.zeros(2, 2, 320, device="cuda")
    kept = torch.empty(2, 2, 300, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(2, dtype=torch.int32, device="cuda")

    def step():
        hmd.attn_verify_scored(q, nk, nv, c.k, c.v, c.w, c.table, c.lens, c.max_len, o, ws)
        hmd.kv_cache_evict(300, 20, c.k, c.v, c.table, c.lens, c.max_len, c.w, dst, w_out, kept, new_lens)

    w0 = c.w.clone()
    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (o, c.w, w_out, kept, new_lens, c.k, c.v)]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    for t in (o, w_out, kept, new_lens):
        t.zero_()
    c.w.copy_(w0)
    g.replay()
    torch.cuda.synchronize()
    for t, r in zip((o, c.w, w_out, kept, new_lens, c.k, c.v), ref):
        assert torch.equal(t, r)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_budget_far_above_the_lengths(in_place):
    c = Cache([300, 0, 65], 2, 64, seed=12, extra=15)
    check_evict(c, 200_000, 77, in_place)
