"""attn_latent_decode on the GPU against the expanded definition in 64 bits.

Tolerance: o is rounded once to bf16 (2^-8 of the value) and its softmax weights are rounded to bf16
(2^-8 of sum_j p_j |v_j|, with |v_j| <= |W_uv| |c_j|). The query on the latent and the latent
output are bf16 pairs (2^-17 relative), which with fp32 sums moves a score by at most
2^-15 * sum|terms|: 2^-14 * that more on sum_j p_j |v_j|.
"""
import pytest
import torch

import hybrid_mixer_decoding_b200 as hmd

pytestmark = pytest.mark.gpu
PT, DR = 64, 64
BF = torch.bfloat16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Latent:
    """A batch's paged latent cache in random order, the rows behind each sequence NaN."""

    def __init__(self, lens, H, d, d_c, seed, max_len=None, w_scale=1.0, joint=False):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens_list, self.H, self.d, self.d_c = list(lens), H, d, d_c
        B, self.max_len = len(lens), max_len or max(1, max(lens))
        per = -(-self.max_len // PT)
        self.table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
        self.pool = self.randn(B * per, PT, d_c + DR)
        for b, L in enumerate(lens):
            t = self.table[b].long()
            self.pool[t[-(-L // PT):]] = float("nan")
            if L % PT:
                self.pool[t[L // PT], L % PT:] = float("nan")
        if joint:  # both up-projections as slices of one weight
            w = self.randn(H, 2 * d, d_c, scale=w_scale * d_c ** -0.5)
            self.w_uk, self.w_uv = w[:, :d], w[:, d:]
        else:
            self.w_uk = self.randn(H, d, d_c, scale=w_scale * d_c ** -0.5)
            self.w_uv = self.randn(H, d, d_c, scale=d_c ** -0.5)
        self.lens = i32(self.lens_list)

    def randn(self, *s, scale=1.0):
        return (torch.randn(*s, generator=self.g, device="cuda") * scale).to(BF)

    def rows(self, b, n):
        return self.pool[self.table[b].long()].reshape(-1, self.d_c + DR)[:n]

    def workspace(self, nq):
        return torch.empty(hmd.attn_latent_decode_workspace_size(
            nq, len(self.lens_list), self.H, self.d, self.d_c, DR, PT, self.max_len),
            dtype=torch.uint8, device="cuda")

    def decode(self, q, new_c, scale=None, ws=None, o=None):
        o = torch.full((*q.shape[:3], self.d), 9.0, device="cuda", dtype=BF) if o is None else o
        hmd.attn_latent_decode(q, new_c, self.w_uk, self.w_uv, self.pool, self.table, self.lens,
                               self.max_len, o, self.workspace(q.shape[1]) if ws is None else ws,
                               scale=scale)
        return o

    def new(self, nq):
        B = len(self.lens_list)
        return self.randn(B, nq, self.H, self.d + DR), self.randn(B, nq, self.d_c + DR)


def reference(c, b, C, q, first, scale):
    """o [n, H, d] and its tolerance for n queries from position `first` over the rows C."""
    n, C = q.shape[0], C.double()
    hidden = torch.arange(len(C), device="cuda")[None] > first + torch.arange(n, device="cuda")[:, None]
    K = torch.einsum("jc,hnc->hjn", C[:, :c.d_c], c.w_uk.double())
    V = torch.einsum("jc,hvc->hjv", C[:, :c.d_c], c.w_uv.double())
    Va = torch.einsum("jc,hvc->hjv", C[:, :c.d_c].abs(), c.w_uv.double().abs())
    qn, qr = q.double().transpose(0, 1).split([c.d, DR], -1)  # [H, n, .]
    x = (qn @ K.transpose(1, 2) + qr @ C[:, c.d_c:].T) * scale
    terms = (qn.abs() @ torch.einsum("jc,hnc->hjn", C[:, :c.d_c].abs(), c.w_uk.double().abs()).transpose(1, 2)
             + qr.abs() @ C[:, c.d_c:].abs().T).amax() * scale
    p = torch.softmax(x.masked_fill(hidden, -torch.inf), -1)
    ref = (p @ V).transpose(0, 1)
    # the weights' rounding acts on p_j c_j, 512 dims of which W_uv mixes: |W_uv| |c| bounds |v|, and
    # independent roundings average; the bound without averaging is the one used
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -14 * terms) * (p @ Va).transpose(0, 1)
    rms = (p ** 2 @ V ** 2).sqrt().transpose(0, 1)  # independent roundings of the keys' weights
    return ref, tol, rms


def check_decode(c, q, new_c, o, scale=None):
    nq = q.shape[1]
    scale = (c.d + DR) ** -0.5 if scale is None else scale
    for b, L in enumerate(c.lens_list):
        if L == 0:
            assert (o[b] == 0).all()
            continue
        C = c.rows(b, L)
        assert torch.equal(C[L - nq:], new_c[b])  # the append
        ref, tol, rms = reference(c, b, C, q[b], L - nq, scale)
        err = (o[b].double() - ref).abs()
        assert (err <= tol).all(), (b, L, (err / tol).max().item())
        # and far inside it on the whole: the output's rounding, and the weights' at random signs
        typical = (2.0 ** -8 * ref.abs() + 2.0 ** -8 * rms).square().mean().sqrt()
        assert err.square().mean().sqrt() <= typical


@pytest.mark.parametrize("H,d,d_c,nq", [(16, 128, 512, 1), (32, 128, 512, 1), (5, 64, 256, 1),
                                        (16, 64, 128, 2), (20, 128, 384, 3), (40, 64, 512, 2),
                                        (1, 128, 256, 4), (33, 64, 128, 1), (32, 128, 512, 4)])
def test_decode_ragged(H, d, d_c, nq):
    lens = [max(nq, n) for n in (1, 2, 63, 64, 65, 127, 128, 129, 300, 1000, 4, 777)]
    c = Latent(lens, H, d, d_c, seed=H + nq, max_len=1100)
    q, new_c = c.new(nq)
    before = c.pool.clone()
    o = c.decode(q, new_c)
    check_decode(c, q, new_c, o)
    for b, L in enumerate(lens):  # nothing else of the pool changed
        for i in range(nq):
            before[c.table[b, (L - nq + i) // PT], (L - nq + i) % PT] = new_c[b, i]
    assert torch.equal(before.view(torch.int16), c.pool.view(torch.int16))
    assert hmd.hmd_device_errors(clear=True) == 0


@pytest.mark.parametrize("B,L", [(1, 1), (1, 65), (1, 20000), (2, 30011), (150, 70), (300, 1)])
def test_decode_batches_and_lengths(B, L):
    lens = [max(1, L - 13 * b) for b in range(B)]
    c = Latent(lens, 8, 64, 256, seed=B)
    q, new_c = c.new(1)
    check_decode(c, q, new_c, c.decode(q, new_c))
    assert hmd.hmd_device_errors(clear=True) == 0


def test_decode_many_tokens_per_head():
    """More (head, 16 tokens) pairs than SMs: the merge takes 32 tokens a CTA, the last one fewer."""
    c = Latent([1 + 3 * (b % 50) for b in range(99)], 32, 128, 512, seed=9)
    q, new_c = c.new(1)
    check_decode(c, q, new_c, c.decode(q, new_c))
    assert hmd.hmd_device_errors(clear=True) == 0


def test_decode_unused_rows_and_a_bad_length():
    c = Latent([0, 130, 0, 0, 64, 0], 16, 128, 512, seed=1, max_len=200)
    q, new_c = c.new(2)
    check_decode(c, q, new_c, c.decode(q, new_c))
    assert hmd.hmd_device_errors(clear=True) == 0
    c.lens[1] = 201
    o = c.decode(q, new_c)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_SEQLEN
    assert (o[1] == 0).all()
    c.lens[1] = 1  # shorter than the new tokens
    o = c.decode(q, new_c)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_SEQLEN
    c.lens_list[1], c.lens[1] = 130, 130
    c.lens.zero_()
    assert (c.decode(q, new_c) == 0).all()
    assert hmd.hmd_device_errors(clear=True) == 0


def test_decode_leaves_out_a_bad_page():
    c = Latent([300], 16, 128, 512, seed=2)
    q, new_c = c.new(1)
    c.table[0, 1] = -5
    o = c.decode(q, new_c)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_PAGE
    good = torch.cat([torch.arange(64), torch.arange(128, 300)]).cuda()
    t = c.table[0].long().clone()
    t[1] = 0
    C = c.pool[t].reshape(-1, 576)[:300][good]
    ref, tol, _ = reference(c, 0, C, q[0], len(C) - 1, 192 ** -0.5)
    assert ((o[0].double() - ref).abs() <= tol).all()


def test_decode_steep_softmax_joint_weights_and_scale():
    """Large scores that grow along the sequence (the exponent base moves again and again), weights
    that are slices of one projection, an explicit scale."""
    c = Latent([900, 333], 16, 128, 512, seed=3, w_scale=4.0, joint=True)
    ramp = torch.linspace(0.02, 3.0, c.max_len, device="cuda")
    for b, L in enumerate(c.lens_list):
        pos = torch.arange(L, device="cuda")
        c.pool[c.table[b].long()[pos // PT], pos % PT] *= ramp[:L, None].to(BF)
    q, new_c = c.new(1)
    check_decode(c, q, new_c, c.decode(q, new_c, scale=0.2), scale=0.2)


def test_decode_is_deterministic_and_captured():
    c = Latent([500, 80, 1000], 32, 128, 512, seed=4, max_len=1024)
    q, new_c = c.new(1)
    ws, o = c.workspace(1), torch.empty(3, 1, 32, 128, device="cuda", dtype=BF)
    ws.fill_(0xff)  # NaN everywhere: nothing is read before it is written
    c.decode(q, new_c, ws=ws, o=o)
    ref = o.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.decode(q, new_c, ws=ws, o=o)
            c.decode(q, new_c, ws=ws, o=o)
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, ref)
    # the captured call follows lengths changed on the device
    c.lens_list = [400, 64, 7]
    c.lens.copy_(i32(c.lens_list))
    g.replay()
    torch.cuda.synchronize()
    check_decode(c, q, new_c, o)


def test_verify_equals_successive_decode_steps():
    nq = 3
    c = Latent([200, 64, 131], 16, 128, 512, seed=5)
    q, new_c = c.new(nq)
    pool = c.pool.clone()
    o = c.decode(q, new_c)
    c.pool.copy_(pool)
    for i in range(nq):
        c.lens.copy_(i32([L - nq + 1 + i for L in c.lens_list]))
        oi = c.decode(q[:, i:i + 1].contiguous(), new_c[:, i:i + 1].contiguous())
        assert (oi[:, 0].double() - o[:, i].double()).abs().max() <= 2.0 ** -6 * o.double().abs().max()


# ---- expanded form -------------------------------------------------------------------------------
# o is rounded once to bf16 (2^-8 of the value). Keys, values, queries and weights are fp16 (half a
# step, 2^-11 of each; absolute 2^-25 below 2^-14): a score moves by at most 3 * 2^-11 of its terms,
# the weights by as much and by 2^-11 themselves and the exponential's 2^-13, the values by 2^-11.
def prefill(c, q, new_c, prefix=None, prompt=None, heads_in_ws=None, scale=None, o=None, ws=None):
    B, T = q.shape[:2]
    mp = int(max(prefix)) if prefix is not None else 0
    if ws is None:
        ws = torch.empty(hmd.attn_latent_prefill_workspace_size(B, T, heads_in_ws or c.H, c.d, c.d_c, DR,
                                                                PT, mp), dtype=torch.uint8, device="cuda")
        ws.fill_(0xff)  # NaN everywhere
    o = torch.full((B, T, c.H, c.d), 9.0, device="cuda", dtype=BF) if o is None else o
    hmd.attn_latent_prefill(q, new_c, c.w_uk, c.w_uv, c.pool, c.table, o, ws,
                            prefix_lens=None if prefix is None else i32(prefix), max_prefix=mp,
                            prompt_lens=None if prompt is None else i32(prompt), scale=scale)
    return o


def check_prefill(c, q, new_c, o, prefix, prompt, scale=None):
    scale = (c.d + DR) ** -0.5 if scale is None else scale
    for b, (pre, n) in enumerate(zip(prefix, prompt)):
        assert (o[b, n:] == 9.0).all()  # behind the prompt: as it was
        if n == 0:
            continue
        C = c.rows(b, pre + n)
        assert torch.equal(C[pre:], new_c[b, :n])  # the append
        ref, _, rms = reference(c, b, C, q[b, :n], pre, scale)
        qn, qr = q[b, :n].double().transpose(0, 1).split([c.d, DR], -1)
        K = torch.einsum("jc,hnc->hjn", C.double()[:, :c.d_c], c.w_uk.double())
        V = torch.einsum("jc,hvc->hjv", C.double()[:, :c.d_c], c.w_uv.double())
        hidden = torch.arange(pre + n, device="cuda")[None] > pre + torch.arange(n, device="cuda")[:, None]
        x = (qn @ K.transpose(1, 2) + qr @ C.double()[:, c.d_c:].T) * scale
        p = torch.softmax(x.masked_fill(hidden, -torch.inf), -1)
        terms = (qn.abs() @ K.abs().transpose(1, 2) + qr.abs() @ C.double()[:, c.d_c:].abs().T).amax() * scale
        pv = (p @ V.abs()).transpose(0, 1)
        err = (o[b, :n].double() - ref).abs()
        tol = 2.0 ** -8 * ref.abs() + (2 * 3 * 2.0 ** -11 * terms + 2 * 2.0 ** -11 + 2.0 ** -13) * pv
        assert (err <= tol).all(), (b, (err / tol).max().item())
        typical = (2.0 ** -8 * ref.abs() + 2.0 ** -10 * rms).square().mean().sqrt()
        assert err.square().mean().sqrt() <= typical


@pytest.mark.parametrize("H,d,d_c,T", [(4, 128, 512, 1), (3, 128, 512, 127), (2, 64, 256, 128),
                                       (5, 64, 128, 129), (2, 128, 384, 257), (7, 64, 512, 600),
                                       (3, 128, 512, 1300)])
def test_prefill_whole_prompts(H, d, d_c, T):
    c = Latent([T, T], H, d, d_c, seed=T)
    q, new_c = c.randn(2, T, H, d + DR), c.randn(2, T, d_c + DR)
    o = prefill(c, q, new_c)
    check_prefill(c, q, new_c, o, [0, 0], [T, T])
    assert hmd.hmd_device_errors(clear=True) == 0
    # fewer heads at a time: the same bits
    for heads in {1, 2, H - 1} - {0, H}:
        assert torch.equal(prefill(c, q, new_c, heads_in_ws=heads), o)


@pytest.mark.parametrize("d,d_c", [(128, 512), (64, 256)])
def test_prefill_after_ragged_prefixes(d, d_c):
    prefix, prompt, T = [0, 1, 63, 64, 100, 700, 512, 5], [300, 1, 65, 128, 0, 299, 256, 7], 300
    c = Latent([max(1, a) for a in prefix], 4, d, d_c, seed=21, max_len=1000)
    q, new_c = c.randn(8, T, 4, d + DR), c.randn(8, T, d_c + DR)
    for b, n in enumerate(prompt):  # padding: never read
        q[b, n:], new_c[b, n:] = float("nan"), float("nan")
    before = c.pool.clone()
    o = prefill(c, q, new_c, prefix, prompt)
    check_prefill(c, q, new_c, o, prefix, prompt)
    assert hmd.hmd_device_errors(clear=True) == 0
    for b, (pre, n) in enumerate(zip(prefix, prompt)):
        pos = torch.arange(pre, pre + n, device="cuda")
        before[c.table[b].long()[pos // PT], pos % PT] = new_c[b, :n]
    assert torch.equal(before.view(torch.int16), c.pool.view(torch.int16))


def test_prefill_reports_bad_lengths_pages_and_range():
    c = Latent([100, 100], 2, 64, 128, seed=22, max_len=300)
    q, new_c = c.randn(2, 50, 2, 128), c.randn(2, 50, 192)
    o = prefill(c, q, new_c, [100, 64], [51, 50])
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_SEQLEN
    check_prefill(c, q, new_c, o, [0, 64], [0, 50])
    q[1, 3, 0, 5] = 1e6
    prefill(c, q, new_c)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVWARN_RANGE
    c.table[0, 0] = c.pool.shape[0]
    q[1, 3, 0, 5] = 1.0
    o = prefill(c, q, new_c)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_PAGE
    check_prefill(c, q[1:], new_c[1:], o[1:], [], [])


def test_prefill_steep_softmax_and_large_values():
    """Scores that grow along the sequence, values of several thousand (fp16's range is 65504)."""
    c = Latent([400], 4, 128, 512, seed=23, w_scale=3.0)
    c.w_uv *= 512
    q, new_c = c.randn(1, 400, 4, 192), c.randn(1, 400, 576)
    new_c *= torch.linspace(0.05, 2.0, 400, device="cuda")[None, :, None].to(BF)
    o = prefill(c, q, new_c, scale=0.1)
    assert hmd.hmd_device_errors(clear=True) == 0
    check_prefill(c, q, new_c, o, [0], [400], scale=0.1)


def test_prefill_in_parts_then_decode():
    """As they are used: two parts of a prompt, then decode steps and a verification pass, against
    the definition over the whole sequence."""
    H, d, d_c, lens = 16, 128, 512, [300, 171]
    c = Latent([1, 1], H, d, d_c, seed=24, max_len=400)
    C, Q = c.randn(2, 320, d_c + DR), c.randn(2, 320, H, d + DR)
    done = [0, 0]
    for part in ([200, 100], [100, 71]):
        T = max(part)
        q, new_c = torch.zeros(2, T, H, d + DR, device="cuda", dtype=BF), torch.zeros(2, T, d_c + DR, device="cuda", dtype=BF)
        for b, n in enumerate(part):
            q[b, :n], new_c[b, :n] = Q[b, done[b]:done[b] + n], C[b, done[b]:done[b] + n]
        o = prefill(c, q, new_c, done, part)
        check_prefill(c, q, new_c, o, done, part)
        done = [a + n for a, n in zip(done, part)]
    assert done == lens
    for nq in (1, 1, 3):
        done = [n + nq for n in done]
        c.lens_list = done
        c.lens.copy_(i32(done))
        q = torch.stack([Q[b, L - nq:L] for b, L in enumerate(done)])
        new_c = torch.stack([C[b, L - nq:L] for b, L in enumerate(done)])
        check_decode(c, q, new_c, c.decode(q, new_c))
    assert hmd.hmd_device_errors(clear=True) == 0


def test_prefill_captured_on_another_stream():
    c = Latent([1], 4, 64, 256, seed=25, max_len=400)
    q, new_c = c.randn(1, 333, 4, 128), c.randn(1, 333, 320)
    ref = prefill(c, q, new_c)
    ws = torch.empty(hmd.attn_latent_prefill_workspace_size(1, 333, 4, 64, 256, DR, PT),
                     dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            prefill(c, q, new_c, o=o, ws=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, ref)


def test_cache_handle_holds_the_layers_pools():
    cache = hmd.LatentCache([0, -1, 1, 0], 2, 5, 128)
    a, b = cache.layer_pool(0), cache.layer_pool(2)
    assert a.shape == (5, PT, 192) and (a == 0).all() and (b == 0).all()
    a.fill_(3.0)
    assert torch.equal(cache.layer_pool(3), a) and (b == 0).all()
    for layer in (-1, 1, 4):
        with pytest.raises(hmd.HmdError, match="HMD_ERR_ARG"):
            cache.layer_pool(layer)
    # a decode step on the handle's pool
    c = Latent([70], 4, 64, 128, seed=30, max_len=128)
    cache.layer_pool(2)[:2] = c.pool
    q, new_c = c.new(1)
    want = c.decode(q, new_c)
    c.pool = cache.layer_pool(2)
    assert torch.equal(c.decode(q, new_c), want)
    cache.free()


def test_two_streams_with_their_own_workspaces():
    cs = [Latent([700 + i, 300], 16, 128, 512, seed=40 + i) for i in range(2)]
    new = [c.new(1) for c in cs]
    ws = [c.workspace(1) for c in cs]
    outs = [torch.empty(2, 1, 16, 128, device="cuda", dtype=BF) for _ in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        for c, (q, n), w, o, s in zip(cs, new, ws, outs, streams):
            hmd.attn_latent_decode(q, n, c.w_uk, c.w_uv, c.pool, c.table, c.lens, c.max_len, o, w, stream=s)
    torch.cuda.synchronize()
    for c, (q, n), o in zip(cs, new, outs):
        check_decode(c, q, n, o)


def test_offsets_beyond_32_bits():
    """A pool whose last pages lie beyond 2^32 bytes, and beyond 2^31 elements."""
    n_pages = 2**32 // (64 * 576 * 2) + 4000
    if torch.cuda.mem_get_info()[0] < 2 * n_pages * 64 * 576 * 2:
        pytest.skip("not enough free memory")
    c = Latent([130, 70], 16, 128, 512, seed=50, max_len=192)
    pool = torch.zeros(n_pages, PT, 576, device="cuda", dtype=BF)
    at = torch.arange(n_pages - c.pool.shape[0], n_pages, device="cuda")
    pool[at] = c.pool
    c.table = at.to(torch.int32)[c.table.long()].contiguous()
    c.pool = pool
    q, new_c = c.new(1)
    check_decode(c, q, new_c, c.decode(q, new_c))
    qp, cp = c.randn(2, 40, 16, 192), c.randn(2, 40, 576)
    c.lens_list = [152, 110]
    check_prefill(c, qp, cp, prefill(c, qp, cp, [112, 70], [40, 40]), [112, 70], [40, 40])
    assert hmd.hmd_device_errors(clear=True) == 0


@pytest.mark.parametrize("H,d,d_c,T", [(12, 128, 512, 300), (5, 64, 256, 150)])
def test_inputs_written_just_before_calls_that_share_a_workspace(H, d, d_c, T):
    """Weights, queries and rows written by the kernel before each call, calls one after another on one
    workspace, eager and captured: as with a synchronisation between all of them."""
    c = Latent([T + 1] * 2, H, d, d_c, seed=60)
    ws = torch.empty(max(hmd.attn_latent_prefill_workspace_size(2, T, H, d, d_c, DR, PT, 0),
                         c.workspace(1).numel()), dtype=torch.uint8, device="cuda")
    sets = [(c.randn(H, d, d_c, scale=d_c ** -0.5), c.randn(H, d, d_c, scale=d_c ** -0.5),
             c.randn(2, T, H, d + DR), c.randn(2, T, d_c + DR), *c.new(1)) for _ in range(3)]
    q, rows, q1, row1 = (torch.empty_like(x) for x in sets[0][2:])
    n = 9
    outs = [(torch.empty(2, T, H, d, device="cuda", dtype=BF), torch.empty(2, 1, H, d, device="cuda", dtype=BF))
            for _ in range(n)]

    def chain(pause):
        for i in range(n):
            for dst, src in zip((c.w_uk, c.w_uv, q, rows, q1, row1), sets[i % 3]):
                dst.copy_(src)
            pause()
            prefill(c, q, rows, o=outs[i][0], ws=ws)
            pause()
            c.decode(q1, row1, ws=ws, o=outs[i][1])
            pause()

    chain(torch.cuda.synchronize)
    want = [[o.clone() for o in pair] for pair in outs]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        chain(lambda: None)
    for run in (lambda: chain(lambda: None), graph.replay, graph.replay):
        for pair in outs:
            for o in pair:
                o.fill_(7.0)
        run()
        torch.cuda.synchronize()
        for pair, ref in zip(outs, want):
            assert all(torch.equal(o, r) for o, r in zip(pair, ref))


@pytest.mark.parametrize("d,d_c", [(128, 512), (64, 128)])
def test_prefill_outputs_on_16_byte_boundaries(d, d_c):
    """o, q and the rows at addresses that are multiples of 16 bytes, not of 32."""
    c = Latent([150, 70], 3, d, d_c, seed=70)

    def shifted(x):
        y = torch.empty(x.numel() + 8, device="cuda", dtype=BF)[8:].view(x.shape)
        assert y.data_ptr() % 32 == 16
        return y.copy_(x)

    q, new_c = shifted(c.randn(2, 150, 3, d + DR)), shifted(c.randn(2, 150, d_c + DR))
    o = shifted(torch.full((2, 150, 3, d), 9.0, device="cuda", dtype=BF))
    check_prefill(c, q, new_c, prefill(c, q, new_c, prompt=[150, 70], o=o), [0, 0], [150, 70])
    assert hmd.hmd_device_errors(clear=True) == 0
