"""attn_latent_prefill on values, weights and scales far from one, against the definition in 64 bits.

Tolerance: o is rounded once to bf16 (2^-8 of the value). Keys, values, queries and weights are fp16
times a power of two (half a step, 2^-11 of each; three values of a tile 2^-10): a score moves by at
most 3 * 2^-11 of its terms, weights by as much, by 2^-11 themselves and by the exponential's 2^-13. The
part of a score that comes from the shared rows is exact here (small integers and powers of two).
"""
import copy

import pytest
import torch

import hybrid_mixer_decoding_b200 as hmd
from test_gpu_latent import DR, Latent, check_prefill, prefill

pytestmark = pytest.mark.gpu


class Split(Latent):
    """The first half of the latent dims makes the keys, the second half the values, so that either can
    have any size at any position; the shared part of the rows and queries is zero."""

    def __init__(self, L, H, d, d_c, seed, T=None, q_scale=0.05):
        super().__init__([L], H, d, d_c, seed)
        self.w_uk[..., d_c // 2:] = 0
        self.w_uv[..., :d_c // 2] = 0
        T = T or L
        self.q, self.c = self.randn(1, T, H, d + DR, scale=q_scale), self.randn(1, T, d_c + DR)
        self.q[..., d:], self.c[..., d_c:] = 0, 0

    def check(self, o, scale, first=0, extra=0.0):
        n, d, d_c = self.q.shape[1], self.d, self.d_c
        C = self.rows(0, first + n).double()
        K = torch.einsum("jc,hnc->hjn", C[:, :d_c], self.w_uk.double())
        V = torch.einsum("jc,hvc->hjv", C[:, :d_c], self.w_uv.double())
        qn, qr = self.q[0].double().transpose(0, 1).split([d, DR], -1)
        hidden = torch.arange(first + n, device="cuda")[None] > first + torch.arange(n, device="cuda")[:, None]
        x = (qn @ K.transpose(1, 2) + qr @ C[:, d_c:].T) * scale
        p = torch.softmax(x.masked_fill(hidden, -torch.inf), -1)
        ref, pv = (p @ V).transpose(0, 1), (p @ V.abs()).transpose(0, 1)
        terms = (qn.abs() @ K.abs().transpose(1, 2)).amax() * scale
        assert terms < 2
        tol = 2.0 ** -8 * ref.abs() + (2 * 3 * 2.0 ** -11 * terms + 2 * 2.0 ** -11 + 2.0 ** -13) * pv + extra
        err = (o[0].double() - ref).abs()
        assert (err <= tol).all(), (err / tol).max().item()
        assert hmd.hmd_device_errors(clear=True) == 0


@pytest.mark.parametrize("d,d_c", [(128, 512), (64, 256)])
@pytest.mark.parametrize("e", [0, 16, 20, 24, 40, 64])
def test_values_of_any_size(d, d_c, e):
    c = Split(300, 3, d, d_c, seed=e)
    c.w_uv *= 2.0 ** -e
    c.check(prefill(c, c.q, c.c, scale=0.125), 0.125)


@pytest.mark.parametrize("d,d_c", [(128, 512), (64, 256)])
@pytest.mark.parametrize("gap", [0, 20, 120])
def test_values_whose_size_changes_along_the_sequence(d, d_c, gap):
    """Every second 128 positions hold values 2^-30 of the others' size, and scores that are `gap` / 4
    higher: the small ones count for nothing, for as much, or for all."""
    c = Split(700, 2, d, d_c, seed=gap)
    small = torch.arange(700, device="cuda") // 128 % 2 == 1
    c.c[0, small, d_c // 2:d_c] *= 2.0 ** -30
    c.c[0, small, d_c] = gap
    c.q[..., d] = 1
    c.check(prefill(c, c.q, c.c, scale=0.25), 0.25)


def test_zero_values_beside_small_ones():
    c = Split(300, 2, 64, 128, seed=3)
    c.c[0, :128, 64:128] = 0
    c.c[0, 128:, 64:128] *= 2.0 ** -40
    o = prefill(c, c.q, c.c, scale=0.125)
    assert (o[0, :128] == 0).all()
    c.check(o, 0.125)


@pytest.mark.parametrize("d,d_c", [(128, 256), (64, 128)])
def test_many_keys_of_little_weight(d, d_c):
    """One key takes nearly all of the weight and has no value; 100,000 others, 2^-25.5 of its weight
    each, make the output. Weights are held to 2^-34 of a row's largest."""
    L, T = 100_000, 3
    c = Split(L + T, 1, d, d_c, seed=5, T=T)
    c.pool.zero_()
    t = c.table[0].long()
    pos = torch.arange(L, device="cuda")
    rows = c.randn(L, d_c + DR)
    rows[:, :d_c // 2], rows[:, d_c:] = 0, 0
    rows[0, :d_c], rows[0, d_c] = 0, 17.625   # 25.4 bits above the others
    rows[:, d_c // 2:d_c] = rows[:, d_c // 2:d_c].abs()
    c.pool[t[pos // 64], pos % 64] = rows
    c.w_uv.abs_()
    c.q[..., d], c.q[..., :d] = 1, 0
    c.c[..., :d_c // 2] = 0
    c.c[..., d_c // 2:d_c].abs_()
    V = torch.einsum("jc,vc->jv", rows[:, :d_c].double(), c.w_uv[0].double())
    o = prefill(c, c.q, c.c, prefix=[L], prompt=[T], scale=1.0)
    c.check(o, 1.0, first=L, extra=2.0 ** -34 * V.abs().sum(0))


@pytest.mark.parametrize("e", [-6, 6, 20])
def test_scales_of_any_size(e):
    """Queries 2^-e of the usual size with a scale of 2^e: the same scores."""
    c = Split(300, 2, 128, 512, seed=30 + e)
    c.q *= 2.0 ** -e
    c.check(prefill(c, c.q, c.c, scale=0.125 * 2.0 ** e), 0.125 * 2.0 ** e)


@pytest.mark.parametrize("scale", [1.0, 1.999, 2.0, 3.0, 40.0])
def test_scales_on_both_sides_of_two(scale):
    c = Split(300, 2, 64, 128, seed=40, q_scale=0.01 / scale)
    c.check(prefill(c, c.q, c.c, scale=scale), scale)


def test_values_beyond_fp16_are_clipped_and_reported():
    c = Split(200, 2, 64, 128, seed=9)
    c.w_uv *= 2.0 ** 18
    o = prefill(c, c.q, c.c, scale=0.125)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVWARN_RANGE
    assert o.isfinite().all() and o.abs().max() <= 65536
    c.w_uv *= 2.0 ** -18
    c.check(prefill(c, c.q, c.c, scale=0.125), 0.125)


def alone(c, b):
    """Sequence b of a batch as a batch of one, on the same pool."""
    one = copy.copy(c)
    one.table, one.lens_list = c.table[b:b + 1], c.lens_list[b:b + 1]
    return one


def test_a_clipped_query_counts_as_the_end_of_the_range():
    c = Latent([150, 150], 2, 64, 128, seed=51)
    q, new_c = c.randn(2, 150, 2, 128), c.randn(2, 150, 192)
    q[1, 100, 1, 5] = -1e6
    o = prefill(c, q, new_c)
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVWARN_RANGE
    # every other row is as with a query inside the range
    q[1, 100, 1, 5] = -65280
    near = prefill(c, q, new_c)
    assert hmd.hmd_device_errors(clear=True) == 0
    rest = torch.ones_like(o, dtype=torch.bool)
    rest[1, 100, 1] = False
    assert torch.equal(o[rest], near[rest])
    check_prefill(c, q, new_c, near, [0, 0], [150, 150])
    # that row's scores are thousands, in which fp16 keys leave errors of about 3, so its weights are not
    # determined: it is some mean of the values up to its position (to the output's rounding)
    V = c.rows(1, 101)[:, :128].double() @ c.w_uv[1].double().T
    row, half_step = o[1, 100, 1].double(), 2.0 ** -8 * V.abs().amax(0)
    assert (row <= V.amax(0) + half_step).all() and (row >= V.amin(0) - half_step).all()


@pytest.mark.parametrize("bad", [0, 1])
def test_a_bad_page_leaves_the_other_sequence(bad):
    c = Latent([100, 100], 3, 128, 256, seed=52, max_len=300)
    q, new_c = c.randn(2, 50, 3, 192), c.randn(2, 50, 320)
    c.table[bad, 0] = c.pool.shape[0]
    o = prefill(c, q, new_c, [64, 70], [50, 41])
    assert hmd.hmd_device_errors(clear=True) == hmd.DEVERR_PAGE
    b = 1 - bad
    check_prefill(alone(c, b), q[b:b + 1], new_c[b:b + 1], o[b:b + 1], [[64, 70][b]], [[50, 41][b]])
