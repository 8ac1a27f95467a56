"""Refusals of attn_verify_scored and kv_cache_evict: a status on the host, before any launch."""
import pytest
import torch

import hybrid_mixer_decoding_b200 as hmd

FAKE = 0x10000  # an aligned non-null address that validation never dereferences
OTHER = 0x20000
OK, ARG, SHAPE, UNSUP = 0, 1, 2, 6


def _scored(n_q=1, B=2, Hq=8, Hkv=2, d=128, pt=64, q=FAKE, pool=FAKE, n_pages=100, max_pages=10,
            max_seq=640, w=FAKE, w_len=640, n_slots=2, slots=None, ws_bytes=1 << 30, ws=FAKE):
    return hmd.lib().attn_verify_scored(n_q, B, Hq, Hkv, d, pt, q, FAKE, FAKE, pool, pool, n_pages,
                                        FAKE, max_pages, FAKE, max_seq, w, w_len, n_slots, slots,
                                        FAKE, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), ARG), (dict(w=None), ARG), (dict(pool=FAKE + 8), ARG), (dict(ws=None), ARG),
    (dict(n_q=0), SHAPE), (dict(Hq=7), SHAPE), (dict(w_len=639), SHAPE), (dict(n_slots=1), SHAPE),
    (dict(n_slots=-1, slots=FAKE), SHAPE), (dict(max_pages=9), SHAPE), (dict(ws_bytes=16), SHAPE),
    (dict(max_pages=1 << 24, max_seq=1 << 30, w_len=1 << 30), UNSUP),
    (dict(d=96), UNSUP), (dict(n_q=5), UNSUP), (dict(pt=32, max_pages=20), UNSUP), (dict(B=0), OK)])
def test_scored_refusals(bad, status):
    hmd.hmd_last_error()  # clear this thread's last status
    assert _scored(**bad) == status
    assert hmd.hmd_last_error() == status


def test_scored_workspace_holds_the_scores():
    plain = hmd.attn_verify_workspace_size(hmd.FA, 0, 2, 4, 16, 4, 128, 64, 1000)
    assert hmd.attn_verify_scored_workspace_size(2, 4, 16, 4, 128, 64, 1000) == \
        plain + 4 * 2 * 16 * 1024 * 4
    assert hmd.attn_verify_scored_workspace_size(1, 0, 16, 4, 128, 64, 1000) == 16


def _evict(budget=64, recent=8, B=2, Hkv=2, d=128, pt=64, pool=FAKE, n_pages=100, table=FAKE,
           max_pages=10, max_seq=640, w=FAKE, w_len=640, n_slots=2, slots=None, dst=OTHER,
           dst_pages=1, w_out=OTHER, w_out_len=64, kept=FAKE):
    return hmd.lib().kv_cache_evict(budget, recent, B, Hkv, d, pt, pool, pool, n_pages, table,
                                    max_pages, FAKE, max_seq, w, w_len, n_slots, slots, dst,
                                    dst_pages, w_out, w_out_len, kept, FAKE, None)


@pytest.mark.parametrize("bad,status", [
    (dict(pool=None), ARG), (dict(w_out=None), ARG), (dict(kept=None), ARG), (dict(dst=None), ARG),
    (dict(pool=FAKE + 2), ARG), (dict(budget=0), SHAPE), (dict(recent=65), SHAPE),
    (dict(recent=-1), SHAPE), (dict(max_pages=9), SHAPE), (dict(budget=65), SHAPE),
    (dict(w_len=600), SHAPE), (dict(w_out_len=63), SHAPE), (dict(n_slots=1), SHAPE),
    (dict(dst=FAKE, dst_pages=9), SHAPE), (dict(w_out=FAKE, w_out_len=64), SHAPE),
    (dict(max_pages=1 << 24, max_seq=1 << 30, w_len=1 << 30), UNSUP),
    (dict(d=256), UNSUP), (dict(pt=16, max_pages=40, dst_pages=4), UNSUP), (dict(B=0), OK)])
def test_evict_refusals(bad, status):
    hmd.hmd_last_error()  # clear this thread's last status
    assert _evict(**bad) == status
    assert hmd.hmd_last_error() == status


def test_binding_refuses_types_layouts_and_devices():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    i = lambda *s: t(*s, dt=torch.int32)  # noqa: E731
    args = dict(q=t(2, 1, 4, 64), new_k=t(2, 1, 2, 64), new_v=t(2, 1, 2, 64), k_pool=t(4, 2, 64, 64),
                v_pool=t(4, 2, 64, 64), weights=t(2, 2, 128, dt=torch.float32), page_table=i(2, 2),
                seq_lens=i(2), max_seq_len=128, o=t(2, 1, 4, 64), workspace=t(64, dt=torch.uint8))
    with pytest.raises(TypeError, match="q must be"):
        hmd.attn_verify_scored(**{**args, "q": args["q"].float()})
    with pytest.raises(ValueError, match="k_pool must be contiguous"):
        hmd.attn_verify_scored(**{**args, "k_pool": args["k_pool"].transpose(0, 1)})
    with pytest.raises(ValueError, match="current CUDA device"):
        hmd.attn_verify_scored(**args)


@pytest.mark.parametrize("budget", [1 << 30, (1 << 31) - 1])
def test_evict_refuses_budgets_its_loops_cannot_count(budget):
    assert _evict(budget=budget, dst_pages=10, w_out_len=640) == UNSUP
    assert _evict(budget=budget, recent=budget, dst=FAKE, dst_pages=10, w_out=FAKE, w_out_len=640) == UNSUP
