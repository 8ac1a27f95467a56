"""Refusals of the latent-attention entry points: a status on the host, before any launch."""
import ctypes
import re

import pytest
import torch

import hybrid_mixer_decoding_b200 as hmd

FAKE = 0x10000  # an aligned non-null address that validation never dereferences
OK, ARG, SHAPE, UNSUP = 0, 1, 2, 6
BIG = 1 << 40


def _decode(n_q=1, B=2, H=16, d=128, d_c=512, d_r=64, pt=64, scale=0.07, q=FAKE, c=FAKE, uk=FAKE,
            uk_head=128 * 512, uv=FAKE, uv_head=128 * 512, pool=FAKE, n_pages=100, max_pages=10,
            max_seq=640, o=FAKE, ws=FAKE, ws_bytes=BIG):
    return hmd.lib().attn_latent_decode(n_q, B, H, d, d_c, d_r, pt, scale, q, c, uk, uk_head, uv,
                                        uv_head, pool, n_pages, FAKE, max_pages, FAKE, max_seq, o, ws,
                                        ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), ARG), (dict(uk=None), ARG), (dict(pool=None), ARG), (dict(ws=None), ARG),
    (dict(q=FAKE + 8), ARG), (dict(uv=FAKE + 2), ARG), (dict(o=FAKE + 2), ARG),
    (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(n_q=0), SHAPE), (dict(H=0), SHAPE), (dict(max_pages=9), SHAPE),
    (dict(uk_head=128 * 512 - 8), SHAPE), (dict(uv_head=128 * 512 + 4), SHAPE),
    (dict(ws_bytes=1000), SHAPE), (dict(d=96, uk_head=1 << 20), UNSUP), (dict(d_c=576), UNSUP),
    (dict(d_c=64), UNSUP), (dict(d_r=32), UNSUP), (dict(pt=32, max_pages=20), UNSUP),
    (dict(n_pages=1 << 26), UNSUP), (dict(B=1, max_pages=1 << 24, max_seq=1 << 30), UNSUP),
    (dict(B=0), OK)])
def test_decode_refusals(bad, status):
    hmd.hmd_last_error()  # clear this thread's last status
    assert _decode(**bad) == status
    assert hmd.hmd_last_error() == status


def _prefill(B=2, T=300, H=16, d=128, d_c=512, d_r=64, pt=64, scale=0.07, q=FAKE, uk_head=128 * 512,
             prefix=None, max_prefix=0, pool=FAKE, n_pages=100, max_pages=5, o=FAKE, ws=FAKE,
             ws_bytes=BIG):
    return hmd.lib().attn_latent_prefill(B, T, H, d, d_c, d_r, pt, scale, q, FAKE, FAKE, uk_head, FAKE,
                                         128 * 512, prefix, max_prefix, None, pool, n_pages, FAKE,
                                         max_pages, o, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), ARG), (dict(pool=None), ARG), (dict(ws=FAKE + 8), ARG), (dict(o=FAKE + 8), ARG),
    (dict(ws=FAKE + 16), ARG),
    (dict(scale=-1.0), ARG), (dict(max_prefix=-1), SHAPE), (dict(max_pages=4), SHAPE),
    (dict(prefix=FAKE, max_prefix=21), SHAPE), (dict(uk_head=0), SHAPE),
    (dict(ws_bytes=100), SHAPE), (dict(d=32), UNSUP), (dict(d_c=100), UNSUP),
    (dict(T=1 << 30, max_pages=1 << 24), UNSUP), (dict(B=0), OK), (dict(T=0), OK)])
def test_prefill_refusals(bad, status):
    hmd.hmd_last_error()  # clear this thread's last status
    assert _prefill(**bad) == status
    assert hmd.hmd_last_error() == status


def test_prefix_bound_counts_only_with_prefixes():
    least = hmd.attn_latent_prefill_workspace_size(2, 300, 1, 128, 512, 64, 64, 0)
    assert _prefill(max_prefix=10_000, ws_bytes=least - 1) == SHAPE
    assert hmd.attn_latent_prefill_workspace_size(2, 300, 1, 128, 512, 64, 64, 100) > least


def test_workspace_sizes():
    # keys and values of whole 128-position tiles and the shared part, 2 bytes each
    assert hmd.attn_latent_prefill_workspace_size(2, 300, 16, 128, 512, 64, 64, 85) == \
        2 * 512 * (64 + 2 * 128 * 16) * 2
    assert hmd.attn_latent_decode_workspace_size(1, 0, 16, 128, 512, 64, 64, 640) == 16
    assert hmd.attn_latent_decode_workspace_size(1, 4, 16, 128, 500, 64, 64, 640) == 16
    assert hmd.attn_latent_decode_workspace_size(2, 4, 16, 128, 512, 64, 64, 640) > 4 * 73728


def test_cache_handle_refusals():
    L, out = hmd.lib(), ctypes.c_void_p()
    pools = (ctypes.c_int32 * 2)(0, 1)
    assert L.latent_cache_alloc(2, None, 1, 4, 512, 64, 64, None, ctypes.byref(out)) == ARG
    assert L.latent_cache_alloc(2, pools, 1, 4, 512, 64, 64, None, ctypes.byref(out)) == ARG
    assert L.latent_cache_alloc(2, pools, 2, 0, 512, 64, 64, None, ctypes.byref(out)) == SHAPE
    assert L.latent_cache_free(None, None) == ARG
    assert L.latent_cache_layer(None, 0, ctypes.byref(out)) == ARG
    assert out.value is None


def test_binding_refuses_types_layouts_and_devices():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    i = lambda *s: t(*s, dt=torch.int32)  # noqa: E731
    args = dict(q=t(2, 1, 4, 128), new_c=t(2, 1, 192), w_uk=t(4, 64, 128), w_uv=t(4, 64, 128),
                pool=t(6, 64, 192), page_table=i(2, 2), seq_lens=i(2), max_seq_len=128,
                o=t(2, 1, 4, 64), workspace=t(64, dt=torch.uint8))
    for bad, kind, match in [
            (dict(q=args["q"].float()), TypeError, "q must be"),
            (dict(seq_lens=args["seq_lens"].long()), TypeError, "seq_lens must be"),
            (dict(new_c=t(2, 2, 192)), ValueError, "new_c must have shape"),
            (dict(q=t(2, 1, 128, 4).transpose(2, 3)), ValueError, "q must be contiguous"),
            (dict(q=t(2, 4, 128)), ValueError, "4 dimensions"),
            ({}, ValueError, "current CUDA device")]:
        with pytest.raises(kind, match=match):
            hmd.attn_latent_decode(**{**args, **bad})


def test_binding_refuses_weights():
    from hybrid_mixer_decoding_b200 import _lib
    w = torch.zeros(4, 128, 128, dtype=torch.bfloat16)
    for bad, match in [(w[:, :64].float(), "must be"), (w[:, :32], "shape"),
                       (w.transpose(1, 2)[:, :64], "contiguous"),
                       (torch.zeros(1, 64, 128, dtype=torch.bfloat16).expand(4, 64, 128), "overlap"),
                       (w[:, :64], "current CUDA device")]:
        with pytest.raises((TypeError, ValueError), match=match):
            _lib._head_stride(-1, "w_uk", bad, 4, 64, 128)


def test_warnings_can_be_told_from_errors():
    errors = (hmd.DEVERR_TIMEOUT, hmd.DEVERR_PAGE, hmd.DEVERR_SLOT, hmd.DEVERR_SEQLEN, hmd.DEVERR_GATE)
    assert not any(e & hmd.DEVWARN_ALL for e in errors)
    assert hmd.DEVWARN_RANGE & ~hmd.DEVWARN_ALL == 0
    text = open(hmd._lib.__file__.replace("hybrid_mixer_decoding_b200/_lib.py", "include/hmd.h")).read()
    for name in ("RANGE", "ALL"):
        value = re.search(rf"#define HMD_DEVWARN_{name}\s+0x([0-9a-f]+)u", text).group(1)
        assert int(value, 16) == getattr(hmd, f"DEVWARN_{name}")
