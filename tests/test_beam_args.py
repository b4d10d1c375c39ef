"""Refusals of the page planning, the slot-mapped store and the beam calls, found on the host before any
launch (CPU only).

The C entry points get addresses that are never dereferenced: every call here returns an argument
error, or KVARN_OK where there is nothing to do.
"""

import ctypes

import pytest
import torch

A, B, ODD = 1 << 20, 1 << 21, (1 << 20) + 8  # 16-byte aligned, another, and not


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def _plan(kv, batch=2, chunk=3, lens=A, new=A, table=A, width=4, pages=8, open_tiles=1, out=B, slots=A):
    return kv._lib.kvarn_plan_pages(batch, chunk, lens, new, table, width, pages, open_tiles, out, slots, A, None)


def _store(kv, d=128, heads=2, tokens=3, k=A, v=A, ts=256, hs=128, slots=A, pool=A, pages=4):
    return kv._lib.kvarn_fp16_store(d, heads, tokens, k, v, ts, hs, slots, pool, pages, A, None)


def _select(kv, batch=2, beams=3, vocab=100, count=6, logits=A, kind=0, stride=100, scores=A, done=A, end=5, os=A,
            op=A, ot=A, od=A, ws=A, nbytes=1 << 30):
    return kv._lib.kvarn_beam_select(batch, beams, vocab, count, logits, kind, stride, scores, done, end, os, op, ot, od,
                                     ws, nbytes, A, None)


def _reorder(kv, desc=None, batch=2, beams=3, layers=2, parents=A, lens=A, lens_out=B, table=A, table_out=B, width=4,
             k=A, v=A, ko=B, vo=B):
    desc = desc or kv.desc_from_preset(128, 2)
    return kv._lib.kvarn_beam_reorder(ctypes.byref(desc), batch, beams, layers, parents, lens, lens_out, table, table_out,
                                      width, k, v, ko, vo, A, None)


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(chunk=0), dict(width=0), dict(pages=0), dict(lens=None),
                                 dict(table=None), dict(out=None), dict(out=A)], ids=str)
def test_plan_invalid(kv, bad):
    assert _plan(kv, **bad) == kv.KVARN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(batch=16385), dict(width=(1 << 23) + 1), dict(pages=(1 << 23) + 1),
                                 dict(chunk=(1 << 30) + 1)], ids=str)
def test_plan_unsupported(kv, bad):
    assert _plan(kv, **bad) == kv.KVARN_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(heads=0), dict(tokens=-1), dict(pages=0), dict(k=None), dict(v=None),
                                 dict(slots=None), dict(pool=None), dict(k=ODD), dict(v=ODD), dict(pool=ODD),
                                 dict(ts=252), dict(hs=4), dict(ts=-8), dict(hs=-8)], ids=str)
def test_store_invalid(kv, bad):
    assert _store(kv, **bad) == kv.KVARN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(d=96), dict(d=256), dict(heads=65536), dict(tokens=1 << 31),
                                 dict(pages=1 << 31)], ids=str)
def test_store_unsupported(kv, bad):
    assert _store(kv, **bad) == kv.KVARN_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(beams=0), dict(vocab=0), dict(count=0), dict(logits=None),
                                 dict(scores=None), dict(os=None), dict(op=None), dict(ot=None), dict(ws=None),
                                 dict(ws=ODD), dict(stride=99), dict(end=-2), dict(end=100), dict(end=-1),
                                 dict(logits=A + 1), dict(logits=A + 2, kind=2)], ids=str)
def test_select_invalid(kv, bad):
    assert _select(kv, **bad) == kv.KVARN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(beams=33), dict(count=65), dict(vocab=(1 << 26) + 1, stride=1 << 27),
                                 dict(batch=(1 << 20) + 1), dict(kind=3), dict(kind=-1)], ids=str)
def test_select_unsupported(kv, bad):
    assert _select(kv, **bad) == kv.KVARN_ERR_UNSUPPORTED


def test_select_workspace(kv):
    need = kv.beam_select_workspace_bytes(2, 3, 100, 6)
    assert need >= 2 * 3 * (6 + 1) * 8
    assert _select(kv, nbytes=need - 1) == kv.KVARN_ERR_WORKSPACE_TOO_SMALL
    assert kv.beam_select_workspace_bytes(2, 33, 100, 6) == kv.beam_select_workspace_bytes(2, 3, 0, 6) == 0
    # no more candidates of a group than the merge holds: 8192
    for beams, count in ((1, 1), (1, 64), (4, 8), (32, 64)):
        assert kv.beam_select_workspace_bytes(1, beams, 1 << 26, count) <= 8192 * 8 + 8192 * 8 // count + 32
    with pytest.raises(ValueError):
        kv.alloc_beam_select_workspace(1, 33, 100, 6, device="cpu")


@pytest.mark.parametrize("bad", [dict(batch=-1), dict(beams=0), dict(layers=-1), dict(width=0), dict(parents=None),
                                 dict(lens=None), dict(lens_out=None), dict(lens_out=A), dict(table=None),
                                 dict(table_out=None), dict(k=None), dict(v=None), dict(ko=None), dict(vo=None),
                                 dict(k=ODD), dict(v=ODD), dict(ko=ODD), dict(vo=ODD)], ids=str)
def test_reorder_invalid(kv, bad):
    assert _reorder(kv, **bad) == kv.KVARN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(beams=33), dict(layers=16384), dict(width=(1 << 23) + 1),
                                 dict(batch=1 << 23)], ids=str)
def test_reorder_unsupported(kv, bad):
    assert _reorder(kv, **bad) == kv.KVARN_ERR_UNSUPPORTED


def test_reorder_descriptor(kv):
    d = kv.desc_from_preset(128, 2)
    d.head_dim_padded = 64
    assert _reorder(kv, desc=d) == kv.KVARN_ERR_UNSUPPORTED
    assert kv._lib.kvarn_beam_reorder(None, 1, 1, 0, A, A, B, A, B, 1, None, None, None, None, A, None) == \
        kv.KVARN_ERR_INVALID_ARG


def test_nothing_to_do_is_ok(kv):
    assert _plan(kv, batch=0, lens=None, table=None, out=None) == kv.KVARN_OK
    assert _store(kv, tokens=0, k=None, v=None, slots=None) == kv.KVARN_OK
    assert _select(kv, batch=0, logits=None, scores=None, ws=None) == kv.KVARN_OK
    assert _reorder(kv, batch=0, parents=None, k=None) == kv.KVARN_OK


def test_host_tensors_and_shapes_are_refused(kv):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        kv.plan_pages(i(2), i(2, 3), 5, i(2))
    k = torch.zeros(2, 1, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        kv.fp16_store(k, k, torch.zeros(2, dtype=torch.int64), torch.zeros(1, 1, 2, 128, 128, dtype=torch.float16))
    with pytest.raises(ValueError, match="matching strides"):
        kv.fp16_store(k, k.transpose(0, 1), torch.zeros(2, dtype=torch.int64), k)
    with pytest.raises(ValueError, match="CUDA"):
        kv.beam_select(f(1, 2, 9), f(1, 2), f(1, 2), i(1, 2), i(1, 2), f(99))
    with pytest.raises(ValueError, match="CUDA"):
        kv.beam_reorder(kv.desc_from_preset(64, 1), i(1, 2), i(2), i(2, 1), i(2), i(2, 1))
