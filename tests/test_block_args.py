"""Refusals of the tree and windowed calls, found on the host before any launch (CPU only).

The C entry points get addresses that are never dereferenced: every call here returns an argument
error, or KVARN_OK for an empty batch.
"""

import ctypes

import pytest
import torch

A, ODD = 1 << 20, (1 << 20) + 8  # 16-byte aligned, and not


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def _desc(kv, d0=128, hkv=2, preset="kvarn_k4v2_g128", **kw):
    d = kv.desc_from_preset(d0, hkv, preset=preset)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _tree(kv, desc=None, batch=2, hq=8, nodes=5, q=A, k=A, v=A, mask=A, lens=A, pool=A, pages=4, table=A, width=3,
          clens=A, pk=A, pv=A, scale=0.1, out=A, ws=A, nbytes=1 << 40, status=A):
    desc = desc or _desc(kv)
    return kv._lib.kvarn_tree_attention(ctypes.byref(desc), batch, hq, nodes, q, k, v, mask, lens, pool, pages, table,
                                        width, clens, pk, pv, scale, out, ws, nbytes, status, None)


def _prefill(kv, desc=None, batch=2, hq=8, chunk=5, q=A, k=A, v=A, lens=A, pool=A, pages=4, table=A, width=3, clens=A,
             pk=A, pv=A, sink=4, window=100, scale=0.1, out=A, ws=A, nbytes=1 << 40, status=A):
    desc = desc or _desc(kv)
    return kv._lib.kvarn_window_prefill_attention(ctypes.byref(desc), batch, hq, chunk, q, k, v, lens, pool, pages,
                                                  table, width, clens, pk, pv, sink, window, scale, out, ws, nbytes,
                                                  status, None)


def _decode(kv, desc=None, batch=2, hq=8, q=A, pool=A, pages=4, table=A, width=3, lens=A, pk=A, pv=A, sink=4,
            window=100, scale=0.1, out=A, ws=A, nbytes=1 << 40, status=A):
    desc = desc or _desc(kv)
    return kv._lib.kvarn_window_decode_attention(ctypes.byref(desc), batch, hq, q, pool, pages, table, width, lens, pk,
                                                 pv, sink, window, scale, out, ws, nbytes, status, None)


COMMON = [dict(batch=-1), dict(hq=0), dict(width=0), dict(q=None), dict(pool=None), dict(table=None), dict(out=None),
          dict(ws=None), dict(pool=ODD), dict(ws=ODD), dict(pk=ODD), dict(pv=ODD), dict(pk=None), dict(pv=None),
          dict(pages=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))]


@pytest.mark.parametrize("bad", COMMON + [dict(nodes=0), dict(k=None), dict(v=None), dict(k=ODD), dict(v=ODD),
                                          dict(clens=None)], ids=str)
def test_tree_invalid(kv, bad):
    assert _tree(kv, **bad) == kv.KVARN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", COMMON + [dict(chunk=0), dict(k=None), dict(v=None), dict(k=ODD), dict(v=ODD),
                                          dict(clens=None), dict(sink=-1), dict(window=0), dict(window=-5)], ids=str)
def test_window_prefill_invalid(kv, bad):
    assert _prefill(kv, **bad) == kv.KVARN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", COMMON + [dict(lens=None), dict(sink=-1), dict(window=0)], ids=str)
def test_window_decode_invalid(kv, bad):
    assert _decode(kv, **bad) == kv.KVARN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(hq=6), dict(hq=32), dict(hq=3), dict(width=(1 << 23) + 1)], ids=str)
def test_unsupported(kv, bad):
    assert _tree(kv, **bad) == kv.KVARN_ERR_UNSUPPORTED
    assert _prefill(kv, **bad) == kv.KVARN_ERR_UNSUPPORTED
    assert _decode(kv, **bad) == kv.KVARN_ERR_UNSUPPORTED


def test_unsupported_sizes(kv):
    assert _tree(kv, batch=65536) == kv.KVARN_ERR_UNSUPPORTED
    assert _tree(kv, nodes=(1 << 20) + 1) == kv.KVARN_ERR_UNSUPPORTED        # 2^22 rows of a kv head
    assert _tree(kv, batch=65535, nodes=1 << 20) == kv.KVARN_ERR_UNSUPPORTED  # output rows beyond int32
    d = _desc(kv, head_dim_padded=64)
    assert _tree(kv, desc=d) == kv.KVARN_ERR_UNSUPPORTED
    assert _decode(kv, desc=_desc(kv, d0=256), hq=16) == kv.KVARN_ERR_UNSUPPORTED  # as the whole-cache decode
    assert _tree(kv, desc=_desc(kv, page_record_bytes=16)) == kv.KVARN_ERR_INVALID_ARG


def test_null_descriptor(kv):
    f = kv._lib.kvarn_tree_attention
    assert f(None, 1, 8, 1, A, A, A, A, A, A, 1, A, 1, A, A, A, 0.1, A, A, 1 << 30, A, None) == kv.KVARN_ERR_INVALID_ARG
    assert kv._lib.kvarn_tree_workspace_bytes(None, 1, 8, 1, 1) == 0


def test_empty_batch_is_ok(kv):
    none = dict(batch=0, q=None, pool=None, table=None, out=None, ws=None, nbytes=0)
    assert _tree(kv, k=None, v=None, clens=None, **none) == kv.KVARN_OK
    assert _prefill(kv, k=None, v=None, clens=None, **none) == kv.KVARN_OK
    assert _decode(kv, lens=None, **none) == kv.KVARN_OK


def test_workspace_too_small(kv):
    d = _desc(kv)
    need = kv.tree_workspace_bytes(d, 2, 8, 5, 3)
    assert need > 0 and _tree(kv, nbytes=need - 1) == kv.KVARN_ERR_WORKSPACE_TOO_SMALL
    need = kv.window_prefill_workspace_bytes(d, 2, 8, 5, 3, 4, 100)
    assert need > 0 and _prefill(kv, nbytes=need - 1) == kv.KVARN_ERR_WORKSPACE_TOO_SMALL
    need = kv.window_decode_workspace_bytes(d, 2, 8, 3, 4, 100)
    assert need > 0 and _decode(kv, nbytes=need - 1) == kv.KVARN_ERR_WORKSPACE_TOO_SMALL


def test_workspace_sizes(kv):
    d = _desc(kv)
    # one slot a CTA and row tile, the raw partials, a pair of int32 a row tile
    for batch, nodes, rows, tiles in ((1, 1, 16, 1), (3, 5, 32, 1), (2, 16, 64, 1), (2, 17, 64, 2)):
        slot, n = rows * 132 * 4, batch * 2 * tiles
        assert kv.tree_workspace_bytes(d, batch, 8, nodes, 7) == (152 + 2 * n) * slot + (8 * n + 15) // 16 * 16
    # a windowed decode's does not grow with the table once it is wider than the window
    a = kv.window_decode_workspace_bytes(d, 4, 8, 200, 4, 4096)
    assert a == kv.window_decode_workspace_bytes(d, 4, 8, 20000, 4, 4096) > 0
    for bad in (dict(sink_tokens=-1, window=5), dict(sink_tokens=0, window=0)):
        assert kv.window_decode_workspace_bytes(d, 4, 8, 20, **bad) == 0
        assert kv.window_prefill_workspace_bytes(d, 4, 8, 3, 20, **bad) == 0
    # token counts past the C int are taken as "all of it"
    assert kv.window_decode_workspace_bytes(d, 1, 8, 64, 1 << 40, 1 << 40) == \
        kv.window_decode_workspace_bytes(d, 1, 8, 64, 0x7FFFFFFF, 0x7FFFFFFF)
    with pytest.raises(ValueError):
        kv.alloc_tree_workspace(d, 1, 6, 4, 8, device="cpu")


def test_host_tensors_are_refused(kv):
    d = _desc(kv)
    h = torch.zeros
    q = h(1, 2, 8, 128, dtype=torch.float16)
    k = h(1, 2, 2, 128, dtype=torch.float16)
    pool = h(2, 2, d.page_record_bytes, dtype=torch.uint8)
    table, lens = h(1, 1, dtype=torch.int32), h(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kv.tree_attention(d, q, k, k, None, pool, table, lens, q, h(1 << 20))
    with pytest.raises(ValueError, match="CUDA"):
        kv.window_prefill_attention(d, q, k, k, pool, table, lens, q, h(1 << 20), 1, 2)
    with pytest.raises(ValueError, match="CUDA"):
        kv.window_decode_attention(d, q[:, 0], pool, table, lens, q[:, 0], h(1 << 20), 1, 2)
