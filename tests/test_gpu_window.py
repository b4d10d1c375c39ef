"""Windowed decode and prefill over the packed cache against 64-bit attention over the same records."""

import numpy as np
import pytest
import torch

from tests import block_cases as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def _hide(cache, b, first, rows, sink, window):
    """Table entries of the sealed pages that no query of sequence b sees point outside the pool."""
    n = cache.lens[b] // 128
    if n:
        on = B.window_mask(first, rows, 128 * n, sink, window).any(axis=0).reshape(n, 128).any(axis=1)
        cache.unseen(b, [i for i in range(n) if not on[i]])


def _decode(kv, lens, hkv, group, d0, sink, window, seed, preset="kvarn_k4v2_g128"):
    cache = B.Cache(kv, lens, hkv, d0, seed, preset)
    g = torch.Generator().manual_seed(seed + 1)
    n, hq = len(lens), hkv * group
    q = torch.randn((n, hq, d0), generator=g).half()
    for b in range(n):
        _hide(cache, b, lens[b] - 1, 1, sink, window)
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    ws = kv.alloc_window_decode_workspace(cache.desc, n, hq, cache.table.shape[1], sink, window)
    ws.fill_(float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.window_decode_attention(cache.desc, q.cuda(), cache.pool, cache.table.cuda(), cache.lens_t, out, ws, sink, window,
                               status=status, **cache.args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    worst = 0.0
    for b in range(n):
        on = B.window_mask(lens[b] - 1, 1, lens[b], sink, window)
        ref = B.expected(cache, b, q[b:b + 1].double().numpy(), None, None, on, B.scale_of(d0), group)
        worst = max(worst, B.close(out[b:b + 1].cpu().double().numpy(), ref, "window decode b=%d" % b))
    return worst


LENS = [0, 1, 77, 128, 129, 1000, 1023, 4096 + 5]


@pytest.mark.parametrize("sink,window", [(0, 1), (0, 128), (4, 100), (4, 300), (128, 256), (130, 129), (300, 1000),
                                         (1, 10 ** 9), (2 * 10 ** 9, 5)])
@pytest.mark.parametrize("group,d0", [(4, 128), (8, 128), (2, 256)])
def test_window_decode_parity(kv, sink, window, group, d0):
    err = _decode(kv, LENS, 2, group, d0, sink, window, seed=group + d0)
    print("window decode sink=%d window=%d G=%d d0=%d: %.2e" % (sink, window, group, d0, err))


@pytest.mark.parametrize("preset", ["kvarn_k4v4_g128", "kvarn_k2v2_g128", "kvarn_k8v4_g128"])
@pytest.mark.parametrize("group,d0", [(1, 64), (8, 64), (4, 96), (4, 256)])
def test_window_decode_presets(kv, preset, group, d0):
    err = _decode(kv, [400, 2000], 2, group, d0, 6, 700, seed=d0, preset=preset)
    print("window decode %s G=%d d0=%d: %.2e" % (preset, group, d0, err))


def test_window_decode_of_everything_is_decode(kv):
    # a window that covers the sequences gives the same softmax as the whole-cache call
    cache = B.Cache(kv, [300, 128, 0, 1999], 2, 128, 20)
    q = torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(21)).half().cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    table = cache.table.cuda()
    kv.window_decode_attention(cache.desc, q, cache.pool, table, cache.lens_t, a,
                               kv.alloc_window_decode_workspace(cache.desc, 4, 8, table.shape[1], 0, 5000), 0, 5000,
                               **cache.args)
    kv.decode_attention(cache.desc, q, cache.pool, table, cache.lens_t, b,
                        kv.alloc_workspace(cache.desc, 4, 8, table.shape[1]), **cache.args)
    torch.cuda.synchronize()
    B.close(a.cpu().double().numpy(), b.cpu().double().numpy(), "window over everything")


def _prefill(kv, lens, chunk, hkv, group, d0, sink, window, seed, preset="kvarn_k4v2_g128", chunk_lens=None):
    cache = B.Cache(kv, lens, hkv, d0, seed, preset)
    g = torch.Generator().manual_seed(seed + 1)
    n, hq = len(lens), hkv * group
    q = torch.randn((n, chunk, hq, d0), generator=g).half()
    k = (2 * torch.randn((n, chunk, hkv, d0), generator=g)).half()
    v = torch.randn((n, chunk, hkv, d0), generator=g).half()
    sizes = [chunk] * n if chunk_lens is None else chunk_lens
    for b in range(n):
        _hide(cache, b, lens[b], max(sizes[b], 1), sink, window)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = kv.alloc_window_prefill_workspace(cache.desc, n, hq, chunk, cache.table.shape[1], sink, window)
    ws.fill_(float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cl = None if chunk_lens is None else torch.tensor(chunk_lens, dtype=torch.int32, device="cuda")
    kv.window_prefill_attention(cache.desc, q.cuda(), k.cuda(), v.cuda(), cache.pool, cache.table.cuda(), cache.lens_t,
                                out, ws, sink, window, chunk_lens=cl, status=status, **cache.args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    worst = 0.0
    for b in range(n):
        m = sizes[b]
        on = B.window_mask(lens[b], chunk, lens[b] + chunk, sink, window)
        ref = B.expected(cache, b, q[b].double().numpy(), k[b].double().numpy(), v[b].double().numpy(), on,
                         B.scale_of(d0), group)
        if m:
            worst = max(worst, B.close(out[b, :m].cpu().double().numpy(), ref[:m], "window prefill b=%d" % b))
        assert bool((out[b, m:] == 7.0).all()), "rows past the chunk were written"
    return worst


@pytest.mark.parametrize("chunk,sink,window", [(1, 0, 1), (3, 4, 2), (17, 4, 100), (64, 0, 64), (70, 130, 200),
                                               (150, 4, 100), (150, 300, 1000), (40, 1, 10 ** 9), (5, 2 * 10 ** 9, 3)])
@pytest.mark.parametrize("group,d0", [(4, 128), (1, 64), (2, 256)])
def test_window_prefill_parity(kv, chunk, sink, window, group, d0):
    err = _prefill(kv, [0, 77, 128, 1000, 1500], chunk, 2, group, d0, sink, window, seed=chunk + d0)
    print("window prefill chunk=%d sink=%d window=%d G=%d d0=%d: %.2e" % (chunk, sink, window, group, d0, err))


@pytest.mark.parametrize("preset", ["kvarn_k4v4_g128", "kvarn_k2v2_g128", "kvarn_k8v4_g128"])
@pytest.mark.parametrize("group,d0", [(8, 64), (8, 96), (8, 256)])
def test_window_prefill_presets(kv, preset, group, d0):
    err = _prefill(kv, [900, 131], 23, 1, group, d0, 3, 400, seed=d0, preset=preset)
    print("window prefill %s G=%d d0=%d: %.2e" % (preset, group, d0, err))


def test_window_prefill_ragged(kv):
    err = _prefill(kv, [640, 0, 200, 1281], 50, 2, 4, 128, 5, 150, seed=30, chunk_lens=[50, 3, 0, 21])
    print("window prefill ragged: %.2e" % err)


def test_window_prefill_then_append_then_decode(kv):
    # a chunk of one token under the window is the windowed decode step after appending it
    cache = B.Cache(kv, [500, 127, 1300], 2, 128, 31)
    g = torch.Generator().manual_seed(32)
    q = torch.randn((3, 1, 8, 128), generator=g).half().cuda()
    k, v = (torch.randn((3, 1, 2, 128), generator=g).half().cuda() for _ in range(2))
    table = torch.cat([cache.table, torch.full((3, 1), cache.free_page, dtype=torch.int32)], 1).cuda()
    table[1, 0] = cache.free_page
    a = torch.empty_like(q)
    kv.window_prefill_attention(cache.desc, q, k, v, cache.pool, table, cache.lens_t, a,
                                kv.alloc_window_prefill_workspace(cache.desc, 3, 8, 1, table.shape[1], 4, 300), 4, 300,
                                **cache.args)
    lens = cache.lens_t.clone()
    kv.append_token(cache.desc, k[:, 0].contiguous(), v[:, 0].contiguous(), cache.args["partial_k"],
                    cache.args["partial_v"], cache.lens_t, table, cache.pool, seq_lens_out=lens)
    b = torch.empty((3, 8, 128), dtype=torch.float16, device="cuda")
    kv.window_decode_attention(cache.desc, q[:, 0].contiguous(), cache.pool, table, lens, b,
                               kv.alloc_window_decode_workspace(cache.desc, 3, 8, table.shape[1], 4, 300), 4, 300,
                               **cache.args)
    torch.cuda.synchronize()
    # sequence 1 sealed a tile in between: its raw tokens became a quantised page
    for i in (0, 2):
        B.close(a[i, 0].cpu().double().numpy(), b[i].cpu().double().numpy(), "chunk of one against decode")
    assert torch.isfinite(b).all()


def test_window_graph_replay(kv):
    cache = B.Cache(kv, [500, 1300], 2, 128, 33)
    g = torch.Generator().manual_seed(34)
    q = torch.randn((2, 8, 128), generator=g).half().cuda()
    out = torch.empty_like(q)
    table = cache.table.cuda()
    ws = kv.alloc_window_decode_workspace(cache.desc, 2, 8, table.shape[1], 4, 300)

    def call():
        kv.window_decode_attention(cache.desc, q, cache.pool, table, cache.lens_t, out, ws, 4, 300, **cache.args)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
