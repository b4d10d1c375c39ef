"""Tree attention over the packed cache against 64-bit attention over the same records."""

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


def _inputs(cache, nodes, hq, seed):
    g = torch.Generator().manual_seed(seed)
    n = len(cache.lens)
    q = torch.randn((n, nodes, hq, cache.d0), generator=g).half()
    k = (2 * torch.randn((n, nodes, cache.hkv, cache.d0), generator=g)).half()
    v = torch.randn((n, nodes, cache.hkv, cache.d0), generator=g).half()
    return q, k, v, g


def _run(kv, cache, q, k, v, mask, tree_lens=None, fill=float("nan"), **kw):
    n, nodes, hq, _ = q.shape
    out = torch.full(q.shape, fill, dtype=torch.float16, device="cuda")
    ws = kv.alloc_tree_workspace(cache.desc, n, hq, nodes, cache.table.shape[1])
    ws.fill_(float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = None if tree_lens is None else torch.tensor(tree_lens, dtype=torch.int32, device="cuda")
    kv.tree_attention(cache.desc, q.cuda(), k.cuda(), v.cuda(), None if mask is None else mask.cuda(), cache.pool,
                      cache.table.cuda(), cache.lens_t, out, ws, tree_lens=lens, status=status, **dict(cache.args, **kw))
    torch.cuda.synchronize()
    return out.cpu(), int(status.item())


def _check(kv, lens, nodes, hkv, group, d0, seed, preset="kvarn_k4v2_g128", tree_lens=None, sees=None, plain=False):
    cache = B.Cache(kv, lens, hkv, d0, seed, preset, plain)
    q, k, v, g = _inputs(cache, nodes, hkv * group, seed + 1)
    if sees is None:
        sees = np.stack([B.ancestors(nodes, g) for _ in lens])
    out, status = _run(kv, cache, q, k, v, B.pack_mask(sees), tree_lens, fill=7.0)
    assert status == 0
    worst = 0.0
    for b, n in enumerate(lens):
        m = nodes if tree_lens is None else tree_lens[b]
        on = np.concatenate([np.ones((nodes, n), dtype=bool), sees[b] & (np.arange(nodes) < m)], axis=1)
        ref = B.expected(cache, b, q[b].double().numpy(), k[b].double().numpy(), v[b].double().numpy(), on,
                         B.scale_of(d0), group)
        if m:
            worst = max(worst, B.close(out[b, :m].double().numpy(), ref[:m], "tree b=%d" % b))
        assert bool((out[b, m:] == 7.0).all()), "rows of absent nodes were written"
    return worst


@pytest.mark.parametrize("nodes,group,d0", [(1, 1, 128), (1, 4, 128), (5, 4, 128), (8, 8, 128), (9, 2, 128),
                                            (16, 4, 128), (33, 4, 128), (64, 8, 128), (3, 8, 64), (40, 1, 64),
                                            (7, 4, 96), (26, 4, 80), (4, 4, 256), (6, 2, 256), (21, 8, 200)])
def test_tree_parity(kv, nodes, group, d0):
    # no cache, an open tile only, whole pages only, both, and a longer sequence
    err = _check(kv, [0, 77, 128, 1000, 4096 + 5], nodes, 2, group, d0, seed=nodes + group + d0)
    print("tree nodes=%d G=%d d0=%d: max scaled error %.2e" % (nodes, group, d0, err))


@pytest.mark.parametrize("nodes,group,d0", [(33, 1, 128), (10, 4, 128), (12, 4, 80), (17, 2, 64), (11, 4, 64), (47, 1, 64)])
def test_tree_tiles_of_48_rows(kv, nodes, group, d0):
    # 33 to 48 rows: their last row group full, ragged and a single row
    err = _check(kv, [0, 77, 128, 1000, 4096 + 5], nodes, 2, group, d0, seed=nodes + group + d0)
    print("tree nodes=%d G=%d d0=%d: max scaled error %.2e" % (nodes, group, d0, err))


@pytest.mark.parametrize("preset", ["kvarn_k4v4_g128", "kvarn_k2v2_g128", "kvarn_k8v4_g128"])
@pytest.mark.parametrize("d0", [64, 128, 256])
def test_tree_presets(kv, preset, d0):
    err = _check(kv, [300, 1500], 11, 2, 4, d0, seed=d0 + len(preset), preset=preset)
    print("tree %s d0=%d: max scaled error %.2e" % (preset, d0, err))


def test_tree_one_sequence_over_many_ctas(kv):
    # one (sequence, kv head): its pages are cut into ranges of a few pages, merged per row
    err = _check(kv, [128 * 150 + 1], 6, 1, 4, 128, seed=3)
    print("tree 150 pages: max scaled error %.2e" % err)


def test_tree_ragged_batch(kv):
    # many short sequences (ranges of several row tiles, some of them empty), ragged trees
    lens = [(37 * i * i) % 1400 for i in range(40)]
    nodes = [(7 * i) % 20 for i in range(40)]
    err = _check(kv, lens, 19, 3, 2, 64, seed=4, tree_lens=nodes)
    print("tree ragged: max scaled error %.2e" % err)


def test_tree_masks(kv):
    # rows that see no node, rows that see later nodes, every node; with and without a cache
    nodes = 35
    sees = np.zeros((3, nodes, nodes), dtype=bool)
    sees[:, 1, 34] = True
    sees[:, 2] = True
    sees[:, 3:, 3] = True
    err = _check(kv, [0, 130, 5], nodes, 1, 4, 128, seed=5, sees=sees, tree_lens=[35, 33, 34])
    print("tree masks: max scaled error %.2e" % err)


def test_tree_without_mask_is_a_chain(kv):
    cache = B.Cache(kv, [200, 1290], 2, 128, 6)
    q, k, v, _ = _inputs(cache, 37, 8, 7)
    chain = np.tril(np.ones((2, 37, 37), dtype=bool))
    a, _ = _run(kv, cache, q, k, v, B.pack_mask(chain))
    b, _ = _run(kv, cache, q, k, v, None)
    assert torch.equal(a, b)


def test_tree_of_one_node_matches_decode(kv):
    # a tree of one node over n tokens is the decode step after appending that node
    cache = B.Cache(kv, [300, 128, 5], 2, 128, 8)
    q, k, v, _ = _inputs(cache, 1, 8, 9)
    got, status = _run(kv, cache, q, k, v, torch.ones((3, 1, 1), dtype=torch.int32))
    assert status == 0
    lens, pk, pv = cache.lens_t.clone(), cache.args["partial_k"].clone(), cache.args["partial_v"].clone()
    table = torch.cat([cache.table, torch.zeros((3, 1), dtype=torch.int32)], 1).cuda()
    kv.append_token(cache.desc, k[:, 0].contiguous().cuda(), v[:, 0].contiguous().cuda(), pk, pv, cache.lens_t, table,
                    cache.pool, seq_lens_out=lens)
    out = torch.empty((3, 8, 128), dtype=torch.float16, device="cuda")
    kv.decode_attention(cache.desc, q[:, 0].contiguous().cuda(), cache.pool, table, lens, out,
                        kv.alloc_workspace(cache.desc, 3, 8, table.shape[1]), partial_k=pk, partial_v=pv)
    B.close(got[:, 0].double().numpy(), out.cpu().double().numpy(), "one node against decode")


def test_tree_large_logits(kv):
    # keys that grow along the sequence: the rows' references move on page after page
    cache = B.Cache(kv, [128 * 9], 1, 128, 10, plain=True)
    cache.kv.quantize_tiles(cache.desc, *(t.cuda() for t in _growing(cache)), cache.table[0, :9].cuda(), cache.pool)
    recs = cache.pool[cache.table[0, :9].cuda().long()].cpu().numpy()
    from oracle import kvarn_oracle as ko
    for i in range(9):
        a, c = ko.dequantize_record(bytes(recs[i, 0].tobytes()), 128, 4, 2)
        cache.k[0][128 * i:128 * i + 128, 0], cache.v[0][128 * i:128 * i + 128, 0] = a, c
    q, k, v, _ = _inputs(cache, 5, 4, 11)
    sees = np.eye(5, dtype=bool)[None]
    out, _ = _run(kv, cache, q, k, v, B.pack_mask(sees))
    on = np.concatenate([np.ones((5, 128 * 9), dtype=bool), sees[0]], axis=1)
    ref = B.expected(cache, 0, q[0].double().numpy(), k[0].double().numpy(), v[0].double().numpy(), on, B.scale_of(128), 4)
    B.close(out[0].double().numpy(), ref, "growing logits")


def _growing(cache):
    g = torch.Generator().manual_seed(12)
    k = torch.randn((128 * 9, 1, 128), generator=g) * torch.linspace(0.1, 40.0, 128 * 9)[:, None, None]
    return k.half(), torch.randn((128 * 9, 1, 128), generator=g).half()


def test_tree_is_deterministic_and_replays(kv):
    cache = B.Cache(kv, [700, 2000, 1], 2, 128, 13)
    q, k, v, g = _inputs(cache, 18, 8, 14)
    mask = B.pack_mask(np.stack([B.ancestors(18, g) for _ in range(3)]))
    first, _ = _run(kv, cache, q, k, v, mask)
    q_d, k_d, v_d, mask_d, table_d = q.cuda(), k.cuda(), v.cuda(), mask.cuda(), cache.table.cuda()
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    ws = kv.alloc_tree_workspace(cache.desc, 3, 8, 18, cache.table.shape[1])

    def call():
        kv.tree_attention(cache.desc, q_d, k_d, v_d, mask_d, cache.pool, table_d, cache.lens_t, out, ws, **cache.args)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), first)


def test_tree_device_errors(kv):
    cache = B.Cache(kv, [300, 260], 1, 128, 15)
    q, k, v, _ = _inputs(cache, 4, 4, 16)
    cache.table[0, 1] = 10 ** 6
    _, status = _run(kv, cache, q, k, v, None)
    assert status == kv.DEV_BAD_PAGE_ID
    cache.table[0, 1] = 0
    _, status = _run(kv, cache, q, k, v, None, tree_lens=[5, -1])
    assert status == kv.DEV_SEQ_TOO_LONG
    _, status = _run(kv, cache, q, k, v, None, partial_k=None, partial_v=None)
    assert status == kv.DEV_NO_PARTIAL
    cache.lens_t[1] = 10 ** 6
    _, status = _run(kv, cache, q, k, v, None)
    assert status & kv.DEV_SEQ_TOO_LONG
