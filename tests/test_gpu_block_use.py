"""The tree and windowed calls as a program uses them: together, on streams, with odd buffers."""

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


def _half(g, *shape):
    return torch.randn(shape, generator=g).half().cuda()


def test_speculative_step(kv):
    # draft a chain of four tokens, keep two: the third row of the tree is then the decode step after
    # appending them (one sequence seals its tile with the second token)
    cache = B.Cache(kv, [300, 126, 40], 2, 128, 40)
    g = torch.Generator().manual_seed(41)
    q, k, v = _half(g, 3, 4, 8, 128), _half(g, 3, 4, 2, 128), _half(g, 3, 4, 2, 128)
    table = torch.cat([cache.table, torch.zeros((3, 1), dtype=torch.int32)], 1).contiguous().cuda()
    table[1, 0] = cache.free_page
    out = torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.tree_attention(cache.desc, q, k, v, None, cache.pool, table, cache.lens_t, out,
                      kv.alloc_tree_workspace(cache.desc, 3, 8, 4, table.shape[1]), status=status, **cache.args)
    lens = [cache.lens_t.clone(), torch.zeros_like(cache.lens_t)]
    for i in range(3):
        kv.append_token(cache.desc, k[:, i].contiguous(), v[:, i].contiguous(), cache.args["partial_k"],
                        cache.args["partial_v"], lens[i % 2], table, cache.pool, seq_lens_out=lens[1 - i % 2],
                        status=status)
    step = torch.empty((3, 8, 128), dtype=torch.float16, device="cuda")
    kv.decode_attention(cache.desc, q[:, 2].contiguous(), cache.pool, table, lens[1], step,
                        kv.alloc_workspace(cache.desc, 3, 8, table.shape[1]), status=status, **cache.args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and lens[1].tolist() == [303, 129, 43]
    for b in (0, 2):  # sequence 1's raw tokens became a quantised page in between
        B.close(out[b, 2].cpu().double().numpy(), step[b].cpu().double().numpy(), "kept draft b=%d" % b)
    assert torch.isfinite(step).all()


def test_two_streams_at_once(kv):
    cache = B.Cache(kv, [1500, 700, 2100], 2, 128, 42)
    g = torch.Generator().manual_seed(43)
    table = cache.table.cuda()
    calls, outs = [], []
    for nodes in (5, 20):
        q, k, v = _half(g, 3, nodes, 8, 128), _half(g, 3, nodes, 2, 128), _half(g, 3, nodes, 2, 128)
        out = torch.empty_like(q)
        ws = kv.alloc_tree_workspace(cache.desc, 3, 8, nodes, table.shape[1])
        calls.append(lambda q=q, k=k, v=v, out=out, ws=ws: kv.tree_attention(
            cache.desc, q, k, v, None, cache.pool, table, cache.lens_t, out, ws, **cache.args))
        outs.append(out)
    q = _half(g, 3, 8, 128)
    out = torch.empty_like(q)
    ws = kv.alloc_window_decode_workspace(cache.desc, 3, 8, table.shape[1], 4, 900)
    calls.append(lambda: kv.window_decode_attention(cache.desc, q, cache.pool, table, cache.lens_t, out, ws, 4, 900,
                                                    **cache.args))
    outs.append(out)
    for call in calls:
        call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for call, s in zip(calls, streams):
                with torch.cuda.stream(s):
                    call()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_queries_at_any_address(kv):
    # q and out need no more than their element's alignment
    cache = B.Cache(kv, [700, 5], 2, 96, 44)
    g = torch.Generator().manual_seed(45)
    table = cache.table.cuda()
    q, k, v = _half(g, 2, 9, 8, 96), _half(g, 2, 9, 2, 96), _half(g, 2, 9, 2, 96)
    want = torch.empty_like(q)
    ws = kv.alloc_tree_workspace(cache.desc, 2, 8, 9, table.shape[1])
    kv.tree_attention(cache.desc, q, k, v, None, cache.pool, table, cache.lens_t, want, ws, **cache.args)
    for shift in (1, 2, 4):
        buf = torch.empty(2, q.numel() + 8, dtype=torch.float16, device="cuda")
        q2, out = (buf[i, shift:shift + q.numel()].view(q.shape) for i in range(2))
        q2.copy_(q)
        kv.tree_attention(cache.desc, q2, k, v, None, cache.pool, table, cache.lens_t, out, ws, **cache.args)
        assert torch.equal(out, want)
    qd = q[:, 0].contiguous()
    want = torch.empty_like(qd)
    ws = kv.alloc_window_decode_workspace(cache.desc, 2, 8, table.shape[1], 1, 300)
    kv.window_decode_attention(cache.desc, qd, cache.pool, table, cache.lens_t, want, ws, 1, 300, **cache.args)
    buf = torch.empty(2, qd.numel() + 8, dtype=torch.float16, device="cuda")
    q2, out = (buf[i, 1:1 + qd.numel()].view(qd.shape) for i in range(2))
    q2.copy_(qd)
    kv.window_decode_attention(cache.desc, q2, cache.pool, table, cache.lens_t, out, ws, 1, 300, **cache.args)
    assert torch.equal(out, want)


def test_pages_past_4_gib(kv):
    # the pool is larger than 32-bit offsets reach and the sequence's pages lie at its end
    cache = B.Cache(kv, [128 * 6 + 9], 1, 128, 46)
    far = 330000
    pool = torch.empty((far, 1, cache.desc.page_record_bytes), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    pool[far - cache.n_pool:] = cache.pool
    g = torch.Generator().manual_seed(47)
    q, k, v = _half(g, 1, 6, 4, 128), _half(g, 1, 6, 1, 128), _half(g, 1, 6, 1, 128)
    outs = []
    for p, t in ((cache.pool, cache.table.cuda()), (pool, (cache.table + (far - cache.n_pool)).int().cuda())):
        out = torch.empty_like(q)
        kv.tree_attention(cache.desc, q, k, v, None, p, t, cache.lens_t, out,
                          kv.alloc_tree_workspace(cache.desc, 1, 4, 6, t.shape[1]), **cache.args)
        wd = torch.empty((1, 4, 128), dtype=torch.float16, device="cuda")
        kv.window_decode_attention(cache.desc, q[:, 0].contiguous(), p, t, cache.lens_t, wd,
                                   kv.alloc_window_decode_workspace(cache.desc, 1, 4, t.shape[1], 1, 300), 1, 300,
                                   **cache.args)
        outs.append((out, wd))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_masked_tokens_of_the_lowest_values(kv):
    # infinities and NaN in tokens that no row sees leave the outputs alone
    cache = B.Cache(kv, [260], 1, 128, 48)
    g = torch.Generator().manual_seed(49)
    q, k, v = _half(g, 1, 5, 4, 128), _half(g, 1, 5, 1, 128), _half(g, 1, 5, 1, 128)
    sees = np.zeros((1, 5, 5), dtype=bool)
    sees[0, :, :3] = np.tril(np.ones((5, 3), dtype=bool))
    table = cache.table.cuda()
    ws = kv.alloc_tree_workspace(cache.desc, 1, 4, 5, table.shape[1])

    def run(k, v):
        out = torch.empty_like(q)
        kv.tree_attention(cache.desc, q, k, v, B.pack_mask(sees).cuda(), cache.pool, table, cache.lens_t, out, ws,
                          **cache.args)
        return out

    want = run(k, v)
    for bad in (-65504.0, 65504.0):
        k2, v2 = k.clone(), v.clone()
        k2[:, 3:] = bad
        v2[:, 3:] = bad
        assert torch.equal(run(k2, v2), want)
    # keys that no row sees may hold anything; their values enter a product with 0
    k2 = k.clone()
    k2[:, 3] = float("inf")
    k2[:, 4] = float("nan")
    assert torch.equal(run(k2, v), want)


def test_argument_checks(kv):
    cache = B.Cache(kv, [200], 2, 128, 50)
    g = torch.Generator().manual_seed(51)
    q, k, v = _half(g, 1, 4, 8, 128), _half(g, 1, 4, 2, 128), _half(g, 1, 4, 2, 128)
    table = cache.table.cuda()
    ws = kv.alloc_tree_workspace(cache.desc, 1, 8, 4, table.shape[1])
    good = dict(q=q, tree_k=k, tree_v=v, tree_mask=torch.ones((1, 4, 1), dtype=torch.int32, device="cuda"),
                pool=cache.pool, block_table=table, cache_lens=cache.lens_t, out=torch.empty_like(q), workspace=ws,
                **cache.args)
    kv.tree_attention(cache.desc, **good)
    bad = [dict(q=q.float()), dict(q=q[:, :, :, :64]), dict(tree_k=k[:, :3]), dict(tree_v=v.transpose(1, 2)),
           dict(tree_mask=torch.ones((1, 4, 2), dtype=torch.int32, device="cuda")), dict(tree_mask=good["tree_mask"].long()),
           dict(pool=cache.pool[:, :1]), dict(block_table=table.long()), dict(cache_lens=cache.lens_t.long()),
           dict(out=torch.empty_like(q)[:, :2]), dict(partial_k=cache.args["partial_k"][:, :, :64]),
           dict(tree_lens=torch.ones(2, dtype=torch.int32, device="cuda")),
           dict(status=torch.zeros(0, dtype=torch.int32, device="cuda")), dict(out=torch.empty_like(q).cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            kv.tree_attention(cache.desc, **dict(good, **kw))
    with pytest.raises(kv.KvarnError) as e:
        kv.tree_attention(cache.desc, **dict(good, workspace=ws[:16]))
    assert e.value.status == kv.KVARN_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(kv.KvarnError) as e:
        kv.window_decode_attention(cache.desc, q[:, 0].contiguous(), cache.pool, table, cache.lens_t,
                                   torch.empty_like(q[:, 0]).contiguous(), ws, 0, 0, **cache.args)
    assert e.value.status == kv.KVARN_ERR_INVALID_ARG


def test_a_nan_query_is_not_answered_with_zeros(kv):
    # a query of NaN that sees sealed pages only gives NaN, as the decode call does, and its
    # neighbours keep their outputs
    cache = B.Cache(kv, [256, 1536], 1, 128, 52)
    g = torch.Generator().manual_seed(53)
    q, k, v = _half(g, 2, 5, 4, 128), _half(g, 2, 5, 1, 128), _half(g, 2, 5, 1, 128)
    sees = np.zeros((2, 5, 5), dtype=bool)
    sees[:, 0] = True
    table = cache.table.cuda()
    ws = kv.alloc_tree_workspace(cache.desc, 2, 4, 5, table.shape[1])

    def run(q):
        out = torch.empty_like(q)
        kv.tree_attention(cache.desc, q, k, v, B.pack_mask(sees).cuda(), cache.pool, table, cache.lens_t, out, ws,
                          **cache.args)
        return out.cpu().double()

    want = run(q)
    bad = q.clone()
    bad[0, 2, 1, 7] = float("nan")
    bad[1, 3] = float("nan")
    bad[1, 0, 0] = float("nan")  # sees raw tokens too
    got = run(bad)
    nan = torch.isnan(bad).any(-1).cpu()
    assert torch.isnan(got[nan]).all()
    B.close(got[~nan].numpy(), want[~nan].numpy(), "rows beside a NaN query")
    step = torch.empty((2, 4, 128), dtype=torch.float16, device="cuda")
    kv.decode_attention(cache.desc, bad[:, 3].contiguous(), cache.pool, table, cache.lens_t, step,
                        kv.alloc_workspace(cache.desc, 2, 4, table.shape[1]), **cache.args)
    assert torch.isnan(step[1]).all() and torch.isfinite(step[0]).all()
