"""Block tables and slot maps planned on the GPU, and the slot-mapped store of the fp16 cache (GPU).

Both move or count whole things: everything is compared for equality with a request-by-request restatement.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TILE = 128


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def _pages(n, open_tiles):
    return n // TILE if open_tiles else -(-n // TILE)


def expected(table, lens, new, chunk, pool, open_tiles):
    """(table, lengths, slots, status bits) after the call, by its definition."""
    table, width, status = table.copy(), table.shape[1], 0
    rows = []
    for length, add in zip(lens, new):
        bad = add < 0 or add > chunk
        add = min(max(add, 0), chunk)
        held = min(_pages(max(length, 0), open_tiles), width)
        if length < 0 or _pages(length + add, open_tiles) > width:
            bad, after, add = True, held, None
        else:
            after = _pages(length + add, open_tiles)
        status |= 2 * bad
        rows.append((length, add, held, after))
    named = set()
    for b, (_, _, held, _) in enumerate(rows):
        for p in table[b, :held].tolist():
            if 0 <= p < pool:
                named.add(p)
            else:
                status |= 1
    free = [p for p in range(pool) if p not in named] if pool < 50000 else None
    if free is None:
        mask = np.ones(pool, dtype=bool)
        mask[list(named)] = False
        free = np.nonzero(mask)[0]
    out = np.array(lens)
    slots = np.full((len(lens), chunk), -1, dtype=np.int64)
    wanted, taken = 0, 0
    for b, (length, add, held, after) in enumerate(rows):
        need = after - held
        wanted += need
        if need and wanted > len(free):
            status |= 16
            continue
        table[b, held:after] = free[taken:taken + need]
        taken += need
        if add is None:
            continue
        out[b] = length + add
        for i in range(add):
            at = length + i
            if at // TILE < after:
                p = int(table[b, at // TILE])
                if 0 <= p < pool:
                    slots[b, i] = p * TILE + at % TILE
                else:
                    status |= 1
    return table, out, slots, status


def make_table(lens, width, pool, open_tiles, rng, shared=1):
    """Rows of different pages (the first half common to `shared` rows), -9 past them."""
    table = np.full((len(lens), width), -9, dtype=np.int32)
    perm, at = rng.permutation(pool).astype(np.int32), 0
    for b, n in enumerate(lens):
        held = _pages(max(n, 0), open_tiles)
        first = 0
        if b % shared:
            first = min(held, _pages(max(lens[b - b % shared], 0), open_tiles)) // 2
            table[b, :first] = table[b - b % shared, :first]
        table[b, first:held] = perm[at:at + held - first]
        at += held - first
    return table


def run(kv, table, lens, new, chunk, pool, open_tiles, slots=True, all_new=False, **kw):
    dev = "cuda"
    t = torch.from_numpy(table).to(dev)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    nw = None if all_new else torch.tensor(new, dtype=torch.int32, device=dev)
    out = torch.full((len(lens),), -5, dtype=torch.int32, device=dev)
    sm = torch.full((len(lens), chunk), -7, dtype=torch.int64, device=dev) if slots else None
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kv.plan_pages(ln, t, pool, out, new_lens=nw, chunk_len=chunk, slot_map=sm, open_tiles=open_tiles, status=status, **kw)
    torch.cuda.synchronize()
    return t.cpu().numpy(), out.cpu().numpy(), None if sm is None else sm.cpu().numpy(), int(status.item())


def check(kv, table, lens, new, chunk, pool, open_tiles, **kw):
    et, eo, es, ef = expected(table, lens, new, chunk, pool, open_tiles)
    t, o, s, f = run(kv, table, lens, new, chunk, pool, open_tiles, **kw)
    assert np.array_equal(t, et)
    assert np.array_equal(o, eo)
    if s is not None:
        assert np.array_equal(s, es)
    assert f == ef
    return ef


@pytest.mark.parametrize("open_tiles", [True, False])
@pytest.mark.parametrize("batch,chunk,top,pool,shared", [
    (1, 1, 1, 1, 1), (1, 1, 128, 5, 1), (1, 300, 1000, 40, 1), (3, 7, 500, 64, 1), (33, 1, 2000, 700, 4),
    (64, 129, 3000, 5000, 1), (257, 1, 400, 3000, 8), (1025, 2, 300, 9000, 1), (5, 4000, 100, 4000, 1),
    (2, 1, 70000, 20000, 1), (40, 513, 9000, 100001, 3)])
def test_plan(kv, batch, chunk, top, pool, shared, open_tiles):
    rng = np.random.default_rng(batch * 1000 + chunk)
    lens = rng.integers(0, top + 1, batch)
    lens[0] = top // 2
    lens[-1] = top // TILE * TILE  # a whole number of tiles
    lens = lens.tolist()
    new = rng.integers(0, chunk + 1, batch).tolist()
    width = max(_pages(n + m, open_tiles) for n, m in zip(lens, new)) + 3
    if sum(_pages(n, open_tiles) for n in lens) > pool:
        pytest.skip("the pool does not hold the sequences")
    table = make_table(lens, width, pool, open_tiles, rng, shared)
    check(kv, table, lens, new, chunk, pool, open_tiles)


@pytest.mark.parametrize("pages", [0, 1, 5, 6, 7, 30])
def test_plan_pool_runs_out(kv, pages):
    # wants 2, 0, 4, 1, 0, 3 pages; the pool has `pages` left
    lens, new = [100, 20, 256, 383, 130, 1], [150, 30, 512, 2, 60, 400]
    rng = np.random.default_rng(3)
    held = sum(n // TILE for n in lens)
    table = make_table(lens, 9, held + pages, True, rng)
    flags = check(kv, table, lens, new, 512, held + pages, True)
    assert (flags == 16) == (pages < 10)


def test_plan_bad_lengths_and_pages(kv):
    rng = np.random.default_rng(5)
    lens = [-1, 200, 128 * 6, 128 * 6 - 1, 500, 50, 2**31 - 1, -2**31, 300]
    new = [5, -3, 1, 1, 99, 20, 20, 20, 2**31 - 1]
    table = make_table([max(0, min(n, 700)) for n in lens], 6, 60, True, rng)
    table[4, 1], table[8, 0], table[2, 5], table[6, :] = 60, -1, 2**31 - 1, 7
    for open_tiles in (True, False):
        assert check(kv, table, lens, new, 20, 60, open_tiles) & 3 == 3


def test_plan_without_slots_or_lens(kv):
    rng = np.random.default_rng(6)
    lens = [0, 127, 128, 1000]
    table = make_table(lens, 12, 50, True, rng)
    check(kv, table, lens, [9] * 4, 9, 50, True, all_new=True)
    check(kv, table, lens, [9] * 4, 9, 50, True, all_new=True, slots=False)


def test_plan_gives_back_pages_of_empty_sequences(kv):
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    lens, new = [512, 0, 256], [0, 0, 256]  # the second sequence ended: its pages go to the third
    t, o, _, f = run(kv, table, lens, new, 256, 12, True)
    assert t.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 4, 5]] and o.tolist() == [512, 0, 512] and f == 0


@pytest.mark.parametrize("batch,pool", [(3, 1 << 20), (3, (1 << 20) + 1), (40, 3_000_001)])
def test_plan_large_pools(kv, batch, pool):
    # pools around and past what one CTA keeps a whole bitmap of; all pages but a few at the end are taken
    rng = np.random.default_rng(batch)
    lens = rng.integers(100, 3000, batch).tolist()
    new = rng.integers(0, 700, batch).tolist()
    table = make_table(lens, 32, 600, True, rng, shared=2)
    table = np.where(table >= 0, pool - 1 - table, table).astype(np.int32)
    check(kv, table, lens, new, 700, pool, True)
    check(kv, table, lens, new, 700, pool, False)


def test_plan_largest(kv):
    # the most rows, the largest pool: a few pages at its very end are free
    batch, pool = 16384, 1 << 23
    width = 512
    table = np.arange(batch * width, dtype=np.int32).reshape(batch, width)
    lens = [width * TILE - 1] * batch
    table[:5, 100] = 1  # five pages become free in the middle
    t, o, s, f = run(kv, table, lens, [0] * (batch - 8) + [2] * 8, 2, pool, True)
    # all tables hold 511 pages: page 512 r + 511 is free, beside the five
    et, eo, es, ef = expected(table, lens, [0] * (batch - 8) + [2] * 8, 2, pool, True)
    assert np.array_equal(t, et) and np.array_equal(o, eo) and np.array_equal(s, es) and f == ef


def test_plan_captured_and_other_stream(kv):
    rng = np.random.default_rng(8)
    lens, new = [100, 300, 1000], [60, 90, 200]
    table = make_table(lens, 12, 40, False, rng)
    et, eo, es, _ = expected(table, lens, new, 200, 40, False)
    t = torch.from_numpy(table).cuda()
    ln, nw = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, new))
    out, sm = torch.zeros_like(ln), torch.zeros(3, 200, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kv.plan_pages(ln, t, 40, out, new_lens=nw, chunk_len=200, slot_map=sm, open_tiles=False, stream=side)
    side.synchronize()
    assert np.array_equal(t.cpu().numpy(), et)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.plan_pages(ln, t, 40, out, new_lens=nw, chunk_len=200, slot_map=sm, open_tiles=False)
    for _ in range(3):
        t.copy_(torch.from_numpy(table)), out.zero_(), sm.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(t.cpu().numpy(), et) and np.array_equal(out.cpu().numpy(), eo)
        assert np.array_equal(sm.cpu().numpy(), es)


def stored(k, v, slots, pool):
    """The pool after the tokens are written."""
    out = pool.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pool.shape[0] * TILE:
            out[s // TILE, :, 0, s % TILE] = k[t]
            out[s // TILE, :, 1, s % TILE] = v[t]
    return out


@pytest.mark.parametrize("tokens,heads,dim,layout", [
    (1, 1, 64, "plain"), (1, 8, 128, "fused"), (7, 3, 64, "fused"), (130, 5, 128, "plain"), (1023, 2, 64, "heads"),
    (1025, 1, 128, "plain"), (2051, 8, 128, "fused"), (1500, 65, 64, "plain")])
def test_store(kv, tokens, heads, dim, layout):
    g = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // TILE) + 3
    slots = torch.randperm(pages * TILE, generator=g)[:tokens]
    slots[torch.rand(tokens, generator=g) < 0.1] = -1
    if layout == "plain":
        k, v = (torch.randn(tokens, heads, dim, generator=g).half() for _ in range(2))
    elif layout == "fused":
        qkv = torch.randn(tokens, 4 * heads, dim, generator=g).half()
        k, v = qkv[:, 2 * heads:3 * heads], qkv[:, 3 * heads:]
    else:  # heads first
        k, v = (torch.randn(heads, tokens, dim, generator=g).half().transpose(0, 1) for _ in range(2))
    pool = torch.randn(pages, heads, 2, TILE, dim, generator=g).half()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x) for x in (k, v))
    got = pool.cuda()
    kv.fp16_store(kc, vc, slots.cuda(), got, status=status)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), stored(k, v, slots, pool)) and status.item() == 0


def test_store_bad_slots(kv):
    k = torch.randn(4, 2, 64).half()
    slots = torch.tensor([5, 3 * TILE, -2**62, 2**62])
    pool = torch.zeros(3, 2, 2, TILE, 64).half()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pool.cuda()
    kv.fp16_store(k.cuda(), k.cuda(), slots.cuda(), got, status=status)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), stored(k, k, slots, pool)) and status.item() == kv.DEV_BAD_PAGE_ID


def test_store_past_32_bits(kv):
    # a pool of 4.3e9 bytes and more: the last page's offsets pass 32 bits
    heads, dim = 8, 128
    pages = 8400
    pool = torch.zeros(pages, heads, 2, TILE, dim, dtype=torch.float16, device="cuda")
    k = torch.randn(2, heads, dim, device="cuda").half()
    kv.fp16_store(k, -k, torch.tensor([pages * TILE - 1, 0], device="cuda"), pool)
    torch.cuda.synchronize()
    assert torch.equal(pool[-1, :, 0, -1], k[0]) and torch.equal(pool[-1, :, 1, -1], -k[0])
    assert torch.equal(pool[0, :, 0, 0], k[1]) and int((pool != 0).sum()) == int((k != 0).sum()) * 2


def test_plan_store_decode(kv):
    """Ragged prompts planned, stored and attended to: the same as attention over the tokens themselves."""
    heads, dim, hq = 2, 64, 4
    lens = [5, 128, 300, 1]
    chunk, width, pool_pages = 300, 4, 24
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(4, chunk, heads, dim, generator=g).half() for _ in range(2))
    q = torch.randn(4, hq, dim, generator=g).half()
    table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    zero, new = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out_lens, slots = torch.zeros_like(zero), torch.zeros(4, chunk, dtype=torch.int64, device="cuda")
    pool = torch.full((pool_pages, heads, 2, TILE, dim), float("nan"), dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.plan_pages(zero, table, pool_pages, out_lens, new_lens=new, chunk_len=chunk, slot_map=slots, open_tiles=False,
                  status=status)
    kv.fp16_store(k.cuda().flatten(0, 1), v.cuda().flatten(0, 1), slots, pool, status=status)
    out = torch.empty(4, hq, dim, dtype=torch.float16, device="cuda")
    ws = kv.alloc_fp16_workspace(dim, 4, hq, width)
    kv.fp16_decode_attention(heads, q.cuda(), pool, table, out_lens, out, ws, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and out_lens.tolist() == lens
    for b, n in enumerate(lens):
        for h in range(hq):
            kk, vv = k[b, :n, h // 2].double(), v[b, :n, h // 2].double()
            p = torch.softmax(kk @ q[b, h].double() / dim ** 0.5, 0)
            assert (out[b, h].double().cpu() - p @ vv).abs().max() <= 2e-3 * max(1.0, float((p @ vv).abs().max()))
