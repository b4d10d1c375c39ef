"""The windowed and tree calls at sizes where rows, splits and CTAs outnumber each other, against 64 bits.

Tolerance of the calls of thousands of rows.  All but one row in a thousand are held to the decode
tolerance (tests/helpers.py).  It is a share of max |out|, which does not bound a row whose weight lies on
two or three tokens that differ by far more than its output: there an error e of a logit moves the output
by e p1 p2 |V1 - V2|.  With keys of outlier channels a logit of some hundreds is a sum of terms of thousands,
and the whole-cache decode, which splits its operands the same way, has such rows too (2-bit keys, head_dim
64: one of 16,384 at 2.6e-3).  So every element is held to what the arithmetic allows it:
  output      rounded to fp16: 2^-11 |o|, and 2^-25 below fp16's normal range;
  weights     P rounded to fp16: 2^-11 relative; logits (powers of two): the chained matrix steps, 2 d / 16
              of the codes and d / 16 of the zeros, are each off by at most one unit (2^-23) of a partial
              sum, which C = sum of |terms| bounds: e = ln 2 (3 d / 16) 2^-23 C.  A weight off by w moves
              o by at most p w (|V| + |o|);
  V~          rounded twice, 2^-11 relative each, and rotated back: five standard deviations of 2^-11 sqrt(2 / 3)
              of the value row's rms.
"""

import math

import numpy as np
import pytest
import torch

from oracle import kvarn_oracle as ko
from tests import block_cases as B
from tests import helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def _term_sizes(cache, b, d):
    """code |s'| + |z'|, times the token factors, of sequence b's sealed keys, [tokens, kv heads, d], rotated basis."""
    n = cache.lens[b] // 128
    recs = cache.pool[cache.table[b, :n].clamp(min=0).cuda().long()].cpu().numpy()
    out = np.zeros((128 * n, cache.hkv, d))
    for i in range(n):
        for h in range(cache.hkv):
            k = ko.unpack_record(bytes(recs[i, h].tobytes()), d, *cache.bits)[0]
            s, z, r = (np.asarray(k[x], dtype=np.float64) for x in ("scale", "zero", "factor"))
            out[128 * i:128 * i + 128, h] = (np.asarray(k["codes"]) * np.abs(s) + np.abs(z)) * np.abs(r)[:, None]
    return out


class RowCheck:
    def __init__(self):
        self.errors, self.share = [], 0.0  # per row: max error over max(1, max |out|); worst share of the bound

    def sequence(self, cache, b, got, q, new_k, new_v, on, group):
        """got, q [rows, Hq, d0] of sequence b, new_k/v [tokens, Hkv, d0], on [rows, cached + tokens]."""
        d0, d = cache.d0, ko.padded_head_dim(cache.d0)
        rot = ko.sylvester_hadamard(d) / math.sqrt(d)
        sizes, n = _term_sizes(cache, b, d), 128 * (cache.lens[b] // 128)
        scale = B.scale_of(d0)
        for hq in range(q.shape[1]):
            h, qh = hq // group, q[:, hq]
            k, v = np.concatenate([cache.k[b][:, h], new_k[:, h]]), np.concatenate([cache.v[b][:, h], new_v[:, h]])
            s = np.where(on, (qh @ k.T) * scale, -np.inf)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - np.where(np.isinf(m), 0.0, m))
            total = p.sum(axis=1, keepdims=True)
            p /= np.where(total == 0, 1.0, total)
            o = p @ v
            c = np.zeros(s.shape)
            c[:, :n] = np.abs(qh @ rot[:d0]) @ sizes[:, h].T
            c[:, n:] = np.abs(qh) @ np.abs(k[n:]).T
            w = p * (2.0 ** -11 + (3 * d / 16) * 2.0 ** -23 * scale * c)  # ln 2 (log2 e) = 1
            rms = np.zeros(len(v))
            rms[:n] = np.sqrt((v[:n] ** 2).sum(axis=1) / d)
            tol = 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + w @ np.abs(v) + w.sum(axis=1, keepdims=True) * np.abs(o)
            tol += (5 * 2.0 ** -11 * math.sqrt(2 / 3)) * (p @ rms)[:, None]
            err = np.abs(got[:, hq] - o)
            assert np.isfinite(got[:, hq]).all()
            worst = np.unravel_index((err / tol).argmax(), err.shape)
            assert err[worst] <= tol[worst], "sequence %d head %d row %d: %.3e of %.3e" % (b, hq, worst[0], err[worst],
                                                                                          tol[worst])
            self.share = max(self.share, float((err / tol).max()))
            self.errors.append(err.max(axis=1) / np.maximum(1.0, np.abs(o).max(axis=1)))

    def finish(self, what):
        e = np.concatenate(self.errors)
        print("%s: %d rows, scaled error %.1e, at most %.1e, %.2f of the bound" % (what, e.size, np.median(e), e.max(),
                                                                                self.share))
        assert (e > H.DECODE_TOL).mean() <= 1e-3


def _inputs(lens, block, hkv, group, d0, seed):
    g = torch.Generator().manual_seed(seed + 1)
    n = len(lens)
    q = torch.randn((n, block, hkv * group, d0), generator=g).half()
    k = (2 * torch.randn((n, block, hkv, d0), generator=g)).half()
    v = torch.randn((n, block, hkv, d0), generator=g).half()
    return q, k, v, g


def _prefill(kv, lens, chunk, hkv, group, d0, sink, window, seed, preset="kvarn_k4v2_g128", chunk_lens=None):
    cache = B.Cache(kv, lens, hkv, d0, seed, preset)
    q, k, v, _ = _inputs(lens, chunk, hkv, group, d0, seed)
    n, hq = len(lens), hkv * group
    sizes = [chunk] * n if chunk_lens is None else chunk_lens
    table = cache.table.clone()
    on = [B.window_mask(lens[b], chunk, lens[b] + chunk, sink, window)[:sizes[b]] for b in range(n)]
    for b in range(n):  # pages that no query sees
        seen = on[b][:, :128 * (lens[b] // 128)].any(axis=0).reshape(-1, 128).any(axis=1)
        table[b, [i for i in range(len(seen)) if not seen[i]]] = -7
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = kv.alloc_window_prefill_workspace(cache.desc, n, hq, chunk, table.shape[1], sink, window)
    ws.fill_(float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.window_prefill_attention(cache.desc, q.cuda(), k.cuda(), v.cuda(), cache.pool, table.cuda(), cache.lens_t, out, ws,
                                sink, window, chunk_lens=torch.tensor(sizes, dtype=torch.int32, device="cuda"),
                                status=status, **cache.args)
    assert int(status.item()) == 0
    check, out = RowCheck(), out.cpu().double().numpy()
    for b, m in enumerate(sizes):
        check.sequence(cache, b, out[b, :m], *(x[b, :m].double().numpy() for x in (q, k, v)), on[b][:, :lens[b] + m], group)
        assert (out[b, m:] == 7.0).all()
    check.finish("window prefill %dx%d G=%d d0=%d %s" % (n, chunk, group, d0, preset))


@pytest.mark.parametrize("group,d0,preset", [(4, 128, "kvarn_k4v2_g128"), (8, 64, "kvarn_k2v2_g128"),
                                             (2, 256, "kvarn_k4v2_g128")])
def test_window_prefill_of_more_row_tiles_than_ctas(kv, group, d0, preset):
    # 1100 tokens a sequence: 35 to 138 row tiles of each of 6 (sequence, kv head) pairs, 152 CTAs; the
    # window (1500) is longer than the chunk, the first 70 tokens stay
    _prefill(kv, [5000, 700, 129], 1100, 2, group, d0, 70, 1500, seed=80 + d0, preset=preset,
             chunk_lens=[1100, 1037, 64])


def test_window_prefill_of_a_chunk_longer_than_its_window(kv):
    # rows whose window has left the cache, and the chunk's own first tokens
    _prefill(kv, [1000, 0], 1500, 1, 4, 128, 5, 300, seed=84)


def test_window_prefill_row_tiles_cut_over_many_ctas(kv):
    # three row tiles of 118 visible pages each, a CTA for every few of them
    _prefill(kv, [128 * 150 + 77], 40, 1, 4, 128, 300, 14700, seed=85)


def test_tree_of_more_row_tiles_than_ctas(kv):
    lens, sizes, group = [128 * 3, 77, 1000, 513], [300, 299, 1, 128], 8
    cache = B.Cache(kv, lens, 2, 128, 86)
    q, k, v, g = _inputs(lens, 300, 2, group, 128, 86)
    sees = np.stack([B.ancestors(300, g) for _ in lens])
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = kv.alloc_tree_workspace(cache.desc, 4, 16, 300, cache.table.shape[1])
    ws.fill_(float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.tree_attention(cache.desc, q.cuda(), k.cuda(), v.cuda(), B.pack_mask(sees).cuda(), cache.pool, cache.table.cuda(),
                      cache.lens_t, out, ws, tree_lens=torch.tensor(sizes, dtype=torch.int32, device="cuda"),
                      status=status, **cache.args)
    assert int(status.item()) == 0
    check, out = RowCheck(), out.cpu().double().numpy()
    for b, m in enumerate(sizes):
        on = np.concatenate([np.ones((m, lens[b]), dtype=bool), sees[b, :m, :m]], axis=1)
        check.sequence(cache, b, out[b, :m], *(x[b, :m].double().numpy() for x in (q, k, v)), on, group)
        assert (out[b, m:] == 7.0).all()
    check.finish("tree 4x300")


def test_window_decode_of_more_than_32_splits(kv):
    # one row of 605 visible pages in ranges of at least 16: 50 pages that the table names 14 times
    reps, sink, window = 14, 200, 77000
    cache = B.Cache(kv, [128 * 50 + 77], 1, 128, 87)
    k, v = (np.concatenate([np.tile(x[:6400], (reps, 1, 1)), x[6400:]]) for x in (cache.k[0], cache.v[0]))
    n = len(k)
    cache.k, cache.v = [k], [v]
    table = cache.table[:, :50].repeat(1, reps)
    on = B.window_mask(n - 1, 1, n, sink, window)
    seen = on[0, :128 * 50 * reps].reshape(-1, 128).any(axis=1)
    assert seen.sum() > 33 * 16 and not seen.all()
    table[0, torch.from_numpy(~seen)] = -7
    q = torch.randn((1, 4, 128), generator=torch.Generator().manual_seed(88)).half()
    out = torch.empty((1, 4, 128), dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = kv.alloc_window_decode_workspace(cache.desc, 1, 4, table.shape[1], sink, window)
    ws.fill_(float("nan"))
    kv.window_decode_attention(cache.desc, q.cuda(), cache.pool, table.cuda(),
                               torch.tensor([n], dtype=torch.int32, device="cuda"), out, ws, sink, window, status=status,
                               **cache.args)
    assert int(status.item()) == 0
    ref = B.expected(cache, 0, q.double().numpy(), None, None, on, B.scale_of(128), 4)
    print("window decode 605 pages: %.2e" % B.close(out.cpu().double().numpy(), ref, "window decode"))


def test_window_prefill_replays_beside_other_calls(kv):
    # a captured call (two chunks of one stream in a row) replayed while a tree call runs on another
    # stream with a workspace of its own
    cache = B.Cache(kv, [500, 1300], 2, 128, 89)
    g = torch.Generator().manual_seed(90)
    table = cache.table.cuda()
    q, k, v = (torch.randn((2, 200, h, 128), generator=g).half().cuda() for h in (8, 2, 2))
    lens = torch.tensor([200, 133], dtype=torch.int32, device="cuda")
    out, tree = torch.full_like(q, 7.0), torch.empty((2, 9, 8, 128), dtype=torch.float16, device="cuda")
    ws = kv.alloc_window_prefill_workspace(cache.desc, 2, 8, 200, table.shape[1], 4, 300)
    ws_t = kv.alloc_tree_workspace(cache.desc, 2, 8, 9, table.shape[1])
    qt, kt, vt = (x[:, :9].contiguous() for x in (q, k, v))

    def prefill():
        kv.window_prefill_attention(cache.desc, q, k, v, cache.pool, table, cache.lens_t, out, ws, 4, 300,
                                    chunk_lens=lens, **cache.args)

    def draft():
        kv.tree_attention(cache.desc, qt, kt, vt, None, cache.pool, table, cache.lens_t, tree, ws_t, **cache.args)

    prefill()
    draft()
    torch.cuda.synchronize()
    want, want_t = out.clone(), tree.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prefill()
        prefill()
    side = torch.cuda.Stream()
    for _ in range(5):
        out.fill_(7.0)
        tree.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            draft()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(tree, want_t)
    assert bool((out[1, 133:] == 7.0).all())
