"""Selection over beams and vocabulary, and the reordering of the cache's state (GPU).

Selection against 64 bits.  Tolerance of a score: half a step of its own rounding to 32 bits (2^-24 of its
size) and the error of the log-sum-exp.  A term exp(x - ref) is off by 2^-22 (the exponential) and by
2^-23 |x - ref| (two roundings of its argument), weighted by its share of the sum: the mean of |x - ref| is
at most log(vocab) < 17, so 2^-22 + 17 x 2^-23 = 2.3e-6; the 32-bit additions, at most 32 a tile and one a
tile, add 2^-24 each at worst but part of them cancels: 1e-5 in all.  Candidates in another order than the
64-bit one have to be of two beams and no further apart than twice that.
Reordering moves whole things: equality.
"""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

LSE_TOL = 1e-5
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def select(kv, logits, scores, count, done=None, end=-1, **kw):
    batch, beams, vocab = logits.shape
    dev = "cuda"
    outs = [torch.full((batch, count), 7, dtype=t, device=dev) for t in (torch.float32, torch.int32, torch.int32, torch.uint8)]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = kv.alloc_beam_select_workspace(batch, beams, vocab, count)
    ws.fill_(float("nan"))
    kv.beam_select(logits, scores, *outs[:3], ws, done=done, end_token=end, out_done=outs[3], status=status, **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in outs], int(status.item())


def check(kv, logits, scores, count, done=None, end=-1, flags=0):
    """Against the definition, group by group."""
    (got_s, got_p, got_t, got_d), status = select(kv, logits, scores, count, done, end)
    assert status == flags
    batch, beams, vocab = logits.shape
    x = logits.cpu().double().numpy()
    sc = scores.cpu().double().numpy()
    fin = np.zeros((batch, beams), bool) if done is None else done.cpu().numpy().astype(bool)
    for b in range(batch):
        cand = np.full((beams, vocab), -np.inf)
        for k in range(beams):
            row = x[b, k]
            if not sc[b, k] > -np.inf or sc[b, k] == np.inf:
                continue
            if fin[b, k]:
                cand[k, end] = sc[b, k]
                continue
            top = row.max()
            if not abs(top) < np.inf:
                continue
            # the difference from the greatest first: next to 3e38 a logarithm is lost even in 64 bits
            cand[k] = (row - top) + (sc[b, k] - np.log(np.exp(row - top).sum()))
        flat = cand.reshape(-1)
        order = np.argsort(-flat, kind="stable")[:count]
        best = flat[order]
        live = best > -np.inf
        n = int(live.sum())
        assert (got_s[b, n:] == -np.inf).all() and (got_p[b, n:] == -1).all() and (got_t[b, n:] == -1).all()
        assert (got_d[b, n:] == 0).all()
        tol = 2.0 ** -24 * np.abs(best[:n]) + LSE_TOL
        assert (np.abs(got_s[b, :n] - best[:n]) <= tol).all(), np.abs(got_s[b, :n] - best[:n]).max()
        mine = got_p[b, :n].astype(np.int64) * vocab + got_t[b, :n]
        assert (got_p[b, :n] >= 0).all() and (got_p[b, :n] < beams).all() and len(set(mine.tolist())) == n
        assert (np.abs(flat[mine] - best[:n]) <= 2 * LSE_TOL).all()
        for k in range(beams):  # a beam's own candidates: its best, in exact order
            own = [i for i in mine.tolist() if i // vocab == k]
            exact = [i for i in np.argsort(-cand[k], kind="stable")[:len(own)] + k * vocab]
            assert own == [int(i) for i in exact]
        swapped = mine != order[:n]
        assert swapped.mean() <= 0.2 if n > 5 else True
        for j in np.nonzero(swapped)[0]:
            near = np.abs(best[:n] - best[j]) <= 2 * LSE_TOL
            assert near.sum() > 1 or j == n - 1
        ends = np.array([fin[b, p] or t == end for p, t in zip(got_p[b, :n], got_t[b, :n])], dtype=bool)
        assert (got_d[b, :n].astype(bool) == ends).all()


def make(batch, beams, vocab, dtype, seed, scale=3.0, pad=0, shift=0):
    """Logits of the given row padding and offset (elements) from an aligned start; NaN around them."""
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn(batch, beams, vocab, generator=g)
    stride = vocab + pad
    store = torch.full((shift + batch * beams * stride + 64,), float("nan"), dtype=TYPES[dtype], device="cuda")
    out = store[shift:shift + batch * beams * stride].view(batch, beams, stride)[..., :vocab]
    out.copy_(x.to(TYPES[dtype]))
    scores = -30 * torch.rand(batch, beams, generator=g)
    return out, scores.cuda()


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("batch,beams,vocab,count", [
    (1, 1, 1, 1), (1, 1, 1, 3), (2, 1, 2, 2), (1, 3, 5, 15), (1, 3, 5, 20), (2, 4, 33, 8), (3, 5, 1000, 10),
    (1, 4, 2047, 8), (1, 4, 2049, 8), (1, 1, 4096, 64), (1, 32, 4097, 64), (2, 7, 8191, 13), (1, 2, 8193, 1),
    (5, 3, 12289, 6), (1, 4, 100003, 8), (40, 16, 5003, 32), (3, 8, 50257, 16)])
def test_select(kv, batch, beams, vocab, count, dtype):
    logits, scores = make(batch, beams, vocab, dtype, vocab + count)
    check(kv, logits, scores, count, end=vocab // 2)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (2, 2), (4, 4), (8, 8), (7, 3), (24, 2)])
def test_select_alignment(kv, pad, shift, dtype):
    logits, scores = make(2, 3, 20001, dtype, pad * 10 + shift, pad=pad, shift=shift)
    check(kv, logits, scores, 6)


@pytest.mark.parametrize("rows", [150, 700])
def test_select_many_rows(kv, rows):
    logits, scores = make(rows, 2, 3001, "bf16", rows)
    check(kv, logits, scores, 4)


def test_select_finished_and_dead_beams(kv):
    logits, scores = make(6, 4, 999, "bf16", 1)
    done = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    done[0, 1] = done[1, :] = done[2, 3] = done[4, 0] = True
    logits[0, 1] = float("nan")  # a finished beam's logits are not read
    logits[1] = float("inf")
    scores[2, 1] = scores[3, 0] = -math.inf
    scores[4] = -math.inf
    logits[2, 1] = float("nan")
    scores[5, 1:] = -math.inf  # the first step of a search: one live beam
    check(kv, logits, scores, 8, done=done, end=17)
    check(kv, logits, scores, 8, done=done.to(torch.uint8), end=17)


def test_select_finished_scores_tie(kv):
    # Two finished beams of one score: the lower beam first.  -2 + log 4 rounds up to 32 bits, so the live beam's
    # four candidates are -2 + 3.7e-9 and come before them.
    logits = torch.zeros(1, 3, 4, device="cuda")
    scores = torch.tensor([[-2.0, -2.0, -2.0 + math.log(4.0)]], device="cuda")
    done = torch.tensor([[True, True, False]], device="cuda")
    (s, p, t, d), _ = select(kv, logits, scores, 6, done=done, end=1)
    assert 0.0 < float(scores[0, 2]) - math.log(4.0) + 2.0 < 1e-8
    assert p.tolist()[0] == [2, 2, 2, 2, 0, 1] and t.tolist()[0] == [0, 1, 2, 3, 1, 1]
    assert d.tolist()[0] == [0, 1, 0, 0, 1, 1]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_select_masked(kv, dtype):
    logits, scores = make(4, 3, 9001, dtype, 2)
    g = torch.Generator().manual_seed(9)
    logits[0, 0, torch.randperm(9001, generator=g)[:8990].cuda()] = -math.inf
    logits[0, 1] = -math.inf            # nothing left
    logits[0, 2, :9000] = -math.inf     # one token
    logits[1, :, :8500] = -math.inf     # whole tiles masked
    logits[2] = torch.finfo(TYPES[dtype]).min
    logits[2, 1, 4000:4003] = -5.0
    logits[3, :, 3:] = -math.inf        # fewer candidates than asked for
    check(kv, logits, scores, 12)
    logits[:] = -math.inf
    check(kv, logits, scores, 3)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", [0, 4000, 8999])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_select_bad_logits(kv, dtype, where, bad):
    logits, scores = make(2, 3, 9000, dtype, 3)
    logits[0, 1, where] = bad
    check(kv, logits, scores, 6, flags=kv.DEV_BAD_LOGITS)
    logits[0, 1] = -math.inf
    logits[0, 1, where] = bad
    check(kv, logits, scores, 6, flags=kv.DEV_BAD_LOGITS)
    logits[0, 1] = bad
    check(kv, logits, scores, 6, flags=kv.DEV_BAD_LOGITS)
    logits[0, 1] = 0.0
    scores[0, 1] = bad
    check(kv, logits, scores, 6, flags=kv.DEV_BAD_LOGITS)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("kind", ["equal", "rising", "steps", "two values", "zeros", "late"])
def test_select_ties_and_order(kv, kind, dtype):
    """Rows that put more candidates into a tile than the list holds."""
    vocab, t = 40000, TYPES[dtype]
    i = torch.arange(vocab, dtype=torch.float64)
    row = {"equal": torch.full((vocab,), 1.5), "rising": i / 5000, "steps": (i // 700) / 16,
           "two values": torch.where(i % 3 == 0, 2.0, -1.0), "zeros": torch.where(i % 2 == 0, 0.0, -0.0),
           "late": torch.where(i < 30000, -50.0, i / 4000)}[kind]
    logits = row.to(t).expand(2, 3, vocab).contiguous().cuda()
    scores = torch.tensor([[0.0, -1.0, -2.0], [-3.0, -3.0, -3.0]], device="cuda")
    check(kv, logits, scores, 16)
    check(kv, logits, scores, 1)
    check(kv, logits, scores, 64)  # equal scores in all of the merge's lists


def test_select_equal_beams_tie_exactly(kv):
    """Equal rows at different alignments: equal scores, the lower beam first."""
    for vocab in (5001, 70001):
        logits, _ = make(1, 5, vocab, "bf16", 11)
        logits[0, 1:] = logits[0, :1].clone()
        scores = torch.full((1, 5), -4.0, device="cuda")
        (s, p, t, _), _ = select(kv, logits, scores, 15)
        assert (s.reshape(3, 5) == s.reshape(3, 5)[:, :1]).all()
        order = np.argsort(-logits[0, 0].cpu().float().numpy(), kind="stable")
        top, flat = logits[0, 0].cpu().float().numpy()[order], []
        for value in sorted(set(top[:3].tolist()), reverse=True):
            same = sorted(order[top == value].tolist())
            flat += [(k, v) for k in range(5) for v in same]
        assert list(zip(p[0].tolist(), t[0].tolist())) == flat[:15]


@pytest.mark.parametrize("scale", [0.0, 1e-3, 100.0, 1e30])
def test_select_range_of_values(kv, scale):
    logits, scores = make(2, 3, 10007, "fp32", 21, scale=scale)
    if scale == 1e30:  # differences far past 32-bit exponents' arguments
        assert logits.abs().max() > 1e29
    check(kv, logits, scores, 6)
    logits -= 3e5 if scale < 1e30 else 0
    check(kv, logits, scores, 6)


def test_select_again_captured_and_other_stream(kv):
    logits, scores = make(4, 6, 30011, "bf16", 31)
    args = dict(count=12, done=None)
    first, _ = select(kv, logits, scores, **args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for kw in ({}, {"stream": side}):
        again, _ = select(kv, logits, scores, **args, **kw)
        assert all(np.array_equal(a, b) for a, b in zip(first, again))
    outs = [torch.zeros(4, 12, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    ws = kv.alloc_beam_select_workspace(4, 6, 30011, 12)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.beam_select(logits, scores, *outs, ws)
    graph.replay()
    logits[:, :, 5] += 50.0
    second, _ = select(kv, logits, scores, **args)
    graph.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip(second, outs))


@pytest.mark.parametrize("dtype,vocab", [("bf16", 700_003), ("fp32", 400_001)])
@pytest.mark.parametrize("kind", ["random", "rising", "equal", "far", "late inf"])
def test_select_long_chunks(kv, kind, dtype, vocab):
    """Chunks of more elements than are noted at a time: 64 candidates of 32 beams leave a row in one."""
    logits, scores = make(1, 32, vocab, dtype, 41)
    if kind == "rising":
        logits[0, 3] = torch.linspace(-20, 20, vocab, device="cuda").to(logits.dtype)
    elif kind == "equal":
        logits[0, 5:8] = 0.5
    elif kind == "far":  # beyond what the fast path's references hold, late in a chunk
        logits[0, 2, 173_000 if dtype == "bf16" else 98_000] = 3e5
        logits[0, 9] -= 2e5
    elif kind == "late inf":
        logits[0, 4, -1] = math.inf
        logits[0, 6, :600] = -math.inf
    scores[0, 2:10] = -1.0
    check(kv, logits, scores, 64, flags=kv.DEV_BAD_LOGITS if kind == "late inf" else 0)


def test_select_in_place(kv):
    """As many candidates as beams: the new scores and flags may take the place of the old ones."""
    logits, scores = make(5, 4, 2003, "bf16", 51)
    done = torch.zeros(5, 4, dtype=torch.bool, device="cuda")
    done[1, 2] = done[3] = True
    (s, p, t, d), _ = select(kv, logits, scores, 4, done=done, end=11)
    parents, tokens = (torch.zeros(5, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = kv.alloc_beam_select_workspace(5, 4, 2003, 4)
    kv.beam_select(logits, scores, scores, parents, tokens, ws, done=done, end_token=11, out_done=done)
    torch.cuda.synchronize()
    for a, b in ((s, scores), (p, parents), (t, tokens), (d.astype(bool), done)):
        assert np.array_equal(a, b.cpu().numpy())


def test_select_two_calls_at_once(kv):
    calls = []
    for seed in (61, 62):
        logits, scores = make(16, 5, 50_001, "fp16", seed, pad=seed % 2)
        want, _ = select(kv, logits, scores, 10)
        outs = [torch.zeros(16, 10, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
        calls.append((logits, scores, want, outs, kv.alloc_beam_select_workspace(16, 5, 50_001, 10), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for logits, scores, _, outs, ws, stream in calls:
            kv.beam_select(logits, scores, *outs, ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, want, outs, _, _ in calls:
        assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip(want, outs))


def test_select_refuses(kv):
    logits, scores = make(2, 3, 100, "fp16", 71)
    f, i = torch.zeros(2, 6, device="cuda"), torch.zeros(2, 6, dtype=torch.int32, device="cuda")
    ws = kv.alloc_beam_select_workspace(2, 3, 100, 6)
    kv.beam_select(logits, scores, f, i, i.clone(), ws)
    with pytest.raises(ValueError, match="out_tokens"):
        kv.beam_select(logits, scores, f, i, i[:1], ws)
    with pytest.raises(ValueError, match="scores"):
        kv.beam_select(logits, scores.double(), f, i, i, ws)
    with pytest.raises(ValueError, match="logits"):
        kv.beam_select(logits.double(), scores, f, i, i, ws)
    with pytest.raises(ValueError, match="logits"):
        kv.beam_select(logits.transpose(0, 1).contiguous().transpose(0, 1), scores, f, i, i, ws)
    with pytest.raises(kv.KvarnError):
        kv.beam_select(logits, scores, f, i, i, ws[:4])
    with pytest.raises(kv.KvarnError):  # one row for all beams
        kv.beam_select(logits[:, :1].expand(2, 3, 100)[:1], scores[:1].clone(), f[:1], i[:1], i[:1], ws)
    desc = kv.desc_from_preset(64, 1)
    t = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    n, p = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    k = torch.zeros(6, 1, 128, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="go together"):
        kv.beam_reorder(desc, p, n, t, n.clone(), t.clone(), partial_k=k)
    with pytest.raises(ValueError, match="block_table_out"):
        kv.beam_reorder(desc, p, n, t, n.clone(), t[:, :1].contiguous())
    with pytest.raises(kv.KvarnError):  # the lengths cannot be moved in place
        kv.beam_reorder(desc, p, n, t, n, t.clone())


def test_select_rows_past_32_bits(kv):
    # the last rows of the logits start past 2^31 elements
    batch, beams, vocab = 34, 32, 2_000_003
    logits = torch.zeros(batch, beams, vocab, dtype=torch.float16, device="cuda")
    logits[-1, -1, -1] = 9.0
    logits[-1, 0, 7] = 8.0
    scores = torch.zeros(batch, beams, device="cuda")
    (s, p, t, _), _ = select(kv, logits, scores, 2)
    assert p[-1].tolist() == [31, 0] and t[-1].tolist() == [vocab - 1, 7]
    assert p[0].tolist() == [0, 0] and t[0].tolist() == [0, 1]
    assert abs(s[-1, 0] - (9 - math.log(vocab - 1 + math.exp(9)))) < 1e-5 + 2 ** -24 * 9
    del logits
    torch.cuda.empty_cache()


# ---- reordering ------------------------------------------------------------------------------


def state(rows, layers, hkv, d0, width, seed):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, width * 128 + 128, (rows,), generator=g, dtype=torch.int32)
    lens[0], lens[-1] = 128, 127
    table = torch.randint(-5, 10**6, (rows, width), generator=g, dtype=torch.int32)
    shape = (layers, rows, hkv, 128, d0) if layers else (rows, hkv, 128, d0)
    k, v = (torch.randint(0, 30000, shape, generator=g, dtype=torch.int16).view(torch.float16) for _ in range(2))
    return lens, table, k, v


def reordered(parents, lens, table, k, v, lens_o, table_o, k_o, v_o, beams):
    lens_o, table_o, k_o, v_o = (t.clone() for t in (lens_o, table_o, k_o, v_o))
    for j, of in enumerate(parents.flatten().tolist()):
        if not 0 <= of < beams:
            lens_o[j] = 0
            continue
        src = j // beams * beams + of
        n = int(lens[src])
        lens_o[j] = n
        if n > 0:
            table_o[j, :n // 128] = table[src, :n // 128]
            for o, i in ((k_o, k), (v_o, v)):
                o[..., j, :, :n % 128, :] = i[..., src, :, :n % 128, :]
    return lens_o, table_o, k_o, v_o


def same(a, b):
    return torch.equal(a.cpu().view(torch.int16) if a.dtype == torch.float16 else a.cpu(),
                       b.view(torch.int16) if b.dtype == torch.float16 else b)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("batch,beams,layers,hkv,d0,width", [
    (1, 1, 0, 1, 64, 1), (1, 2, 1, 1, 40, 1), (2, 4, 2, 3, 128, 300), (3, 5, 1, 2, 80, 7), (1, 8, 3, 8, 96, 5),
    (2, 9, 1, 1, 256, 4), (1, 16, 0, 4, 64, 9), (5, 17, 1, 2, 200, 3), (1, 32, 2, 1, 256, 1100)])
def test_reorder(kv, batch, beams, layers, hkv, d0, width, in_place):
    rows = batch * beams
    lens, table, k, v = state(rows, layers, hkv, d0, width, rows)
    g = torch.Generator().manual_seed(77)
    parents = torch.randint(-1, beams, (batch, beams), generator=g, dtype=torch.int32)
    parents[0, 0] = beams - 1
    if beams > 4:
        parents[0, :3] = torch.tensor([1, 2, 0])  # a cycle
    desc = kv.desc_from_preset(d0, hkv)
    src = [t.cuda() for t in (lens, table, k, v)]
    if in_place:
        dst = [torch.full_like(src[0], -3)] + src[1:]
    else:
        dst = [torch.full_like(t, -3) for t in src]
    want = reordered(parents, lens, table, k, v, *(t.cpu() for t in dst), beams)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.beam_reorder(desc, parents.cuda(), src[0], src[1], dst[0], dst[1], src[2], src[3], dst[2], dst[3], status=status)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(dst, want)) and status.item() == 0


def test_reorder_without_tiles_and_bad_parents(kv):
    lens, table, k, v = state(6, 1, 1, 64, 5, 3)
    lens[1], lens[4] = -7, 5 * 128 + 128
    parents = torch.tensor([[1, 3, 0], [-2, 1, 2**31 - 1]], dtype=torch.int32)
    desc = kv.desc_from_preset(64, 1)
    for tiles in (False, True):
        src = [t.cuda() for t in (lens, table, k, v)]
        dst = [torch.full_like(t, -3) for t in src]
        want = reordered(parents, lens, table, k, v, *(t.cpu() for t in dst), 3)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(partial_k=src[2], partial_v=src[3], partial_k_out=dst[2], partial_v_out=dst[3]) if tiles else {}
        kv.beam_reorder(desc, parents.cuda(), src[0], src[1], dst[0], dst[1], status=status, **kw)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in list(zip(dst, want))[:4 if tiles else 2])
        assert status.item() == kv.DEV_BAD_BEAM | kv.DEV_SEQ_TOO_LONG


def test_reorder_captured(kv):
    lens, table, k, v = state(8, 2, 2, 128, 20, 9)
    parents = torch.tensor([[1, 0, 0, 2], [3, 2, 1, 0]], dtype=torch.int32)
    desc = kv.desc_from_preset(128, 2)
    src = [t.cuda() for t in (lens, table, k, v)]
    dst = [torch.full_like(t, -3) for t in src]
    want = reordered(parents, lens, table, k, v, *(t.cpu() for t in dst), 4)
    p = parents.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.beam_reorder(desc, p, src[0], src[1], dst[0], dst[1], src[2], src[3], dst[2], dst[3])
    for _ in range(2):
        for t in dst:
            t.fill_(-3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(dst, want))


def test_beam_search_over_the_packed_cache(kv):
    """A search of a small model whose state is the cache: plan, append, decode, select, reorder, the tiles sealed
    and their pages shared on the way, against a search that keeps every hypothesis whole."""
    hkv, d0, hq, beams, vocab, steps, prompt = 1, 64, 2, 3, 50, 9, 250
    desc = kv.desc_from_preset(d0, hkv)
    g = torch.Generator().manual_seed(12)
    emb_k, emb_v, emb_q = (torch.randn(vocab, n, d0, generator=g).half().cuda() for n in (hkv, hkv, hq))
    head = (0.3 * torch.randn(vocab, hq * d0, generator=g)).cuda()
    tokens = torch.randint(0, vocab, (prompt,), generator=g).tolist()
    scale, groups = 0.125, 2
    rows, width, pages = groups * beams, 4, 40
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    class Cache:
        def __init__(self, rows):
            self.pool = kv.alloc_pool(desc, pages)
            self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
            self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
            self.pk = torch.zeros(rows, hkv, 128, d0, dtype=torch.float16, device="cuda")
            self.pv = torch.zeros_like(self.pk)
            self.ws = kv.alloc_workspace(desc, rows, hq, width)
            self.rows = rows

        def step(self, toks):
            """Append a token a row and attend from it: logits [rows, vocab]."""
            planned, after = torch.empty_like(self.lens), torch.empty_like(self.lens)
            kv.plan_pages(self.lens, self.table, pages, planned, status=status)
            kv.append_token(desc, emb_k[toks], emb_v[toks], self.pk, self.pv, self.lens, self.table, self.pool,
                            seq_lens_out=after, status=status)
            out = torch.empty(self.rows, hq, d0, dtype=torch.float16, device="cuda")
            kv.decode_attention(desc, emb_q[toks], self.pool, self.table, after, out, self.ws, partial_k=self.pk,
                                partial_v=self.pv, softmax_scale=scale, status=status)
            assert torch.equal(planned, after)
            self.lens = after
            return out.float().flatten(1) @ head.T

    # the cache under test, all beams of a group started from one prompt
    cache = Cache(rows)
    for t in tokens[:-1]:
        logits = cache.step(torch.full((rows,), t, device="cuda"))
        if int(cache.lens[0]) % 128 == 0:  # the beams of all groups hold the same page from here on
            cache.table[:, int(cache.lens[0]) // 128 - 1] = cache.table[0, int(cache.lens[0]) // 128 - 1]
    last = torch.full((rows,), tokens[-1], device="cuda")
    scores = torch.full((groups, beams), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros(groups, beams, dtype=torch.bool, device="cuda")
    history = torch.zeros(rows, 0, dtype=torch.int64, device="cuda")
    bufs = [torch.zeros(groups, beams, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32, torch.bool)]
    ws = kv.alloc_beam_select_workspace(groups, beams, vocab, beams)
    end = 3
    for _ in range(steps):
        logits = cache.step(last).view(groups, beams, vocab)
        kv.beam_select(logits, scores, bufs[0], bufs[1], bufs[2], ws, done=done, end_token=end, out_done=bufs[3], status=status)
        scores, done = bufs[0].clone(), bufs[3].clone()
        lens = torch.empty_like(cache.lens)
        kv.beam_reorder(desc, bufs[1], cache.lens, cache.table, lens, cache.table, cache.pk, cache.pv, cache.pk, cache.pv,
                        status=status)
        cache.lens = lens
        flat = (torch.arange(groups, device="cuda")[:, None] * beams + bufs[1]).flatten().long()
        last = bufs[2].flatten().long()
        history = torch.cat([history[flat], last[:, None]], 1)
    assert status.item() == 0

    # one hypothesis a row, replayed whole through a cache of its own; the scores have to agree
    plain = Cache(rows)
    for t in tokens[:-1]:
        plain.step(torch.full((rows,), t, device="cuda"))
    total, live = torch.zeros(rows, dtype=torch.float64, device="cuda"), torch.ones(rows, dtype=torch.bool, device="cuda")
    last = torch.full((rows,), tokens[-1], device="cuda")
    for j in range(steps):
        logp = torch.log_softmax(plain.step(last).double(), 1)
        last = history[:, j]
        total += torch.where(live, logp.gather(1, last[:, None])[:, 0], 0.0)
        live &= last != end
    # the decode of equal caches is equal to a rounding of fp16 (page ids differ, splits do not): 9 steps of the
    # head's 128 products, each off by at most 2^-11 of about one, stay below 1e-2
    assert (scores.flatten().double() - total).abs().max() < 1e-2
    assert torch.equal(live, ~done.flatten()) and status.item() == 0
    for b in range(groups):
        s = scores[b].tolist()
        assert s == sorted(s, reverse=True) and len({tuple(h) for h in history[b * beams:(b + 1) * beams].tolist()}) == beams
