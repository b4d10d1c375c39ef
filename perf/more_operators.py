"""Pages planned on the GPU and beam search over the paged cache: the measured calls.

Four operators around the decode step of a paged KV cache (128-token pages, a block table per
sequence):

  plan     block tables grown by the pages that the coming tokens need, taken from those no
           sequence names, and the slot of every coming token;
  store    the keys and values of new tokens written to their slots of the fp16 paged cache;
  select   the best continuations over beams and vocabulary, from logits and running scores;
  reorder  the cache's state moved to the beams that go on: lengths, table rows, open tiles.

`run` computes them in elementary torch operations; with `own` set it calls the library.
"""

import math

import torch

own = False

TILE = 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------


def _plan(name, batch, chunk, lo, hi, pool, packed, ragged=False, shared=1):
    return {"name": name, "op": "plan", "batch": batch, "chunk": chunk, "lo": lo, "hi": hi, "pool": pool,
            "packed": packed, "ragged": ragged, "shared": shared}


def _store(name, batch, chunk, kv_heads, dim, ragged=False, fused=False):
    return {"name": name, "op": "store", "batch": batch, "chunk": chunk, "kv_heads": kv_heads, "dim": dim,
            "ragged": ragged, "fused": fused}


def _select(name, batch, beams, vocab, count, dtype, pad=0, done=False):
    return {"name": name, "op": "select", "batch": batch, "beams": beams, "vocab": vocab, "count": count,
            "dtype": dtype, "pad": pad, "done": done}


def _reorder(name, batch, beams, layers, kv_heads, dim, lo, hi):
    return {"name": name, "op": "reorder", "batch": batch, "beams": beams, "layers": layers, "kv_heads": kv_heads,
            "dim": dim, "lo": lo, "hi": hi}


def listed():
    return [
        # one user's decode step: the latency of the smallest call
        _plan("plan 1x1", 1, 1, 5000, 5000, 512, True),
        # a decode step of a large serving batch, four beams to a shared prompt, pool of a many-layer model
        _plan("plan 512x1 of 16k", 512, 1, 2000, 16384, 60000, True, shared=4),
        # a prefill step of ragged chunks into the fp16 cache, which takes the slots
        _plan("plan 32x512 ragged", 32, 512, 0, 8000, 20000, False, ragged=True),
        # one decode step of a serving batch into the fp16 cache
        _store("store 64x1", 64, 1, 8, 128),
        # ragged prompts, keys and values as slices of one fused projection
        _store("store 16x1024 ragged fused", 16, 1024, 8, 128, ragged=True, fused=True),
        # one user, four beams, a small vocabulary: the smallest step
        _select("select 1x4 of 32000", 1, 4, 32000, 8, "bf16"),
        # a batch of a few beams over 32-bit logits, an odd vocabulary, some beams finished
        _select("select 8x5 of 50001 fp32", 8, 5, 50001, 10, "fp32", done=True),
        # the usual serving size: a padded vocabulary, twice as many candidates as beams
        _select("select 32x4 of 128000 padded", 32, 4, 128000, 8, "fp16", pad=256, done=True),
        # the largest: bound by the bytes of the logits
        _select("select 64x8 of 151936", 64, 8, 151936, 16, "bf16"),
        # one user's four beams, one layer: the smallest step
        _reorder("reorder 1x4 1 layer", 1, 4, 1, 8, 128, 1000, 1000),
        # odd lengths, head_dim 64, more beams than a power of two
        _reorder("reorder 6x5 4 layers d64", 6, 5, 4, 4, 64, 300, 9000),
        # all layers of a stack at once: bound by the bytes of the open tiles
        _reorder("reorder 16x4 16 layers", 16, 4, 16, 8, 128, 2000, 16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "select", "reorder"])
    if op == "plan":
        chunk = rng.choice([1, 1, _log(rng, 2, 2048)])
        batch = _log(rng, 1, 1024)
        batch = max(1, min(batch, 65536 // chunk))
        hi = _log(rng, 100, 32768)
        hi = max(100, min(hi, 128 * (1 << 19) // batch))
        shared = rng.choice([1, 1, 4, 8])
        pages = batch * (-(-hi // TILE) + -(-chunk // TILE) + 1)
        pool = int(pages * rng.uniform(1.0, 3.0)) + rng.randint(1, 2000)
        if rng.random() < 0.15:  # a pool that runs out
            pool = pages // 2 + 8
        return {"op": op, "batch": batch, "chunk": chunk, "lo": rng.randint(0, hi), "hi": hi, "pool": pool,
                "packed": rng.random() < 0.5, "ragged": rng.random() < 0.5, "shared": shared}
    if op == "store":
        chunk = rng.choice([1, _log(rng, 2, 2000)])
        batch = max(1, min(_log(rng, 1, 256), 16384 // chunk))
        return {"op": op, "batch": batch, "chunk": chunk, "kv_heads": rng.choice([1, 2, 4, 8]),
                "dim": rng.choice([64, 128, 128]), "ragged": rng.random() < 0.5, "fused": rng.random() < 0.5}
    if op == "select":
        beams = rng.randint(1, 12)
        vocab = _log(rng, 500, 200000)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        batch = _log(rng, 1, 64)
        size = 4 if dtype == "fp32" else 2
        batch = max(1, min(batch, 150000000 // (beams * vocab * size)))
        return {"op": op, "batch": batch, "beams": beams, "vocab": vocab, "count": rng.choice([beams, 2 * beams, 2 * beams]),
                "dtype": dtype, "pad": rng.choice([0, 0, -vocab % 64]), "done": rng.random() < 0.5}
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    kv_heads, beams, layers = rng.choice([1, 2, 4, 8]), rng.randint(2, 12), rng.choice([1, 1, 2, 4, 8, 16])
    batch = _log(rng, 1, 32)
    batch = max(1, min(batch, (1 << 27) // (TILE * dim * kv_heads * beams * layers)))
    hi = _log(rng, 100, 16384)
    return {"op": op, "batch": batch, "beams": beams, "layers": layers, "kv_heads": kv_heads, "dim": dim,
            "lo": rng.randint(1, hi), "hi": hi}


def _lens(n, lo, hi):
    """Tokens of each of n sequences: spread over [lo, hi], odd remainders among them."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((7 * b + 3) % n) // (n - 1) for b in range(n)]


def _new_lens(case):
    """Coming tokens of each sequence: the whole chunk, or fewer in a ragged batch."""
    n, chunk = case["batch"], case["chunk"]
    return [chunk - (37 * b) % chunk if case["ragged"] else chunk for b in range(n)]


def _pages(length, packed):
    return length // TILE if packed else -(-length // TILE)


def work(case):
    if case["op"] == "plan":
        lens, new = _lens(case["batch"], case["lo"], case["hi"]), _new_lens(case)
        held = [_pages(n, case["packed"]) for n in lens]
        need = [_pages(n + m, case["packed"]) - h for n, m, h in zip(lens, new, held)]
        return {"bytes": 4 * sum(held) + 4 * sum(need) + 12 * case["batch"] + 8 * case["batch"] * case["chunk"],
                "flops": sum(held) + sum(need)}
    if case["op"] == "store":
        tokens = sum(_new_lens(case))
        return {"bytes": 8 * tokens * case["kv_heads"] * case["dim"] + 8 * case["batch"] * case["chunk"], "flops": 0}
    if case["op"] == "select":
        rows, size = case["batch"] * case["beams"], 4 if case["dtype"] == "fp32" else 2
        return {"bytes": rows * (case["vocab"] * size + 5) + 13 * case["batch"] * case["count"],
                "flops": 4 * rows * case["vocab"]}
    rows = _lens(case["batch"], case["lo"], case["hi"])
    # live rows of the open tiles: each beam's written, the parents' read (about 0.7 of the beams are one)
    tail = sum(n % TILE for n in rows) * case["kv_heads"] * case["dim"] * 2 * 2 * case["layers"]
    parents = case["beams"] * (1 - (1 - 1 / case["beams"]) ** case["beams"])
    sealed = sum(n // TILE for n in rows)
    return {"bytes": int((tail + 4 * sealed) * (case["beams"] + parents)) + 12 * case["batch"] * case["beams"], "flops": 0}


# ---- inputs --------------------------------------------------------------------------------


def _prepare_plan(case, gen, dev):
    n, shared = case["batch"], case["shared"]
    lens = torch.tensor(_lens(n, case["lo"], case["hi"]), dtype=torch.int64)
    new = torch.tensor(_new_lens(case), dtype=torch.int64)
    # sequences of another seed are other ones
    lens = (lens - torch.randint(0, 64, (n,), generator=gen, device=dev).cpu()).clamp(min=case["lo"])
    if shared > 1:  # sequences of a group have the same length and the first half of their pages in common
        lens = lens[torch.arange(n) // shared * shared]
    held = _pages(lens, case["packed"])
    width = -(-(case["hi"] + case["chunk"]) // TILE)
    group = torch.arange(n) // shared * shared
    col = torch.arange(width)
    owner = torch.where(col < (held // 2).unsqueeze(1), group.unsqueeze(1), torch.arange(n).unsqueeze(1))
    flat = owner * width + col
    live = col < held.unsqueeze(1)
    named, index = torch.unique(flat[live], return_inverse=True)
    perm = torch.randperm(max(case["pool"], named.numel()), generator=gen, device=dev).cpu()
    perm = perm[perm < case["pool"]] if named.numel() <= case["pool"] else perm % case["pool"]
    table = torch.full((n, width), -1, dtype=torch.int64)
    table[live] = perm[index]
    return {"lens": lens.int().to(dev), "new": new.int().to(dev), "table": table.int().to(dev),
            "lens_out": torch.zeros(n, dtype=torch.int32, device=dev),
            "slots": torch.zeros(n, case["chunk"], dtype=torch.int64, device=dev)}


def _prepare_store(case, gen, dev):
    n, chunk, heads, dim = (case[k] for k in ("batch", "chunk", "kv_heads", "dim"))
    width = -(-chunk // TILE) + 1
    pages = n * width
    table = torch.randperm(pages, generator=gen, device=dev).reshape(n, width)
    first = torch.randint(0, TILE, (n, 1), generator=gen, device=dev)
    at = first + torch.arange(chunk, device=dev)
    slots = table.gather(1, at // TILE) * TILE + at % TILE
    new = torch.tensor(_new_lens(case), device=dev).unsqueeze(1)
    slots = torch.where(torch.arange(chunk, device=dev) < new, slots, -1)
    if case["fused"]:  # queries, keys and values of a token side by side
        qkv = torch.randn(n * chunk, 6, heads, dim, generator=gen, device=dev).half()
        k, v = qkv[:, 4], qkv[:, 5]
    else:
        k, v = (torch.randn(n * chunk, heads, dim, generator=gen, device=dev).half() for _ in range(2))
    # one page more than the cache has: the plain form's place for tokens without a slot
    pool = torch.zeros(pages + 1, heads, 2, TILE, dim, dtype=torch.float16, device=dev)
    return {"k": k, "v": v, "slots": slots.flatten(), "pool": pool}


def _prepare_select(case, gen, dev):
    n, beams, vocab = case["batch"], case["beams"], case["vocab"]
    # next-token logits: a broad bulk, a few likely tokens that the beams of a group largely share
    bulk = 2.0 * torch.randn(n, beams, vocab + case["pad"], generator=gen, device=dev)
    top = min(64, vocab)
    likely = torch.randint(0, vocab // top, (n, 1, top), generator=gen, device=dev).expand(-1, beams, -1)
    likely = likely + torch.arange(top, device=dev) * (vocab // top)
    lift = 8.0 + 3.0 * torch.randn(n, 1, top, generator=gen, device=dev) + torch.randn(n, beams, top, generator=gen, device=dev)
    logits = bulk.scatter_add(2, likely, lift)
    logits[..., vocab:] = 1e4  # columns past the vocabulary hold anything
    logits = logits.to(TYPES[case["dtype"]])[..., :vocab]
    scores = -20.0 - 6.0 * torch.rand(n, beams, generator=gen, device=dev)
    done = torch.rand(n, beams, generator=gen, device=dev) < (0.25 if case["done"] else 0.0)
    s = {"logits": logits, "scores": scores, "done": done, "end": vocab - 1}
    for name, dtype in (("out_scores", torch.float32), ("parents", torch.int32), ("tokens", torch.int32), ("out_done", torch.bool)):
        s[name] = torch.zeros(n, case["count"], dtype=dtype, device=dev)
    return s


def _prepare_reorder(case, gen, dev):
    n, beams = case["batch"], case["beams"]
    rows = n * beams
    lens = torch.tensor(_lens(n, case["lo"], case["hi"]), device=dev).repeat_interleave(beams)
    width = max(1, -(-case["hi"] // TILE))
    own_pages = torch.randperm(rows * width, generator=gen, device=dev).reshape(n, beams, width)
    prompt = torch.arange(width, device=dev) < (width + 1) // 2
    table = torch.where(prompt, own_pages[:, :1], own_pages).reshape(rows, width)
    # a beam goes on from itself or from a better one
    parents = torch.randint(0, beams, (n, beams), generator=gen, device=dev)
    shape = (case["layers"], rows, case["kv_heads"], TILE, case["dim"])
    s = {"parents": parents.int(), "lens": lens.int(), "table": table.int(),
         "lens_out": torch.zeros(rows, dtype=torch.int32, device=dev),
         "table_out": torch.full((rows, width), -1, dtype=torch.int32, device=dev)}
    for name in ("k", "v"):
        s[name] = torch.randn(shape, generator=gen, device=dev, dtype=torch.float16)
        s[name + "_out"] = torch.zeros(shape, dtype=torch.float16, device=dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    make = {"plan": _prepare_plan, "store": _prepare_store, "select": _prepare_select, "reorder": _prepare_reorder}
    s = make[case["op"]](case, gen, dev)
    s["case"] = dict(case)
    if own and case["op"] == "select":
        from calibration_free_kv_gb300 import kvarn
        s["workspace"] = kvarn.alloc_beam_select_workspace(case["batch"], case["beams"], case["vocab"], case["count"])
    if own and case["op"] == "reorder":
        from calibration_free_kv_gb300 import kvarn
        s["desc"] = kvarn.desc_from_preset(case["dim"], case["kv_heads"])
    return s


# ---- the plain forms -----------------------------------------------------------------------


def _plain_plan(s):
    case, dev = s["case"], s["lens"].device
    lens, new, table, pool = s["lens"].long(), s["new"].long(), s["table"].long(), case["pool"]
    held, after = _pages(lens, case["packed"]), _pages(lens + new, case["packed"])
    need = after - held
    col = torch.arange(table.shape[1], device=dev)
    free = torch.ones(pool + 1, dtype=torch.int64, device=dev)
    free[torch.where(col < held.unsqueeze(1), table, pool)] = 0
    free = free[:pool].cumsum(0)
    end = need.cumsum(0)
    served = (need == 0) | (end <= free[-1])
    rank = (end - need).unsqueeze(1) + col - held.unsqueeze(1)
    fresh = (col >= held.unsqueeze(1)) & (col < after.unsqueeze(1)) & served.unsqueeze(1)
    table = torch.where(fresh, torch.searchsorted(free, rank.clamp(min=0) + 1), table)
    i = torch.arange(case["chunk"], device=dev)
    at = lens.unsqueeze(1) + i
    page = at // TILE
    on = served.unsqueeze(1) & (i < new.unsqueeze(1)) & (page < after.unsqueeze(1))
    slot = table.gather(1, page.clamp(max=table.shape[1] - 1)) * TILE + at % TILE
    return {"table": table.int(), "lens": torch.where(served, lens + new, lens).int(), "slots": torch.where(on, slot, -1)}


def _plain_store(s):
    pool, slots = s["pool"], s["slots"]
    at = torch.where(slots >= 0, slots, (pool.shape[0] - 1) * TILE)
    page, row = at // TILE, at % TILE
    pool[page, :, 0, row] = s["k"]
    pool[page, :, 1, row] = s["v"]
    return pool[:-1]


def _plain_select(s):
    case = s["case"]
    # 64 bits: candidates of two beams may be as near as the rounding of a 32-bit sum
    x, scores = s["logits"].double(), s["scores"].double().unsqueeze(2)
    top = x.amax(2, keepdim=True)
    x = x - top
    x = x - torch.log(torch.exp(x).sum(2, keepdim=True)) + scores
    ends = torch.arange(case["vocab"], device=x.device) == s["end"]
    x = torch.where(s["done"].unsqueeze(2), torch.where(ends, scores, -math.inf), x)
    best, at = torch.sort(x.flatten(1), dim=1, descending=True, stable=True)
    best, at = best[:, :case["count"]], at[:, :case["count"]]
    none = best == -math.inf
    parent = torch.where(none, -1, at // case["vocab"])
    token = torch.where(none, -1, at % case["vocab"])
    done = (s["done"].gather(1, parent.clamp(min=0)) | (token == s["end"])) & ~none
    return {"scores": best.float(), "parents": parent.int(), "tokens": token.int(), "done": done}


def _plain_reorder(s):
    case = s["case"]
    dev, beams, lens = s["lens"].device, case["beams"], s["lens"].long()
    rows = torch.arange(lens.numel(), device=dev)
    source = rows // beams * beams + s["parents"].flatten().long()
    lens = lens[source]
    col = torch.arange(s["table"].shape[1], device=dev)
    table = torch.where(col < (lens // TILE).unsqueeze(1), s["table"][source], s["table_out"])
    live = (torch.arange(TILE, device=dev) < (lens % TILE).unsqueeze(1))[None, :, None, :, None]
    k, v = (torch.where(live, s[x][:, source], s[x + "_out"]) for x in ("k", "v"))
    return {"lens": lens.int(), "table": table, "k": k, "v": v}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "store": _plain_store, "select": _plain_select, "reorder": _plain_reorder}[op](s)
    from calibration_free_kv_gb300 import kvarn
    if op == "plan":
        kvarn.plan_pages(s["lens"], s["table"], s["case"]["pool"], s["lens_out"], new_lens=s["new"],
                         chunk_len=s["case"]["chunk"], slot_map=s["slots"], open_tiles=s["case"]["packed"])
        return {"table": s["table"], "lens": s["lens_out"], "slots": s["slots"]}
    if op == "store":
        pool = s["pool"][:-1]
        kvarn.fp16_store(s["k"], s["v"], s["slots"], pool)
        return pool
    if op == "select":
        kvarn.beam_select(s["logits"], s["scores"], s["out_scores"], s["parents"], s["tokens"], s["workspace"],
                          done=s["done"], end_token=s["end"], out_done=s["out_done"])
        return {"scores": s["out_scores"], "parents": s["parents"], "tokens": s["tokens"], "done": s["out_done"]}
    kvarn.beam_reorder(s["desc"], s["parents"], s["lens"], s["table"], s["lens_out"], s["table_out"],
                       s["k"], s["v"], s["k_out"], s["v_out"])
    return {"lens": s["lens_out"], "table": s["table_out"], "k": s["k_out"], "v": s["v_out"]}


# ---- the definition ------------------------------------------------------------------------


def _exact_plan(case, s):
    """Request by request, page by page."""
    pool = case["pool"]
    table, lens, new = s["table"].tolist(), s["lens"].tolist(), s["new"].tolist()
    held = [_pages(n, case["packed"]) for n in lens]
    named = {p for row, h in zip(table, held) for p in row[:h]}
    free = [p for p in range(pool) if p not in named]
    taken, wanted, lens_out, slots = 0, 0, [], []
    for b, (row, h) in enumerate(zip(table, held)):
        need = _pages(lens[b] + new[b], case["packed"]) - h
        wanted += need
        fits = need == 0 or wanted <= len(free)
        if fits and need:
            row[h:h + need] = free[taken:taken + need]
            taken += need
        lens_out.append(lens[b] + new[b] if fits else lens[b])
        at = [lens[b] + i for i in range(new[b])] if fits else []
        line = [row[p // TILE] * TILE + p % TILE if p // TILE < h + need else -1 for p in at]
        slots.append(line + [-1] * (case["chunk"] - len(line)))
    dev = s["lens"].device
    return {"table": torch.tensor(table, dtype=torch.int32, device=dev), "lens": torch.tensor(lens_out, dtype=torch.int32, device=dev),
            "slots": torch.tensor(slots, device=dev)}


def _exact_store(s):
    pool = s["pool"].double()[:-1]
    lines = pool.transpose(1, 3).reshape(-1, 2, pool.shape[1], pool.shape[4])  # [slot][key or value][head][channel]
    on = s["slots"] >= 0
    lines[s["slots"][on]] = torch.stack([s["k"], s["v"]], 1)[on].double()
    return lines.reshape(pool.shape[0], TILE, 2, pool.shape[1], pool.shape[4]).transpose(1, 3).contiguous()


def _exact_select(case, s):
    """Group by group: every candidate's score, the best one taken `count` times."""
    out = {"scores": [], "parents": [], "tokens": [], "done": []}
    for b in range(case["batch"]):
        score = torch.log_softmax(s["logits"][b].double(), 1) + s["scores"][b].double().unsqueeze(1)
        for k in range(case["beams"]):
            if s["done"][b, k]:
                score[k] = -math.inf
                score[k, s["end"]] = s["scores"][b, k].double()
        # the best of each beam are among its `count` greatest; equal ones are all kept
        floor = torch.topk(score.flatten(), min(case["count"], score.numel())).values[-1]
        k, v = (t.tolist() for t in torch.nonzero((score >= floor) & (score > -math.inf), as_tuple=True))
        value = score[k, v].tolist()
        order = sorted(range(len(k)), key=lambda i: (-value[i], k[i], v[i]))[:case["count"]]
        fill = case["count"] - len(order)
        out["scores"].append([value[i] for i in order] + [-math.inf] * fill)
        out["parents"].append([k[i] for i in order] + [-1] * fill)
        out["tokens"].append([v[i] for i in order] + [-1] * fill)
        done = s["done"][b].tolist()
        out["done"].append([done[k[i]] or v[i] == s["end"] for i in order] + [False] * fill)
    dev = s["scores"].device
    kinds = {"scores": torch.float64, "parents": torch.int32, "tokens": torch.int32, "done": torch.bool}
    return {name: torch.tensor(rows, dtype=kinds[name], device=dev) for name, rows in out.items()}


def _exact_reorder(case, s):
    lens, parents = s["lens"].tolist(), s["parents"].tolist()
    out = {"lens": s["lens_out"].clone(), "table": s["table_out"].clone(), "k": s["k_out"].double(), "v": s["v_out"].double()}
    for b in range(case["batch"]):
        for j in range(case["beams"]):
            to, of = b * case["beams"] + j, b * case["beams"] + parents[b][j]
            out["lens"][to] = lens[of]
            out["table"][to, :lens[of] // TILE] = s["table"][of, :lens[of] // TILE]
            for x in ("k", "v"):
                out[x][:, to, :, :lens[of] % TILE] = s[x][:, of, :, :lens[of] % TILE].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(case, s)
    if case["op"] == "store":
        return _exact_store(s)
    return (_exact_select if case["op"] == "select" else _exact_reorder)(case, s)
