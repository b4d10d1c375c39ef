"""Speculative and windowed attention over the packed KV cache: the measured calls.

Three operators read the same paged cache (128-token page records of 2-, 4- or 8-bit codes, a
block table per sequence, the raw fp16 rows of each sequence's open tile):

  tree            the drafted tokens of a tree attend to the cached tokens and to their own
                  ancestors among the drafted ones (one bit mask row per node);
  window_decode   one new token per sequence attends to the first `sink` cached tokens and to the
                  last `window` tokens (its own included);
  window_prefill  a chunk of new tokens does the same, causally.

`run` computes them in elementary torch operations, in 32 bits, from the same records; with
`own` set it calls the library.
"""

import math

import torch

own = False

TILE = 128


# ---- cases ---------------------------------------------------------------------------------


def _tree(name, batch, nodes, heads, kv_heads, dim, lo, hi, bits="4,2", ragged=False):
    return {"name": name, "op": "tree", "batch": batch, "new": nodes, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "lo": lo, "hi": hi, "bits": bits, "ragged": ragged}


def _window(name, op, batch, new, heads, kv_heads, dim, lo, hi, sink, window, bits="4,2"):
    return {"name": name, "op": op, "batch": batch, "new": new, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "lo": lo, "hi": hi, "sink": sink, "window": window, "bits": bits, "ragged": False}


def listed():
    return [
        # one user, a short draft over a short context: the latency of a single request
        _tree("tree 1x8 over 1k", 1, 8, 32, 8, 128, 1000, 1000),
        # a serving batch at mixed lengths, the usual draft size; trees of fewer nodes are padded
        _tree("tree 16x26 over 2-16k", 16, 26, 32, 8, 128, 2000, 16384, ragged=True),
        # full 64-node trees over long contexts: the largest verification step
        _tree("tree 16x64 over 16k", 16, 64, 32, 8, 128, 15000, 16500),
        # a 64-layer 32B-class layer's heads (GQA 8), a chain-like draft of five tokens
        _tree("tree 32x5 over 8k gqa8", 32, 5, 64, 8, 128, 4100, 12300),
        # other widths of the packed format: head_dim 64 with 8-bit keys, no head sharing
        _tree("tree 8x33 d64 k8v4 mha", 8, 33, 8, 8, 64, 700, 9000, bits="8,4", ragged=True),
        # one user, a small window: the smallest step
        _window("window decode 1 of 1k", "window_decode", 1, 1, 32, 8, 128, 5000, 5000, 4, 1024),
        # a serving batch with a 4096-token window and four visible first tokens
        _window("window decode 64 of 4k", "window_decode", 64, 1, 32, 8, 128, 1000, 16384, 4, 4096),
        # a large batch with long windows: bound by the bytes of the visible pages
        _window("window decode 128 of 16k", "window_decode", 128, 1, 32, 8, 128, 16000, 40000, 64, 16384),
        # head_dim 256 and 4-bit values, a window that is no multiple of a page
        _window("window decode 16 d256 k4v4", "window_decode", 16, 1, 16, 4, 256, 3000, 20000, 130, 5000, bits="4,4"),
        # a short continuation chunk of one user
        _window("window prefill 1x17 of 1k", "window_prefill", 1, 17, 32, 8, 128, 3000, 3000, 4, 1024),
        # chunked prefill of a batch, chunks of 256
        _window("window prefill 8x256 of 4k", "window_prefill", 8, 256, 32, 8, 128, 2500, 14000, 4, 4096),
        # one long prompt's chunk: the largest prefill step, its causal part as long as the window's
        _window("window prefill 2x2048 of 4k", "window_prefill", 2, 2048, 32, 8, 128, 9000, 12000, 4, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _bounded(case):
    """The case with its batch, then its new tokens, halved until it costs less than the largest listed one."""
    while work(case)["flops"] > 2.5e11 or work(case)["bytes"] > 1.7e9:
        which = "batch" if case["batch"] > 1 else "new"
        case[which] //= 2
    return case


def draw(rng):
    op = rng.choice(["tree", "window_decode", "window_prefill"])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 4] if dim == 256 else [1, 2, 4, 4, 8])
    bits = rng.choice(["4,2", "4,2", "4,4", "2,2", "8,4"])
    if op == "tree":
        new = _log(rng, 1, 64)
        top = _log(rng, 200, 16384)
        batch = _log(rng, 1, 32)
        case = {"op": op, "batch": batch, "new": new, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                "lo": max(1, int(top * rng.uniform(0.1, 1.0))), "hi": top, "bits": bits, "ragged": rng.random() < 0.5}
        return _bounded(case)
    window = _log(rng, 100, 8192)
    sink = rng.choice([0, 1, 4, 64, 128, 200])
    top = _log(rng, 200, 32768)
    if op == "window_decode":
        new, batch = 1, _log(rng, 1, 64)
    else:
        new, batch = _log(rng, 2, 1500), _log(rng, 1, 16)
    return _bounded({"op": op, "batch": batch, "new": new, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                     "lo": max(1, int(top * rng.uniform(0.1, 1.0))), "hi": top, "sink": sink, "window": window, "bits": bits,
                     "ragged": False})


def _lens(case):
    """Cached tokens of each sequence: spread over [lo, hi], odd remainders among them."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((7 * b + 3) % n) // (n - 1) for b in range(n)]


def _new_lens(case):
    """Drafted nodes of each sequence: all of them, or fewer in a ragged batch."""
    n, new = case["batch"], case["new"]
    return [max(1, new - (5 * b) % max(1, new)) if case["ragged"] else new for b in range(n)]


def _padded(dim):
    return 64 if dim <= 64 else (128 if dim <= 128 else 256)


def _visible(case):
    """Per sequence: (cached tokens, (query, key) pairs, sealed pages read, open-tile tokens read)."""
    rows = []
    for length, new in zip(_lens(case), _new_lens(case)):
        if case["op"] == "tree":
            rows.append((length, new * length + new * (new + 1) // 2, length // TILE, length % TILE))
            continue
        sink, window = case["sink"], case["window"]
        # decode: the query is the last of `length` tokens; prefill: it follows them
        first = length - 1 if case["op"] == "window_decode" else length
        total = length if case["op"] == "window_decode" else length + new
        pairs = 0
        for i in range(case["new"]):
            at = first + i
            pairs += min(at + 1, window) + min(sink, max(0, at + 1 - window))
        start = max(0, first + 1 - window)  # the earliest window token of any row
        n = length // TILE
        first_window_page = min(start // TILE, n)
        sink_pages = min(-(-sink // TILE), first_window_page)
        rows.append((total, pairs, n - first_window_page + sink_pages, length % TILE))
    return rows


def work(case):
    kb, vb = (int(x) for x in case["bits"].split(","))
    d, dim = _padded(case["dim"]), case["dim"]
    record = TILE * d * (kb + vb) // 8 + 6 * d + 6 * TILE
    rows = case["batch"] * case["new"]
    nbytes = 2 * rows * case["heads"] * dim * 2  # queries and outputs
    if case["op"] != "window_decode":
        nbytes += 2 * rows * case["kv_heads"] * dim * 2
    if case["op"] == "tree":
        nbytes += rows * -(-case["new"] // 32) * 4
    flops = 0
    for _, pairs, pages, tail in _visible(case):
        nbytes += pages * (record * case["kv_heads"] + 4) + 2 * tail * case["kv_heads"] * dim * 2 + 4
        flops += 4 * dim * pairs * case["heads"]
    return {"bytes": nbytes, "flops": flops}


# ---- the record's code order ---------------------------------------------------------------


def _order(kind, bits, d):
    """Element (row-major [token][channel]) behind each (word, slot) of a half's code words, and
    the bit offset of each slot."""
    per = 32 // bits
    at = torch.empty(TILE * d // per, per, dtype=torch.int64)
    lane = torch.arange(32)
    g, tq = lane // 4, lane % 4
    shifts = torch.arange(per) * bits

    def element(o, i, rho, h, p):  # fragment (o, i): token block o, channel block i
        if kind == "K":
            return (16 * o + g + 8 * rho) * d + 16 * i + 8 * h + 2 * tq + p
        return (16 * o + 8 * h + 2 * tq + p) * d + 16 * i + g + 8 * rho

    for o in range(TILE // 16):
        for i in range(d // 16):
            for rho in range(2):
                for h in range(2):
                    for p in range(2):
                        if bits == 4:
                            word, slot = ((o * (d // 64) + i // 4) * 32 + lane) * 4 + i % 4, h + 2 * rho + 4 * p
                        elif bits == 2:
                            word = ((o // 2 * (d // 64) + i // 4) * 32 + lane) * 4 + i % 4
                            slot = 2 * (o % 2) + h + 4 * rho + 8 * p
                        else:
                            word, slot = ((o * (d // 32) + i // 2) * 32 + lane) * 4 + 2 * (i % 2) + h, rho + 2 * p
                        at[word, slot] = element(o, i, rho, h, p)
    return at.reshape(-1), shifts


def _sections(bits, d):
    kb, vb = bits
    sizes = [TILE * d * kb // 8, 2 * d, 2 * d, 2 * TILE, TILE * d * vb // 8, 2 * TILE, 2 * TILE, 2 * d]
    ends, at = [], 0
    for n in sizes:
        ends.append((at, at + n))
        at += n
    return ends, at


def _pack(codes, order, shifts):
    n = codes.shape[0]
    words = (codes.reshape(n, -1)[:, order].reshape(n, -1, shifts.numel()).long() << shifts).sum(-1)
    return words.to(torch.int64).bitwise_and(0xFFFFFFFF).to(torch.uint32).view(torch.uint8).reshape(n, -1)


def _quantised(gen, tiles, d, kind, bits, dev):
    """Codes, scale, zero and factor of `tiles` rotated, balanced tiles: values near N(0, 1) per
    (token, channel), channel and token factors apart from them."""
    x = torch.randn(tiles, TILE, d, generator=gen, device=dev)
    dim = 1 if kind == "K" else 2  # K: one scale per channel, V: one per token
    lo, hi = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    step = (hi - lo) / (2 ** bits - 1)
    codes = ((x - lo) / step).round().clamp(0, 2 ** bits - 1).to(torch.uint8)
    own_axis = torch.exp(0.3 * torch.randn(step.shape, generator=gen, device=dev))
    factor = torch.exp(0.4 * torch.randn((tiles, TILE if kind == "K" else d), generator=gen, device=dev))
    return codes, (step * own_axis).squeeze(dim).half(), (lo * own_axis).squeeze(dim).half(), factor.half()


def _pool(gen, pages, kv_heads, d, bits, dev):
    """A page pool [pages][kv_heads][record bytes] of random records."""
    kb, vb = bits
    ends, size = _sections(bits, d)
    pool = torch.empty(pages * kv_heads, size, dtype=torch.uint8, device=dev)
    ko, ks = (t.to(dev) for t in _order("K", kb, d))
    vo, vs = (t.to(dev) for t in _order("V", vb, d))
    step = 4096 * 128 // d
    for i in range(0, pages * kv_heads, step):
        n = min(step, pages * kv_heads - i)
        k = _quantised(gen, n, d, "K", kb, dev)
        v = _quantised(gen, n, d, "V", vb, dev)
        parts = [_pack(k[0], ko, ks)] + [t.view(torch.uint8).reshape(n, -1) for t in k[1:]]
        parts += [_pack(v[0], vo, vs)] + [t.view(torch.uint8).reshape(n, -1) for t in v[1:]]
        pool[i:i + n] = torch.cat(parts, 1)
    return pool.reshape(pages, kv_heads, size)


# ---- inputs --------------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    bits = tuple(int(x) for x in case["bits"].split(","))
    batch, new, heads, kv_heads, dim = (case[k] for k in ("batch", "new", "heads", "kv_heads", "dim"))
    d = _padded(dim)
    lens = torch.tensor(_lens(case), dtype=torch.int64)
    pages = [int(n) // TILE for n in lens]
    width = max(1, max(pages))
    used = sum(pages)
    pool = _pool(gen, max(1, used), kv_heads, d, bits, dev)
    perm = torch.randperm(max(1, used), generator=gen, device=dev).int()
    table = torch.zeros(batch, width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n

    def half(*shape):
        return torch.randn(shape, generator=gen, device=dev).half()

    s = {"case": dict(case), "pool": pool, "table": table, "lens": lens.int().to(dev), "scale": 1.0 / math.sqrt(dim),
         "q": half(batch, new, heads, dim), "partial_k": half(batch, kv_heads, TILE, dim),
         "partial_v": half(batch, kv_heads, TILE, dim),
         "out": torch.zeros(batch, new, heads, dim, dtype=torch.float16, device=dev)}
    if case["op"] != "window_decode":
        s["new_k"], s["new_v"] = half(batch, new, kv_heads, dim), half(batch, new, kv_heads, dim)
    if case["op"] == "tree":
        # every node hangs on an earlier one, more often on a recent one
        up = torch.rand(batch, new, generator=gen, device=dev).cpu()
        sees = torch.zeros(batch, new, new, dtype=torch.bool)
        rows = torch.arange(batch)
        for i in range(new):
            if i:
                parent = (i * up[:, i].sqrt()).long().clamp(max=i - 1)
                sees[:, i] = sees[rows, parent]
            sees[:, i, i] = True
        words = -(-new // 32)
        flat = torch.zeros(batch, new, words * 32, dtype=torch.int64)
        flat[:, :, :new] = sees
        packed = (flat.reshape(batch, new, words, 32) << torch.arange(32)).sum(-1)
        s["mask"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).int().to(dev)
        s["new_lens"] = torch.tensor(_new_lens(case), dtype=torch.int32, device=dev)
    s["orders"] = {(k, n): tuple(t.to(dev) for t in _order(k, n, d)) for k, n in (("K", bits[0]), ("V", bits[1]))}
    if own:
        from calibration_free_kv_gb300 import kvarn
        preset = {(4, 2): "kvarn_k4v2_g128", (4, 4): "kvarn_k4v4_g128", (2, 2): "kvarn_k2v2_g128",
                  (8, 4): "kvarn_k8v4_g128"}[bits]
        s["desc"] = kvarn.desc_from_preset(dim, kv_heads, preset)
        if case["op"] == "tree":
            s["workspace"] = kvarn.alloc_tree_workspace(s["desc"], batch, heads, new, width)
        elif case["op"] == "window_decode":
            s["workspace"] = kvarn.alloc_window_decode_workspace(s["desc"], batch, heads, width, case["sink"],
                                                                 case["window"])
        else:
            s["workspace"] = kvarn.alloc_window_prefill_workspace(s["desc"], batch, heads, new, width, case["sink"],
                                                                  case["window"])
    return s


# ---- the plain forms -----------------------------------------------------------------------


def _rotation(d, dev):
    h = torch.ones(1, 1, device=dev)
    two = torch.tensor([[1.0, 1.0], [1.0, -1.0]], device=dev)
    for _ in range(d.bit_length() - 1):
        h = torch.kron(two, h)
    return h / math.sqrt(d)


def _unpack(words, order, shifts, bits, d):
    codes = (words.view(torch.int32).unsqueeze(-1) >> shifts.int()) & (2 ** bits - 1)
    flat = torch.empty(words.shape[:-1] + (TILE * d,), dtype=torch.uint8, device=words.device)
    flat[..., order] = codes.to(torch.uint8).flatten(-2)
    return flat.unflatten(-1, (TILE, d)).float()


def _sealed(s, pages):
    """Keys and values [batch][kv head][page][128][d] (rotated basis) of the given logical pages."""
    case = s["case"]
    bits, d = tuple(int(x) for x in case["bits"].split(",")), _padded(case["dim"])
    ids = torch.gather(s["table"].long(), 1, pages.clamp(0, s["table"].shape[1] - 1))
    rec = s["pool"][ids].transpose(1, 2)  # [batch][kv head][page][bytes]
    ends, _ = _sections(bits, d)
    part = [rec[..., a:b].contiguous() for a, b in ends]
    ks, kz, kr, vs, vz, vc = (part[i].view(torch.float16).float() for i in (1, 2, 3, 5, 6, 7))
    k = _unpack(part[0], *s["orders"][("K", bits[0])], bits[0], d)
    k = (k * ks.unsqueeze(-2) + kz.unsqueeze(-2)) * kr.unsqueeze(-1)
    v = _unpack(part[4], *s["orders"][("V", bits[1])], bits[1], d)
    v = (v * vs.unsqueeze(-1) + vz.unsqueeze(-1)) * vc.unsqueeze(-2)
    return k, v


def _plain(s):
    case = s["case"]
    q, dev = s["q"], s["q"].device
    batch, new, heads, dim = q.shape
    kv_heads, d = case["kv_heads"], _padded(case["dim"])
    group, lens = heads // kv_heads, s["lens"].long()
    sealed_pages = lens // TILE
    decode = case["op"] == "window_decode"
    at = (lens - 1 if decode else lens).unsqueeze(1) + torch.arange(new, device=dev)  # query positions
    if case["op"] == "tree":
        pages = torch.arange(s["table"].shape[1], device=dev).expand(batch, -1)
        live = pages < sealed_pages.unsqueeze(1)
    else:
        start = ((at[:, 0] + 1 - case["window"]).clamp(min=0) // TILE).clamp(max=sealed_pages)
        sinks = -(-case["sink"] // TILE)
        wide = min(s["table"].shape[1], -(-(case["window"] + new) // TILE) + 1)
        first = torch.arange(sinks, device=dev).expand(batch, -1)
        last = start.unsqueeze(1) + torch.arange(wide, device=dev)
        pages = torch.cat([first, last], 1)
        live = torch.cat([first < start.unsqueeze(1), last < sealed_pages.unsqueeze(1)], 1)
    k, v = _sealed(s, pages)
    offset = torch.arange(TILE, device=dev)
    key_at = (pages.unsqueeze(-1) * TILE + offset).flatten(1)  # positions of the sealed keys
    key_on = live.unsqueeze(-1).expand(-1, -1, TILE).flatten(1)
    raw_k, raw_v = s["partial_k"].float(), s["partial_v"].float()
    raw_at = (sealed_pages * TILE).unsqueeze(1) + offset
    raw_on = offset < (lens % TILE).unsqueeze(1)
    if not decode:
        raw_k = torch.cat([raw_k, s["new_k"].float().transpose(1, 2)], 2)
        raw_v = torch.cat([raw_v, s["new_v"].float().transpose(1, 2)], 2)
        raw_at = torch.cat([raw_at, at], 1)
        raw_on = torch.cat([raw_on, torch.ones_like(at, dtype=torch.bool)], 1)
    every_at, every_on = torch.cat([key_at, raw_at], 1), torch.cat([key_on, raw_on], 1)
    if case["op"] == "tree":
        bit = torch.arange(new, device=dev)
        among = ((s["mask"][..., bit // 32] >> (bit % 32).int()) & 1).bool()
        on = torch.cat([every_on[:, None, :-new].expand(-1, new, -1), among], 2)
    else:
        j, i = every_at.unsqueeze(1), at.unsqueeze(2)
        on = every_on.unsqueeze(1) & (j <= i) & ((j < case["sink"]) | (j > i - case["window"]))
    rot = _rotation(d, dev)
    qg = q.float().reshape(batch, new, kv_heads, group, dim).permute(0, 2, 3, 1, 4) * s["scale"]
    q_rot = qg @ rot[:dim]
    n = key_at.shape[1]
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    logits = torch.cat([(q_rot.flatten(2, 3) @ k.transpose(-1, -2)), qg.flatten(2, 3) @ raw_k.transpose(-1, -2)], -1)
    logits = logits.unflatten(2, (group, new)).masked_fill(~on[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p.flatten(2, 3)
    out = (p[..., :n] @ v) @ rot[:, :dim] + p[..., n:] @ raw_v
    out = out.unflatten(2, (group, new)) / torch.where(total == 0, 1.0, total)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, new, heads, dim)
    if case["op"] == "tree":
        real = torch.arange(new, device=dev) < s["new_lens"].unsqueeze(1)
        out = torch.where(real[:, :, None, None], out, 0.0)
    return out.half()


def run(s):
    if not own:
        return _plain(s)
    from calibration_free_kv_gb300 import kvarn
    case = s["case"]
    if case["op"] == "tree":
        kvarn.tree_attention(s["desc"], s["q"], s["new_k"], s["new_v"], s["mask"], s["pool"], s["table"], s["lens"],
                             s["out"], s["workspace"], tree_lens=s["new_lens"], partial_k=s["partial_k"],
                             partial_v=s["partial_v"], softmax_scale=s["scale"])
        return s["out"]
    if case["op"] == "window_decode":
        kvarn.window_decode_attention(s["desc"], s["q"].squeeze(1), s["pool"], s["table"], s["lens"],
                                      s["out"].squeeze(1), s["workspace"], case["sink"], case["window"],
                                      partial_k=s["partial_k"], partial_v=s["partial_v"], softmax_scale=s["scale"])
        return s["out"]
    kvarn.window_prefill_attention(s["desc"], s["q"], s["new_k"], s["new_v"], s["pool"], s["table"], s["lens"],
                                   s["out"], s["workspace"], case["sink"], case["window"],
                                   partial_k=s["partial_k"], partial_v=s["partial_v"], softmax_scale=s["scale"])
    return s["out"]


# ---- the definition, in 64 bits ------------------------------------------------------------


def _exact_tile(rec, bits, d, which, basis):
    """One half of one record in the original basis, by the format's definition: element by
    element positions, (code * scale + zero) * factor, then the inverse rotation."""
    kb, vb = bits
    nb = kb if which == "K" else vb
    base = 0 if which == "K" else TILE * d * kb // 8 + 4 * d + 2 * TILE
    size = TILE * d * nb // 8
    t = torch.arange(TILE, device=rec.device).unsqueeze(1)
    c = torch.arange(d, device=rec.device).unsqueeze(0)
    o, i = t // 16, c // 16
    if which == "K":
        g, rho, h, tq, p = t % 8, t // 8 % 2, c // 8 % 2, c % 8 // 2, c % 2
    else:
        g, rho, h, tq, p = c % 8, c // 8 % 2, t // 8 % 2, t % 8 // 2, t % 2
    lane = 4 * g + tq
    if nb == 4:
        word, bit = ((o * (d // 64) + i // 4) * 32 + lane) * 4 + i % 4, 4 * (h + 2 * rho + 4 * p)
    elif nb == 2:
        word, bit = ((o // 2 * (d // 64) + i // 4) * 32 + lane) * 4 + i % 4, 2 * (2 * (o % 2) + h + 4 * rho + 8 * p)
    else:
        word, bit = ((o * (d // 32) + i // 2) * 32 + lane) * 4 + 2 * (i % 2) + h, 8 * (rho + 2 * p)
    codes = (rec[:, base + 4 * word + bit // 8].long() >> (bit % 8)) & (2 ** nb - 1)

    def meta(start, n):
        return rec[:, start:start + 2 * n].contiguous().view(torch.float16).double()

    if which == "K":
        s, z = meta(base + size, d).unsqueeze(1), meta(base + size + 2 * d, d).unsqueeze(1)
        f = meta(base + size + 4 * d, TILE).unsqueeze(2)
    else:
        s, z = meta(base + size, TILE).unsqueeze(2), meta(base + size + 2 * TILE, TILE).unsqueeze(2)
        f = meta(base + size + 4 * TILE, d).unsqueeze(1)
    return ((codes.double() * s + z) * f) @ basis


def exact(case, seed):
    s = prepare(case, seed)
    bits, dim, d = tuple(int(x) for x in case["bits"].split(",")), case["dim"], _padded(case["dim"])
    dev = s["q"].device
    i = torch.arange(d, device=dev)
    both = i.unsqueeze(0) & i.unsqueeze(1)
    odd = sum((both >> k) & 1 for k in range(8)) % 2
    basis = ((1.0 - 2.0 * odd.double()) / math.sqrt(d))[:, :dim]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    for b, length in enumerate(_lens(case)):
        n, tail, new = length // TILE, length % TILE, _new_lens(case)[b]
        first = length - 1 if case["op"] == "window_decode" else length
        spans = [(0, length)]  # cached tokens that any row sees
        if case["op"] != "tree":
            start = max(0, first + 1 - case["window"])
            spans = [(0, min(case["sink"], start)), (start, length)]
        seen = sorted({p for lo, hi in spans if hi > lo for p in range(lo // TILE, min(n, (hi - 1) // TILE + 1))})
        ids = s["table"][b, torch.tensor(seen, dtype=torch.long, device=dev)].long()
        at = [(torch.tensor(seen, device=dev).unsqueeze(1) * TILE + torch.arange(TILE, device=dev)).flatten(),
              n * TILE + torch.arange(tail, device=dev)]
        if case["op"] != "window_decode":
            at.append(length + torch.arange(new, device=dev))
        at = torch.cat([a.long() for a in at])
        rows = first + torch.arange(new, device=dev)
        if case["op"] == "tree":
            on = torch.ones(new, at.numel(), dtype=torch.bool, device=dev)
            on[:, at.numel() - new:] = False
            words = s["mask"][b].cpu()
            hit = [(a, c) for a in range(new) for c in range(new) if (int(words[a, c // 32]) >> (c % 32)) & 1]
            a, c = (torch.tensor(x, device=dev) for x in zip(*hit))
            on[a, at.numel() - new + c] = True
        else:
            gap = rows.unsqueeze(1) - at.unsqueeze(0)
            on = (gap >= 0) & ((gap < case["window"]) | (at.unsqueeze(0) < case["sink"]))
        for h in range(case["kv_heads"]):
            rec = s["pool"][ids, h]
            k = [_exact_tile(rec, bits, d, "K", basis).reshape(-1, dim), s["partial_k"][b, h, :tail].double()]
            v = [_exact_tile(rec, bits, d, "V", basis).reshape(-1, dim), s["partial_v"][b, h, :tail].double()]
            if case["op"] != "window_decode":
                k.append(s["new_k"][b, :new, h].double())
                v.append(s["new_v"][b, :new, h].double())
            k, v = torch.cat(k), torch.cat(v)
            for g in range(group):
                head = h * group + g
                logit = (s["q"][b, :new, head].double() @ k.T) * s["scale"]
                p = torch.softmax(logit.masked_fill(~on, -math.inf), 1)
                out[b, :new, head] = p @ v
    return out
