"""Selection over logits masked with large finite values, in chunks of several tiles (GPU).

A chunk is streamed in tiles of 4096 16-bit or 2048 32-bit logits, and the references of its sums move from masked
tiles to ordinary ones.  Only NaN and +inf leave a beam out, so the status stays 0 and the result is the 64-bit one,
within the tolerances of test_gpu_beam.
"""

import pytest
import torch
from test_gpu_beam import TYPES, check, kv, make  # noqa: F401

pytestmark = pytest.mark.gpu


def masked(kind, vocab, dtype):
    """Indices of the masked tokens: parts of a chunk's tiles, whose layout follows the loads' width (16 bytes a thread)."""
    i = torch.arange(vocab)
    tile, per = (2048, 4) if dtype == "fp32" else (4096, 8)
    return {"first tile": i < tile, "first two": i < 2 * tile, "inside": (i >= 4) & (i < 2 * tile + 4),
            "a warp's share": (i < tile) & (i % (256 * per) // (32 * per) == 2),
            "a warp's chunk": i % (256 * per) // (32 * per) == 5,
            "middle": (i >= tile + 100) & (i < 2 * tile + 500), "tail": i >= vocab - tile - 700,
            "all but 70": (i < vocab - 700) | (i % 10 != 0)}[kind].cuda()


@pytest.mark.parametrize("dtype,value", [("fp16", "min"), ("bf16", "min"), ("bf16", -1e30), ("bf16", -1e10),
                                         ("bf16", -1e9), ("fp32", "min"), ("fp32", -1e30), ("fp32", -1e10), ("fp32", -5e9),
                                         ("fp32", -7e4)])
@pytest.mark.parametrize("batch,beams,vocab,count", [
    (1, 32, 12289, 64),   # rows in one chunk, the last tile of one logit
    (1, 1, 200_003, 64),  # one row in 14 chunks of four tiles (32 bits: seven)
    (200, 1, 20_001, 8)])
@pytest.mark.parametrize("kind", ["first tile", "first two", "inside", "a warp's share", "a warp's chunk", "middle", "tail",
                                  "all but 70"])
def test_masked(kv, kind, batch, beams, vocab, count, dtype, value):  # noqa: F811
    logits, scores = make(batch, beams, vocab, dtype, vocab)
    logits[..., masked(kind, vocab, dtype)] = torch.finfo(TYPES[dtype]).min if value == "min" else value
    check(kv, logits, scores, count)


@pytest.mark.parametrize("pad,shift", [(0, 1), (2, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_narrow_loads(kv, dtype, pad, shift):  # noqa: F811
    # rows aligned to one and to two elements
    logits, scores = make(2, 32, 12289, dtype, 5, pad=pad, shift=shift)
    logits[0, :, :8192] = torch.finfo(TYPES[dtype]).min
    logits[1, :16, 64:4096] = -1e30
    check(kv, logits, scores, 64)


def test_masked_captured(kv):  # noqa: F811
    # the lowest value moves between replays: no sum of one call is left in the next
    logits, scores = make(4, 8, 20_001, "bf16", 9)
    outs = [torch.zeros(4, 8, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = kv.alloc_beam_select_workspace(4, 8, 20_001, 8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.beam_select(logits, scores, *outs, ws, status=status)
    plain = logits.clone()
    for first in (0, 4096, 8192, 0):
        logits.copy_(plain)
        logits[..., first:first + 8192] = torch.finfo(torch.bfloat16).min
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        kv.beam_select(logits, scores, *outs, ws, status=status)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)) and status.item() == 0
        check(kv, logits, scores, 8)
