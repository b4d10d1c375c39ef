"""Precision of the selection's log-sum-exp (GPU).

A row's score is chosen so that its best candidate ends next to zero: the result's own rounding is then lost beside
the error of the logarithm, which is what it shows.

Tolerance, in steps of 2^-24 of the sum.  A term is 2^y, y = (x - ref) log2(e) in one rounding: 2^-22 of the term (4)
for the exponential, and d + 1 for the rounding of y and d / 4 for log2(e)'s own, d the distance from the row's greatest
(a reference lies at most 1 below its warp's greatest logit).  A thread adds 16 (fp32: 8) terms of a tile in 5 (3)
additions, the tiles without an error; 1 for the correction of the reference's product, 5 for a warp's threads, 5 for each
of the two steps that join warps and chunks (an exponential, a product, an addition), 1 for the logarithm.  A reference moves by
at least 1, so that a term is carried d times at most, each an exponential of 2 and a third of a step for its argument, 2.7.
The mean of d over the terms is at most 9 for 2^18 logits and 14.4 for 2^26 (one peak above equal ones): 27 + 4 x 9 = 63 steps
or 3.7e-6, 27 + 4 x 14.4 = 85 or 5e-6.
"""

import pytest
import torch
from test_gpu_beam import TYPES, check, kv, make  # noqa: F401

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24


def errors(kv, logits, count=1):  # noqa: F811
    """Of every row: the error of the logarithm of its sum, and the tolerance above."""
    rows, vocab = logits.shape
    x = logits.double()
    d = x.amax(1, keepdim=True) - x
    total = torch.exp(-d).sum(1)
    lse = torch.log(total)  # of the differences from the greatest
    scores = lse.float().unsqueeze(1)
    outs = [torch.zeros(rows, count, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = kv.alloc_beam_select_workspace(rows, 1, vocab, count)
    kv.beam_select(logits.unsqueeze(1), scores, *outs, ws, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    mean = (torch.nan_to_num(d, posinf=0.0) * torch.exp(-d)).sum(1) / total
    tol = STEP * (4 + 1 + 5 + 1 + 5 + 10 + 1 + mean * (1 + 0.25 + 2.7))
    return outs[0][:, 0].double() - (scores[:, 0].double() - lse), tol


def rows_of(kind, rows, vocab, dtype, offset):
    g = torch.Generator().manual_seed(rows + vocab)
    x = torch.randn(rows, vocab, generator=g)
    i = torch.arange(vocab)
    x = {"random": 3.0 * x, "wide": 20.0 * x, "rising": x + 12.0 * i / vocab,
         "steps": 2.0 * (i * 8 // vocab) - (2.0 * x).abs() - 8.0 * (i % 40 != 0)}[kind]
    return (x + offset).to(TYPES[dtype]).cuda()


@pytest.mark.parametrize("offset", [0.0, 30.0, -300.0, 3000.0, 60_000.0, -65_000.0])
@pytest.mark.parametrize("kind", ["random", "wide", "rising", "steps"])
@pytest.mark.parametrize("rows,vocab", [(320, 20_001), (3, 200_003)])  # one chunk a row, and many
def test_offset(kv, rows, vocab, kind, offset):  # noqa: F811
    """What is carried when a reference moves is not touched by the rounding of the new one's product."""
    err, tol = errors(kv, rows_of(kind, rows, vocab, "fp32", offset))
    assert (err.abs() <= tol).all(), (float(err.abs().max()), float(tol[err.abs().argmax()]))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind,offset", [("random", 0.0), ("wide", 0.0), ("steps", 0.0), ("random", 2000.0)])
def test_offset_16_bits(kv, kind, offset, dtype):  # noqa: F811
    err, tol = errors(kv, rows_of(kind, 320, 20_001, dtype, offset))
    assert (err.abs() <= tol).all(), (float(err.abs().max()), float(tol[err.abs().argmax()]))


@pytest.mark.parametrize("low", [-65_700.0, -65_540.0, -131_072.0, -3e38])
def test_close_to_the_slower_path(kv, low):  # noqa: F811
    # logits on both sides of -65536, where sums change their form, and behind a first tile of `low`
    logits, scores = make(1, 32, 12289, "fp32", 7, scale=20.0)
    logits -= 65_536.0
    logits[:, 8:16] += 100.0
    logits[:, 16:24] -= 100.0
    logits[..., :2048] = low
    check(kv, logits, scores, 64)


@pytest.mark.parametrize("count", [1, 8])  # 8: all of the equal logits reach the bound, the slower path
@pytest.mark.parametrize("rows,vocab", [(512, 151_936), (160, 1 << 20), (640, 9004)])
def test_peak_over_equal_logits(kv, rows, vocab, count):  # noqa: F811
    """A peak whose warp holds nothing else, over equal logits of which the other warps sum ones, exactly: the step
    that joins the warps shows.

    Of the sum the share w is of the equal logits: an exponential of 2 steps, a product, an addition.  The peak's share has the
    exponential's 4, its argument's 1 and the correction's 1.  1 for the chunk's sum, 1 for the logarithm."""
    i = torch.arange(vocab, device="cuda") % 1024 // 128  # the warp that loads it, 16 bytes a thread
    at = torch.arange(rows, device="cuda") * 7919 % vocab
    peak = 4.0 + 10.0 * torch.arange(rows, device="cuda") / rows
    logits = torch.where(i == i[at].unsqueeze(1), -torch.inf, 0.0)
    logits[torch.arange(rows, device="cuda"), at] = peak
    err, _ = errors(kv, logits, count)
    d = logits.amax(1).double()
    w = 1.0 - 1.0 / (1.0 + (logits == 0).sum(1) * torch.exp(-d))
    tol = STEP * (2 + 4 * w + 6 * (1 - w))
    assert (err.abs() <= tol).all(), (float(err.abs().max()), float(tol[err.abs().argmax()]))


@pytest.mark.parametrize("batch,beams,vocab,dtype", [(64, 8, 151_936, "bf16"), (32, 4, 128_000, "fp16"), (8, 5, 50_001, "fp32")])
def test_random_rows(kv, batch, beams, vocab, dtype):  # noqa: F811
    # the mean square that kvarn.h gives, 8e-8, within a factor of two for the sample and the shape
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 2.0 * torch.randn(batch * beams, vocab, generator=g, device="cuda")
    err, tol = errors(kv, x.to(TYPES[dtype]))
    assert (err.abs() <= tol).all()
    assert float(err.square().mean().sqrt()) <= 1.6e-7


@pytest.mark.parametrize("count", [1, 8])
@pytest.mark.parametrize("rows,vocab", [(512, 151_936), (3, 200_003)])
def test_peak_among_equal_logits(kv, rows, vocab, count):  # noqa: F811
    # the slower path: its terms have 2 + d steps (an exponential, the rounding of its argument), its sums those of the fast path
    at = torch.arange(rows, device="cuda") * 7919 % vocab
    logits = torch.zeros(rows, vocab, device="cuda")
    logits[torch.arange(rows, device="cuda"), at] = 4.0 + 10.0 * torch.arange(rows, device="cuda") / rows
    err, tol = errors(kv, logits, count)
    assert (err.abs() <= tol).all(), (float(err.abs().max()), float(tol[err.abs().argmax()]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("near", [4096, 1])  # whole tiles, the slower path, or one logit in 8
def test_small_terms_are_not_lost(kv, near, dtype):  # noqa: F811
    # each of the small logits' terms is less than half a step of the sum that it is added to
    i = torch.arange(1 << 20, device="cuda")
    high = i < near if near > 1 else (i < 2048) & (i % 8 == 0)
    row = torch.where(high, 0.0, -17.0)
    logits = row.to(TYPES[dtype]).expand(160, -1).contiguous()
    err, tol = errors(kv, logits)
    assert (err.abs() <= tol).all(), (float(err.abs().max()), float(tol[0]))


def test_far_rows_that_rise(kv):  # noqa: F811
    # references beyond 65536 that move often
    x = torch.arange(30_000, device="cuda") / 2000 + 0.01 * torch.randn(160, 30_000, device="cuda")
    for offset in (1e5, -1e5, 4e6):
        err, tol = errors(kv, x + offset)
        assert (err.abs() <= tol).all(), (offset, float(err.abs().max()), float(tol.max()))


@pytest.mark.parametrize("apart", [1e-11, 1e-9, 1e-6])
def test_order_within_a_beam(kv, apart):  # noqa: F811
    # logits of one beam more than 2^-45 of the score apart are in their order, the later token first here
    logits = torch.full((1, 2, 5000), -50.0, device="cuda")
    at = torch.arange(8, device="cuda") * 600
    logits[0, :, at] = apart * torch.arange(8.0, device="cuda")
    outs = [torch.zeros(1, 8, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    ws = kv.alloc_beam_select_workspace(1, 2, 5000, 8)
    kv.beam_select(logits, torch.tensor([[-100.0, -30.0]], device="cuda"), *outs, ws)
    assert apart > 2.0 ** -45 * 33
    assert outs[1].tolist() == [[1] * 8] and outs[2].tolist() == [at.flip(0).tolist()]


def test_finished_rows_hold_anything(kv):  # noqa: F811
    # rows that do not count: no status, and the others' results to the bit
    logits, scores = make(3, 4, 30_000, "bf16", 13)
    done = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    done[0, 1] = done[2] = True
    scores[1, 2] = -torch.inf
    results = []
    for fill in (0.0, float("nan"), float("inf"), -3e38):
        logits[0, 1] = logits[2] = logits[1, 2] = fill
        outs = [torch.zeros(3, 8, dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = kv.alloc_beam_select_workspace(3, 4, 30_000, 8)
        kv.beam_select(logits, scores, *outs, ws, done=done, end_token=9, status=status)
        assert status.item() == 0
        results.append(outs)
    for outs in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs, results[0]))
