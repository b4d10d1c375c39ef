"""Weights far below a row's largest one: tree and windowed chunk against 64 bits.

One token leads by 17.6 nats (25.4 in powers of two) and its value is about zero; thousands of others,
each with a weight of 2.3e-8, carry the output.  Probabilities are held in fp16 relative to the row's
reference, whose smallest step is 2^-24: a weight below 2^-25 of the reference would be lost altogether,
the whole output with it (0.02 to 0.05 here, ten times the tolerance and more).  What is allowed is the
decode tolerance of tests/helpers.py, 2e-3 of max(1, max |out|): a weight of 2^-25.4 that sits 7 powers
of two higher in fp16 is a multiple of 2^-24 of 2^-18.4, off by at most 2^-25 / 2^-18.4 = 1 %, 5e-4 of an
output of 0.05; V~ and the output add 2^-11 of it each.
"""

import numpy as np
import pytest
import torch

from oracle import kvarn_oracle as ko
from tests import block_cases as B

pytestmark = pytest.mark.gpu

LEAD = 17.6  # nats


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def _rows(g, n, d0, lead, value):
    """q [d0], keys [n, d0] and values [n, d0]: key 0 `lead` nats ahead of the others, whose logits are
    about 0, with a value near zero where the others' entries are +-value."""
    u = torch.where(torch.rand(d0, generator=g) < 0.5, -1.0, 1.0)
    k = 0.02 * torch.randn((n, d0), generator=g)
    k[0] = 2.0 * u
    q = u * (lead / (2.0 * d0 * B.scale_of(d0)))
    w = torch.where(torch.rand(d0, generator=g) < 0.5, -value, value)
    v = w * (1.0 + 0.1 * torch.randn((n, d0), generator=g))
    v[0] = 0.01 * torch.randn(d0, generator=g)
    return q.half(), k.half(), v.half()


@pytest.mark.parametrize("group,d0,preset", [(1, 128, "kvarn_k4v2_g128"), (8, 128, "kvarn_k4v4_g128"),
                                             (4, 64, "kvarn_k8v4_g128"), (4, 256, "kvarn_k4v2_g128")])
def test_small_weights_of_sealed_pages(kv, group, d0, preset):
    # enough sequences that most row tiles lie in one CTA; all take the same two pages: the leading
    # token's, then the other one 63 times
    batch, pages = 304, 64
    g = torch.Generator().manual_seed(60 + d0)
    q1, k, v = _rows(g, 256, d0, LEAD, 100.0)
    desc = kv.desc_from_preset(d0, 1, preset=preset)
    pool = kv.alloc_pool(desc, 2)
    kv.quantize_tiles(desc, k[:, None].contiguous().cuda(), v[:, None].contiguous().cuda(),
                      torch.arange(2, dtype=torch.int32, device="cuda"), pool)
    recs = [ko.dequantize_record(bytes(r[0].tobytes()), d0, *ko.PRESETS[preset]) for r in pool.cpu().numpy()]
    kk, vv = (np.concatenate([recs[0][i]] + [recs[1][i]] * (pages - 1)) for i in range(2))
    table = torch.ones((batch, pages), dtype=torch.int32)
    table[:, 0] = 0
    lens = torch.full((batch,), 128 * pages, dtype=torch.int32, device="cuda")
    # queries that differ a little from row to row; the node sees nothing but the cache
    q = (q1 * (1.0 + 0.01 * torch.randn((batch, 1, group, 1), generator=g))).half()
    nk = torch.zeros((batch, 1, 1, d0), dtype=torch.float16, device="cuda")
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    kv.tree_attention(desc, q.cuda(), nk, nk, torch.zeros((batch, 1, 1), dtype=torch.int32, device="cuda"), pool,
                      table.cuda(), lens, out, kv.alloc_tree_workspace(desc, batch, group, 1, pages))
    got = out.cpu().double().numpy().reshape(-1, d0)
    on = np.ones((1, 128 * pages), dtype=bool)
    ref = np.concatenate([B.attend(r[None], kk, vv, on, B.scale_of(d0)) for r in q.double().numpy().reshape(-1, d0)])
    size = np.abs(ref).max(axis=1)
    assert size.min() > 0.005  # the small weights do carry the output
    print("G=%d d0=%d: output up to %.3f, max scaled error %.1e" % (group, d0, size.max(), B.close(got, ref, "sealed")))


@pytest.mark.parametrize("group,d0", [(1, 128), (4, 64), (2, 256)])
def test_small_weights_of_raw_tokens(kv, group, d0):
    # a chunk without a cache whose first token leads for every row
    n = 2048
    g = torch.Generator().manual_seed(70 + d0)
    q1, k, v = _rows(g, n, d0, LEAD, 1000.0)
    desc = kv.desc_from_preset(d0, 1)
    q = (q1 * (1.0 + 0.01 * torch.randn((1, n, group, 1), generator=g))).half()
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    pool, table = kv.alloc_pool(desc, 1), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    kv.window_prefill_attention(desc, q.cuda(), k[None, :, None].contiguous().cuda(), v[None, :, None].contiguous().cuda(),
                                pool, table, torch.zeros(1, dtype=torch.int32, device="cuda"), out,
                                kv.alloc_window_prefill_workspace(desc, 1, group, n, 1, 1, 4096), 1, 4096)
    got = out.cpu().double().numpy()[0]
    on = np.tril(np.ones((n, n), dtype=bool))
    kd, vd = k.double().numpy(), v.double().numpy()
    ref = np.stack([B.attend(q[0, :, h].double().numpy(), kd, vd, on, B.scale_of(d0)) for h in range(group)], 1)
    assert np.abs(ref[n // 2:]).max(axis=-1).min() > 0.01
    print("G=%d d0=%d: max scaled error %.1e" % (group, d0, B.close(got, ref, "raw")))
