"""A packed cache built on the GPU and its attention in 64 bits, for the tests of the operators that
take several or windowed queries.

The records are quantised by the library, read back and dequantised in 64 bits by the oracle, so the
expected values come from the same bytes.  Tolerance: the decode tolerance of tests/helpers.py, 2e-3
of max(1, max |out|) per query head.  What the kernels round to fp16 (half a step, 2^-11, each): the
output, the probabilities, V~ twice (code s + z, then times c).  The three roundings inside are
independent over tokens and channels, and the inverse rotation averages a row's over its channels:
an output element moves by about 2^-11 sqrt(3) / sqrt(3) (uniform in the half step) of the value
row's rms, four standard deviations are 4 x 4.9e-4 = 2e-3 of that rms, and max |out| of a head is
two to three times its rms.
"""

from __future__ import annotations

import math

import numpy as np
import torch

from calibration_free_kv_gb300 import synth
from oracle import kvarn_oracle as ko
from tests import helpers as H


class Cache:
    """Sequences of the given lengths, quantised page by page into a shuffled pool."""

    def __init__(self, kv, lens, hkv, d0, seed, preset="kvarn_k4v2_g128", plain=False):
        self.kv, self.lens, self.hkv, self.d0 = kv, list(lens), hkv, d0
        self.bits = ko.PRESETS[preset]
        self.desc = kv.desc_from_preset(d0, hkv, preset=preset)
        g = torch.Generator().manual_seed(seed)
        pages = [n // 128 for n in lens]
        self.n_pool = sum(pages) + 2
        perm = torch.randperm(self.n_pool, generator=g).int()
        self.table = torch.zeros((len(lens), max(max(pages), 1)), dtype=torch.int32)
        self.pool = kv.alloc_pool(self.desc, self.n_pool)
        self.pk = torch.zeros((len(lens), hkv, 128, d0), dtype=torch.float16)
        self.pv = torch.zeros_like(self.pk)
        self.k, self.v = [], []
        self.free_page = int(perm[sum(pages)])  # a page that no sequence uses
        at = 0
        for b, n in enumerate(lens):
            if plain:
                k, v = (torch.randn((max(n, 1), hkv, d0), generator=g).half()[:n] for _ in range(2))
            else:
                k, v = (t[:n] for t in synth.outlier_kv(max(n, 1), hkv, d0, seed=seed * 100 + b))
            m = pages[b]
            self.table[b, :m] = perm[at:at + m]
            at += m
            kk, vv = k.double().numpy(), v.double().numpy()
            if m:
                ids = self.table[b, :m].cuda()
                kv.quantize_tiles(self.desc, k[:128 * m].contiguous().cuda(), v[:128 * m].contiguous().cuda(), ids,
                                  self.pool)
                recs = self.pool[ids.long()].cpu().numpy()
                for i in range(m):
                    for h in range(hkv):
                        a, c = ko.dequantize_record(bytes(recs[i, h].tobytes()), d0, *self.bits)
                        kk[128 * i:128 * i + 128, h], vv[128 * i:128 * i + 128, h] = a, c
            rem = n - 128 * m
            if rem:
                self.pk[b, :, :rem] = k[128 * m:].transpose(0, 1)
                self.pv[b, :, :rem] = v[128 * m:].transpose(0, 1)
            self.k.append(kk)
            self.v.append(vv)
        # rows of the open tile past its tokens are never used
        for b, n in enumerate(lens):
            self.pk[b, :, n % 128:] = float("nan")
            self.pv[b, :, n % 128:] = float("nan")
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.args = dict(partial_k=self.pk.cuda(), partial_v=self.pv.cuda())

    def unseen(self, b, pages):
        """Point the table's entries of these logical pages outside the pool."""
        self.table[b, list(pages)] = -7


def attend(q, k, v, on, scale):
    """softmax(scale q k^T) v over the keys `on` names, 64 bits; a row without any gives zeros."""
    s = np.where(on, (q @ k.T) * scale, -np.inf)
    m = s.max(axis=1, keepdims=True) if s.shape[1] else np.full((len(q), 1), -np.inf)
    p = np.where(on, np.exp(s - np.where(np.isinf(m), 0.0, m)), 0.0)
    total = p.sum(axis=1, keepdims=True)
    return (p / np.where(total == 0, 1.0, total)) @ v


def expected(cache, b, q, new_k, new_v, on, scale, group):
    """[block, Hq, d0] of sequence b: q [block, Hq, d0], new_k/v [block, Hkv, d0] or None, on
    [block, cached + block]."""
    out = np.zeros(q.shape)
    for hq in range(q.shape[1]):
        h = hq // group
        k, v = cache.k[b][:, h], cache.v[b][:, h]
        if new_k is not None:
            k, v = np.concatenate([k, new_k[:, h]]), np.concatenate([v, new_v[:, h]])
        out[:, hq] = attend(q[:, hq], k, v, on, scale)
    return out


def window_mask(first, rows, cols, sink, window):
    p, j = first + np.arange(rows)[:, None], np.arange(cols)[None, :]
    return (j <= p) & ((j < sink) | (j > p - window))


def ancestors(nodes, gen):
    """A random tree's mask [nodes, nodes]: each node sees itself and its ancestors."""
    sees = np.zeros((nodes, nodes), dtype=bool)
    for i in range(nodes):
        if i:
            sees[i] = sees[int(torch.randint(0, i, (1,), generator=gen))]
        sees[i, i] = True
    return sees


def pack_mask(sees):
    """bool [..., n] -> int32 words [..., ceil(n / 32)]."""
    n = sees.shape[-1]
    words = -(-n // 32)
    flat = np.zeros(sees.shape[:-1] + (words * 32,), dtype=np.uint64)
    flat[..., :n] = sees
    w = (flat.reshape(sees.shape[:-1] + (words, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(w.astype(np.uint32).view(np.int32))


def close(got, ref, what):
    return H.assert_decode_close(got, ref, what)


def scale_of(d0):
    return 1.0 / math.sqrt(d0)
