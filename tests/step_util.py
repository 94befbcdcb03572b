"""Helpers for the tests of what surrounds the decode: E4M3 codes against
float64 values, and batches behind a shared prefix."""
from __future__ import annotations

import numpy as np
import torch

import oracle.e4m3 as e4m3
from workloads import make_batch_from_lengths

POSITIVE = e4m3.TABLE[:0x7F]                     # 0 .. 448 in code order


def nearest(y):
    """float64 -> the E4M3 value nearest to it (ties to the even code), saturating."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(POSITIVE, a), 1, len(POSITIVE) - 1)
    lo = hi - 1
    dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.sign(y) * np.where(take_hi, POSITIVE[hi], POSITIVE[lo])


def assert_codes(codes, y, err, what=""):
    """Every code is the rounding of some value within `err` of y."""
    v = e4m3.decode(np.asarray(codes))
    lo, hi = nearest(np.asarray(y) - err), nearest(np.asarray(y) + err)
    bad = (v < lo) | (v > hi)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} codes off, first at " \
                          f"{np.argwhere(bad)[0]}: {v[bad][0]} for {np.asarray(y)[bad][0]}"


def angle_table(rows):
    """The rope table [rows, 64] FP32 in numpy, angles in 64 bits."""
    a = np.arange(rows)[:, None] * 10000.0 ** (-2.0 * np.arange(32) / 64)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def prefix_batch(lens, k, H, prefix, seed, std=1.0, scaling="amax", fill=0):
    """(batch of the requests' own keys, prefix table, prefix length): the
    prefix's pages are one more request of the same cache."""
    b = make_batch_from_lengths(list(lens) + [prefix], k, H, seed=seed, value_std=std,
                                scaling=scaling, fill=fill, extra_pages=2)
    pages = max(1, -(-prefix // 64))
    table = b.block_table[-1, :pages].contiguous()
    width = max(1, max(-(-n // 64) for n in lens))
    b.block_table = b.block_table[:-1, :width].contiguous()
    b.seq_lens = b.seq_lens[:-1].contiguous()
    b.q = b.q[:len(lens) * k].contiguous()
    return b, table, prefix
