"""The books of a bounded cache, in float64: what each cached key got from a
decode step's rows, and which keys stay when it is cut down.

Test infrastructure only (see the package docstring).
"""
from __future__ import annotations

import math

import numpy as np

from . import attention as att
from . import e4m3


def key_weights(q_codes, kv_codes, block_table, seq_lens, lse, k: int, bmm1: float):
    """Per request: the sum over its k*H rows of 2^(score - lse) [len], and a bound of
    how far FP32 arithmetic may be from it. Rows whose LSE is not finite add nothing.

    The bound: products of E4M3 values are exact in FP32; a sum of 576 of them in any
    order is off by 576 steps of 2^-23 of the sum of their sizes; the scale (two
    roundings), the subtraction and the exponential (2^-22) add 2^-21 of |x| and of |lse|
    at most, and the sum over the rows one rounding per row."""
    sums, bounds = [], []
    q = e4m3.decode(np.asarray(q_codes))
    for r, n in enumerate(seq_lens):
        n = max(int(n), 0)
        keys = att.request_keys(kv_codes, np.asarray(block_table)[r], 0, n, 1.0)
        rows = q[r * k:(r + 1) * k].reshape(-1, 576)
        l = np.asarray(lse[r], dtype=np.float64)
        good = np.isfinite(l)
        c = float(np.float32(bmm1)) / math.log(2.0)
        x = c * (rows[good] @ keys.T)
        size = c * (np.abs(rows[good]) @ np.abs(keys).T)
        p = np.exp2(x - l[good][:, None])
        off = math.log(2.0) * (size * 576 * 2.0 ** -23 + (np.abs(x) + np.abs(l[good])[:, None]) * 2.0 ** -21)
        s = p.sum(0)
        sums.append(s)
        bounds.append((p * np.expm1(off)).sum(0) + s * (2.0 ** -21 + len(p) * 2.0 ** -24) + 1e-30)
    return sums, bounds


def evict(n: int, weights, positions, keep: int, recent: int, sinks: int):
    """(slots of the kept keys, in slot order; moves as (from, to) pairs) of one request
    of n keys: held keys first (position below sinks, or one of the `recent` newest
    positions' range), then by weight, NaN last, ties to the lower slot."""
    n, keep = max(n, 0), max(keep, 0)
    newest = max((int(p) for p in positions[:n]), default=-1) + 1 - recent

    def place(j):
        held = int(positions[j]) < sinks or (recent > 0 and int(positions[j]) >= newest)
        w = float(weights[j])
        return (0, 0, 0.0, j) if held else (1, 1, 0.0, j) if math.isnan(w) else (1, 0, -w, j)

    kept = sorted(sorted(range(n), key=place)[:keep])
    stays = set(kept)
    holes = [j for j in range(min(n, keep)) if j not in stays]
    return kept, list(zip([j for j in kept if j >= keep], holes))
