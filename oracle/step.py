"""What surrounds the decode in a step, in float64: new tokens into the paged
cache, absorbed queries, and the decode of a batch behind a shared prefix.

Test infrastructure only (see the package docstring).

Values are returned before the rounding to E4M3: the CUDA path is checked
against the codes that values within its arithmetic's error round to.
"""
from __future__ import annotations

import math

import numpy as np

from . import attention as att
from . import e4m3

LATENT, ROPE, NOPE = 512, 64, 128


def rotate(x, position, interleaved: bool, base: float = 10000.0):
    """The 64 rope dims of one token at `position`: plane i turns by
    position * base^(-2 i / 64); planes pair dims (2 i, 2 i + 1) or (i, i + 32)."""
    y = np.empty(ROPE)
    for i in range(ROPE // 2):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + ROPE // 2)
        a = position * base ** (-2.0 * i / ROPE)
        y[p] = x[p] * math.cos(a) - x[q] * math.sin(a)
        y[q] = x[q] * math.cos(a) + x[p] * math.sin(a)
    return y


def cache_row(x, weight, eps: float, position: int, interleaved: bool, scale: float):
    """One new token's cache row [576] before rounding: RMS-normed latent
    (weight None: as it is), rotated rope dims, over the cache's scale."""
    x = np.asarray(x, dtype=np.float64)
    lat = x[:LATENT]
    if weight is not None:
        lat = lat / math.sqrt((lat * lat).sum() / LATENT + eps) * np.asarray(weight, np.float64)
    return np.concatenate([lat, rotate(x[LATENT:], position, interleaved)]) / scale


def absorbed_query(q, w_uk, position: int, interleaved: bool, scale: float):
    """One (token, head) query [576] before rounding: q[0:128] . w_uk [128, 512],
    rotated q[128:192], over the query scale."""
    q = np.asarray(q, dtype=np.float64)
    lat = q[:NOPE] @ np.asarray(w_uk, dtype=np.float64)
    return np.concatenate([lat, rotate(q[NOPE:], position, interleaved)]) / scale


def prefix_decode(q_codes, kv_codes, prefix_table, prefix_len: int, block_table, seq_lens,
                  k: int, sm_scale: float, q_scale: float, kv_scale: float):
    """Every row attends to the prefix's keys, then its own request's.
    Returns out [R, k*H, 512], lse2 [R, k*H] and two measures of what errors of
    the weights can move an output by: spread [R, k*H, 512], the attention over
    |v| (relative errors), and reach [R, k*H, 512], the sum of |v| over the sum
    of the weights relative to the largest (absolute ones). Rows without keys
    get 0, -inf, 0, 0."""
    q = np.asarray(q_codes)
    R = len(seq_lens)
    M = k * q.shape[1]
    out, lse = np.zeros((R, M, 512)), np.full((R, M), -np.inf)
    spread, reach = np.zeros((R, M, 512)), np.zeros((R, M, 512))
    shared = att.request_keys(kv_codes, prefix_table, 0, int(prefix_len), kv_scale)
    for r in range(R):
        own = att.request_keys(kv_codes, np.asarray(block_table)[r], 0, int(seq_lens[r]), kv_scale)
        keys = np.concatenate([shared, own])
        if not len(keys):
            continue
        qd = e4m3.decode(q[r * k:(r + 1) * k].reshape(M, 576)) * float(q_scale)
        out[r], lse[r] = att.attend(qd, keys, sm_scale)
        s = sm_scale * (qd @ keys.T)
        e = np.exp(s - s.max(1, keepdims=True))
        z = e.sum(1, keepdims=True)
        size = np.abs(keys[:, :512])
        spread[r] = (e / z) @ size
        reach[r] = size.sum(0)[None] / z
    return out, lse, spread, reach
