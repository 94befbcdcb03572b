"""The attention of packed prompts in 64 bits, request by request and head by head, with what the
tests' tolerances are made of. Runs wherever its tensors are."""
from __future__ import annotations

import math

import torch


def reference(q, k_nope, k_rope, v, cu, cu_keys, sm_scale, causal):
    """out [T, H, 128], lse [T, H] (base 2), tol [T, H, 128], lse_tol [T, H] in float64. Rows of no
    request get NaN in out.

    The kernel's arithmetic: scores from exact BF16 products summed in FP32 in some order, off by
    192 steps of 2^-23 of the sum of their sizes, and by 2^-21 of the score and of the maximum
    for the scale, the subtraction and the exponential: a weight is off by that much times ln 2, in
    the sum of weights too. Its rounding to BF16 for the product: 2^-8 (half a step). FP32 sums of
    m weights and products: m 2^-24 each. The output's own rounding: 2^-8."""
    T, H = q.shape[:2]
    G = H // k_nope.shape[1]
    f64 = torch.float64
    out = torch.full((T, H, 128), math.nan, dtype=f64, device=q.device)
    lse = torch.full((T, H), math.nan, dtype=f64, device=q.device)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    ck = cu if cu_keys is None else cu_keys
    for r in range(len(cu) - 1):
        a, b, c, d = cu[r], cu[r + 1], ck[r], ck[r + 1]
        n, m = b - a, d - c
        if n <= 0:
            continue
        for h in range(H):
            kk = torch.cat([k_nope[c:d, h // G], k_rope[c:d]], 1).to(f64)
            qq, vv = q[a:b, h].to(f64), v[c:d, h // G].to(f64)
            x = qq @ kk.T * sm_scale
            size = qq.abs() @ kk.abs().T * sm_scale / math.log(2)
            if causal:
                i, j = torch.arange(n, device=q.device), torch.arange(m, device=q.device)
                hidden = j[None] > i[:, None] + (m - n)
                x, size = x.masked_fill(hidden, -math.inf), size.masked_fill(hidden, 0)
            if m == 0:
                out[a:b, h], lse[a:b, h] = 0, -math.inf
                continue
            l = torch.logsumexp(x, 1)
            w = torch.exp(x - torch.where(l == -math.inf, 0.0, l)[:, None])
            out[a:b, h], lse[a:b, h] = w @ vv, l / math.log(2)
            spread = w @ vv.abs()
            off = size.amax(1) * (192 * 2.0 ** -23 + 4 * 2.0 ** -21) + 2.0 ** -20
            each = 2 * math.log(2) * off + 2.0 ** -8 + 2 * m * 2.0 ** -24
            tol[a:b, h] = 1.01 * (spread * each[:, None] + (w @ vv).abs() * 2.0 ** -8) + 1e-30
            lse_tol[a:b, h] = off + m * 2.0 ** -23 + torch.nan_to_num(lse[a:b, h].abs(), posinf=0) * 2.0 ** -22
    return out, lse, tol, lse_tol


def check(got, got_lse, ref, what=""):
    """Rows of requests against reference(); returns which rows those are."""
    out, lse, tol, lse_tol = ref
    rows = ~torch.isnan(lse)
    err = (got.to(torch.float64) - out).abs()
    bad = rows[..., None] & ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, first at {bad.nonzero()[0].tolist()}: " \
                          f"{float(err[bad][0])} of {float(tol[bad][0])}"
    if got_lse is not None:
        empty = rows & (lse == -math.inf)
        assert (got_lse[empty] == -math.inf).all(), f"{what}: rows without keys have an LSE"
        full = rows & ~empty
        err = (got_lse.to(torch.float64) - lse).abs()
        assert (err[full] <= lse_tol[full]).all(), f"{what}: lse off by {float(err[full].max())}"
    return rows
