"""Absorbed queries (mla_query_absorb) against the oracle's values.

Tolerance: a code must be the E4M3 rounding of some value within the FP32
arithmetic's error of the exact one: 128 exact BF16 products accumulated in
FP32 (at most 128 roundings of 2^-23 of the running magnitude: below
2^-16 sum |q w|) and one product with the scale's reciprocal (2^-23); rope
dims as for the cache, below 2^-21 (|a| + |b|).
"""
import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.step as st
from tests.step_util import angle_table, assert_codes

pytestmark = pytest.mark.gpu


def _inputs(R, k, H, seed, stride=192, rows=4000):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((R * k, H, stride), generator=g).to(torch.bfloat16).cuda()[:, :, :192]
    w = (torch.randn((H, 128, 512), generator=g) / 128 ** 0.5).to(torch.bfloat16).cuda()
    starts = torch.randint(0, rows - k, (R,), generator=g).int()
    return q, w, starts, rows


def _check(out, q, w, starts, k, interleaved, scale, picks=None):
    out = out.cpu().numpy()
    q, w = q.float().cpu().numpy().astype(np.float64), w.float().cpu().numpy().astype(np.float64)
    T, H = q.shape[:2]
    for t in range(T) if picks is None else picks:
        pos = int(starts[t // k]) + t % k
        for h in range(H):
            y = st.absorbed_query(q[t, h], w[h], pos, interleaved, scale)
            e = np.empty(576)
            e[:512] = (2.0 ** -16 * (np.abs(q[t, h, :128]) @ np.abs(w[h]))) / scale
            pe = np.abs(q[t, h, 128:])
            pair = pe.reshape(32, 2).sum(1).repeat(2) if interleaved else np.tile(pe[:32] + pe[32:], 2)
            e[512:] = 2.0 ** -21 * pair / scale
            assert_codes(out[t, h], y, e, f"token {t} head {h}")


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("R,k,H", [(1, 1, 1), (2, 4, 8), (5, 7, 3), (127, 1, 2), (129, 1, 1),
                                   (64, 2, 2), (43, 3, 5)])
def test_against_the_oracle(R, k, H, interleaved):
    q, w, starts, rows = _inputs(R, k, H, seed=R * k + H)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mla.query_absorb(q, w, angle_table(rows).cuda(), starts.cuda(), 6 / 448,
                           interleaved=interleaved, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _check(out, q, w, starts, k, interleaved, 6 / 448)


@pytest.mark.parametrize("R,k,H", [(16, 4, 64), (128, 7, 64), (64, 7, 8), (100, 5, 20), (20, 1, 160)])
def test_large_batches_on_sampled_tokens(R, k, H):
    q, w, starts, rows = _inputs(R, k, H, seed=R + H)
    out = mla.query_absorb(q, w, angle_table(rows).cuda(), starts.cuda(), 6 / 448)
    T = R * k
    picks = sorted({0, 1, T // 3, T // 2, min(127, T - 1), min(128, T - 1), T - 1})
    _check(out, q, w, starts, k, True, 6 / 448, picks)
    # Every code against the 64-bit product: half a step (2^-4 relative, 2^-10 below the
    # smallest normal) plus the accumulation's error of the module docstring. That error does
    # not shrink with the sum: 2^-16 sum |q w| / scale is about 0.007 for these inputs
    # (sum |q w| near 6.4) beside 2^-10 for a sum that cancels.
    want = torch.einsum("thd,hdl->thl", q[..., :128].double(), w.double()) / (6 / 448)
    err = torch.einsum("thd,hdl->thl", q[..., :128].double().abs(), w.double().abs())
    err = err * (2.0 ** -16 / (6 / 448))
    got = out.view(torch.float8_e4m3fn)[..., :512].double()
    step = (torch.clamp(want.abs(), min=2.0 ** -6) + err) * 2.0 ** -4
    over = (got - want.clamp(-448, 448)).abs() - step - err
    assert float(over.max()) <= 0, float(over.max())
    # In the mean the accumulation is far nearer than that bound: 2^-10 beyond half a step.
    assert float(((got - want.clamp(-448, 448)).abs() - step).clamp(min=0).mean()) < 2.0 ** -10


@pytest.mark.parametrize("layout", ["wide", "heads first", "one head of many"])
def test_strided_queries(layout):
    R, k, H = 9, 3, 6
    q, w, starts, rows = _inputs(R, k, H, seed=1, stride=264)
    if layout == "heads first":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    elif layout == "one head of many":
        q, w, H = q[:, 2:3], w[2:3].contiguous(), 1
    out = mla.query_absorb(q, w, angle_table(rows).cuda(), starts.cuda(), 0.02)
    _check(out, q, w, starts, k, True, 0.02)


def test_padding_and_out_of_range_positions():
    R, k, H = 4, 2, 3
    q, w, starts, rows = _inputs(R, k, H, seed=2, rows=50)
    starts[1], starts[2] = -3, 49                 # padding; its second token is past the table
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mla.query_absorb(q, w, angle_table(50).cuda(), starts.cuda(), 0.02, status=status)
    assert int(status.item()) == mla.FAULT_ROPE_RANGE
    o = out.cpu().numpy()
    assert not o[2:4, :, 512:].any() and not o[5, :, 512:].any()
    _check(out, q, w, starts, k, True, 0.02, picks=[0, 1, 4, 6, 7])


def test_only_the_batch_is_written_and_the_result_repeats():
    R, k, H = 3, 5, 4
    q, w, starts, rows = _inputs(R, k, H, seed=4)
    rope = angle_table(rows).cuda()
    buf = torch.full((R * k + 20, H, 576), 9, dtype=torch.uint8, device="cuda")
    mla.query_absorb(q, w, rope, starts.cuda(), 0.02, out=buf[:R * k])
    assert (buf[R * k:] == 9).all()
    again = mla.query_absorb(q, w, rope, starts.cuda(), 0.02)
    assert torch.equal(again, buf[:R * k])


def test_special_values():
    """Infinities saturate, NaN stays in its own row, zeros give zeros."""
    q = torch.zeros((3, 1, 192), dtype=torch.bfloat16)
    q[0, 0, 0], q[1, 0, 0] = float("nan"), 1e30
    w = torch.zeros((1, 128, 512), dtype=torch.bfloat16)
    w[0, 0, :] = 1.0
    out = mla.query_absorb(q.cuda(), w.cuda(), angle_table(4).cuda(),
                           torch.zeros(1, dtype=torch.int32, device="cuda"), 1.0).cpu()
    assert (out[0, 0, :512] & 0x7F == 0x7F).all()
    assert (out[1, 0, :512] == 0x7E).all()
    assert not (out[2] & 0x7F).any()              # zeros, of either sign


def test_captured_replay_on_another_stream():
    R, k, H = 8, 4, 8
    q, w, starts, rows = _inputs(R, k, H, seed=6)
    rope, dev_starts = angle_table(rows).cuda(), starts.cuda()
    out = torch.empty((R * k, H, 576), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.query_absorb(q, w, rope, dev_starts, 0.02, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            mla.query_absorb(q, w, rope, dev_starts, 0.02, out=out)
        q2 = _inputs(R, k, H, seed=7)[0]
        q.copy_(q2)
        g.replay()
    torch.cuda.synchronize()
    _check(out, q2, w, starts, k, True, 0.02, picks=[0, 9, 31])
