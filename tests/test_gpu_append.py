"""New tokens into the paged cache (mla_kv_append) against the oracle's rows.

Tolerance: a code must be the E4M3 rounding of some value within the FP32
arithmetic's error of the exact one. That error: latent dims, the sum of 512
squares in FP32 (16 per lane, then 5 joins: < 2^-19 relative), rsqrt (2^-22),
four products (2^-24 each), half of the sum's error through the root: below
2^-18 of the value; rope dims, two products of FP32 angles' cosines (2^-24
each) and their sum: below 2^-21 (|a| + |b|) of the plane's coordinates.
"""
import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.step as st
from tests.step_util import angle_table, assert_codes

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _run(starts, new, *, ragged, stride=576, norm=True, interleaved=True, ahead=0, extra_rows=0,
         scale=0.02, seed=0, offset=0):
    rng = np.random.default_rng(seed)
    R = len(starts)
    T = sum(new) + extra_rows
    need = [-(-(max(s, 0) + n) // 64) for s, n in zip(starts, new)]
    pages, width = sum(need) + 3, max(1, max(need))
    perm = rng.permutation(pages)
    table = np.full((R, width), 1 << 30, dtype=np.int32)         # unread entries are bad pages
    at = 0
    for r in range(R):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
    wide = rng.normal(size=(max(T, 1), stride)).astype(np.float32)
    wide *= np.exp(rng.normal(size=(max(T, 1), 1))).astype(np.float32)
    wide = torch.from_numpy(wide).to(torch.bfloat16).cuda()
    x = wide[:T, offset:offset + 576]
    w = torch.from_numpy((1 + 0.2 * rng.normal(size=512)).astype(np.float32)).to(torch.bfloat16)
    kv = torch.from_numpy(rng.integers(0, 0x7F, size=(pages, 64, 576)).astype(np.uint8))
    before = kv.numpy().copy()
    kv = kv.cuda()
    rows = ahead + max([max(s, 0) + n for s, n in zip(starts, new)]) + 1
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    dev_starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.kv_append(x, kv, torch.from_numpy(table).cuda(), dev_starts, angle_table(rows).cuda(),
                  scale, norm_weight=w.cuda() if norm else None, norm_eps=EPS,
                  cu_tokens=cu if ragged else None,
                  rope_starts=dev_starts + ahead if ahead else None, interleaved=interleaved,
                  status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = kv.cpu().numpy()
    xs, ws = x.float().cpu().numpy().astype(np.float64), w.float().numpy()
    t = 0
    written = np.zeros((pages, 64), dtype=bool)
    ys, es, cs = [], [], []
    for r, (s, n) in enumerate(zip(starts, new)):
        for i in range(n):
            if s >= 0:
                j = s + i
                y = st.cache_row(xs[t], ws if norm else None, EPS, ahead + j, interleaved, scale)
                e = 2.0 ** -18 * np.abs(y)
                pe = np.abs(xs[t, 512:])
                pair = pe.reshape(32, 2).sum(1).repeat(2) if interleaved else \
                    np.tile(pe[:32] + pe[32:], 2)
                e[512:] = 2.0 ** -21 * pair / scale
                page, slot = table[r, j // 64], j % 64
                written[page, slot] = True
                ys.append(y)
                es.append(e)
                cs.append(got[page, slot])
            t += 1
    if ys:
        assert_codes(np.stack(cs), np.stack(ys), np.stack(es))
    assert np.array_equal(got[~written], before[~written]), "other cache rows changed"


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("starts,k", [((0,), 1), ((37, 100), 4), ((63, 64, 0, 127, 1), 7),
                                      ((5,) * 33, 3)])
def test_decode_step(starts, k, norm, interleaved):
    _run(starts, [k] * len(starts), ragged=False, norm=norm, interleaved=interleaved,
         seed=k + len(starts))


@pytest.mark.parametrize("new,extra", [((1,), 0), ((0, 5, 0, 0, 130, 1, 0), 9), ((64, 65, 63), 1),
                                       ((0, 0, 0), 4), ((3,) * 70, 0), (tuple(range(40)), 2)])
def test_ragged_prompts_leave_the_rows_behind_them(new, extra):
    rng = np.random.default_rng(len(new))
    _run([int(v) for v in rng.integers(0, 200, len(new))], list(new), ragged=True,
         extra_rows=extra, seed=sum(new))


def test_many_ragged_requests():
    rng = np.random.default_rng(8)
    new = [int(v) for v in rng.integers(0, 3, 1500)]
    _run([int(v) for v in rng.integers(0, 3, 1500)], new, ragged=True, seed=1)


@pytest.mark.parametrize("stride,offset", [(584, 0), (584, 8), (2112, 1536), (1000, 424)])
def test_strided_rows(stride, offset):
    _run((10, 70, 0), [5, 5, 5], ragged=False, stride=stride, offset=offset, seed=stride)


def test_far_positions():
    _run((0, 63, 500), [4, 4, 4], ragged=False, ahead=130000, seed=2)


def test_padding_requests_are_skipped():
    _run((-1, 3, -7, 0), [2, 2, 2, 2], ragged=False, seed=3)
    _run((-1, 3, -7, 0), [2, 0, 4, 3], ragged=True, seed=4)


def test_saturation():
    _run((0, 9), [3, 3], ragged=False, scale=1e-4, seed=5)


def test_special_values_without_norm():
    x = torch.zeros(1, 576, dtype=torch.bfloat16)
    x[0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0])
    kv = torch.full((1, 64, 576), 7, dtype=torch.uint8, device="cuda")
    mla.kv_append(x.cuda(), kv, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                  torch.zeros(1, dtype=torch.int32, device="cuda"), angle_table(1).cuda(), 1.0)
    row = kv[0, 0].cpu()
    assert row[:2].tolist() == [0x7E, 0xFE] and int(row[2]) & 0x7F == 0x7F
    assert not (row[3:] & 0x7F).any() and (kv[0, 1:] == 7).all()


def _small(R=2, k=3, pages=4, width=2):
    x = torch.randn(R * k, 576, device="cuda").to(torch.bfloat16)
    kv = torch.full((pages, 64, 576), 9, dtype=torch.uint8, device="cuda")
    table = torch.arange(R * width, dtype=torch.int32, device="cuda").view(R, width)
    return x, kv, table


def test_out_of_range_tokens_are_reported_and_skipped():
    x, kv, table = _small()
    rope = angle_table(200).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # Request 0 runs off its block-table row after one token, request 1 is fine.
    mla.kv_append(x, kv, table, i32(127, 0), rope, 0.05, status=status)
    assert int(status.item()) == mla.FAULT_PAGE_RANGE
    changed = (kv != 9).any(-1).cpu()
    assert changed[1, 63] and changed[2, :3].all() and int(changed.sum()) == 4
    # A page outside the cache.
    kv.fill_(9)
    status.zero_()
    table[0, 0] = 4
    table[1, 0] = -1
    mla.kv_append(x, kv, table, i32(0, 0), rope, 0.05, status=status)
    assert int(status.item()) == mla.FAULT_PAGE_RANGE and (kv == 9).all()
    # Positions outside the table of angles.
    table[0, 0], table[1, 0] = 0, 2
    status.zero_()
    mla.kv_append(x, kv, table, i32(0, 0), rope, 0.05, rope_starts=i32(-1, 199), status=status)
    assert int(status.item()) == mla.FAULT_ROPE_RANGE
    changed = (kv != 9).any(-1).cpu()
    assert changed[0, 1:3].all() and changed[2, 0] and int(changed.sum()) == 3
    # Without a status word the same calls skip the same tokens.
    kv.fill_(9)
    mla.kv_append(x, kv, table, i32(0, 0), rope, 0.05, rope_starts=i32(500, 500))
    assert (kv == 9).all()


def test_ragged_offsets_out_of_order_stay_in_bounds():
    """Offsets that are no offsets (descending, negative, past the rows): every
    row goes to a request whose range holds it, or nowhere."""
    x, kv, table = _small()
    rope = angle_table(200).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for cu in ((5, 2, 9), (-4, 100, 3), (7, 7, 7), (0, 3, 1)):
        mla.kv_append(x, kv, table, i32(0, 0), rope, 0.05, cu_tokens=i32(*cu))
    torch.cuda.synchronize()


@pytest.mark.parametrize("cu", [(5, 2, 9), (-4, 100, 3), (7, 7, 7), (0, 3, 1), (0, 4, 6), (2, 6, 6),
                                (-(1 << 31), 6, 6), (2 - (1 << 31), 6, 6), (-(1 << 31), 1, 6),
                                (0, -(1 << 31), 6), ((1 << 31) - 1, -(1 << 31), 6),
                                (-1, (1 << 31) - 1, (1 << 31) - 1)])
def test_ragged_offsets_change_only_their_own_rows(cu):
    """Whatever the offsets: a token leaves nothing but the cache row of a request whose
    offsets hold it, and the pages beside the cache's stay. Offsets far below 0 put a
    token past every table: it is skipped and reported."""
    starts = (0, 70)
    x, _, table = _small()
    around = torch.full((12, 64, 576), 9, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mla.kv_append(x, around[4:8], table, i32(starts), angle_table(200).cuda(), 0.05,
                  cu_tokens=i32(cu), status=status)
    torch.cuda.synchronize()
    changed = {tuple(v) for v in (around != 9).any(-1).nonzero().tolist()}
    may, faults = set(), 0
    for t in range(6):
        for r in range(2):
            if cu[r] <= t < cu[r + 1]:
                j = starts[r] + t - cu[r]
                if j < 128:
                    may.add((4 + 2 * r + j // 64, j % 64))
                faults |= (mla.FAULT_PAGE_RANGE if j >= 128 else 0) | \
                    (mla.FAULT_ROPE_RANGE if j >= 200 else 0)
    assert changed <= may
    if cu == (0, 4, 6):
        assert changed == may and len(may) == 6
    assert int(status.item()) & ~faults == 0
    if cu[0] < -1000 and cu[1] == 6:              # past its block-table row and the angles
        assert not changed
        assert int(status.item()) == mla.FAULT_PAGE_RANGE | mla.FAULT_ROPE_RANGE


@pytest.mark.parametrize("scale,eps", [(1e-37, 1e-6), (3e-39, 1e-6), (1e-30, 0.0), (1e37, 1e-6)])
def test_scales_at_the_ends_of_fp32(scale, eps):
    """A scale whose reciprocal is near FP32's end, beside rows whose norm is far from 1:
    zeros stay zeros, the rest saturates or vanishes as its exact value does."""
    x = torch.zeros(3, 576, dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 2] = 1e-15, -1e-15, 1e-38
    x[1, :2] = torch.tensor([1.0, -2e-37])
    x[2, 512:514] = torch.tensor([3e-38, -1.0])
    x[2, 0] = 1.0
    w = torch.ones(512, dtype=torch.bfloat16)
    w[5] = 0.0
    kv = torch.full((1, 64, 576), 7, dtype=torch.uint8, device="cuda")
    i32 = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = torch.cat([torch.ones(4, 32), torch.zeros(4, 32)], 1).cuda()       # no turn
    mla.kv_append(x.cuda(), kv, i32[None], i32, rope, scale, norm_weight=w.cuda(), norm_eps=eps)
    got = kv[0, :3].cpu().numpy()
    xs, ws = x.double().numpy(), w.double().numpy()
    scale = float(np.float32(scale))
    y = np.stack([st.cache_row(xs[t], ws, float(np.float32(eps)), 0, True, scale) for t in range(3)])
    # As for the other rows, and the two products before the scale's, each within half of
    # FP32's smallest step where they are that small.
    assert_codes(got, y, 2.0 ** -18 * np.abs(y) + 2.0 ** -149 / scale)
    assert not (got[:, 5] & 0x7F).any()


def test_no_tokens_launch_nothing():
    x, kv, table = _small()
    mla.kv_append(x[:0], kv, table, torch.zeros(2, dtype=torch.int32, device="cuda"),
                  angle_table(4).cuda(), 1.0)
    torch.cuda.synchronize()
    assert (kv == 9).all()


def test_rows_past_2_31_bytes_of_cache():
    """The last page of a cache of more than 2^31 bytes."""
    pages = (1 << 31) // (64 * 576) + 5
    kv = torch.empty((pages, 64, 576), dtype=torch.uint8, device="cuda")
    kv[-1].fill_(9)
    x = torch.randn(2, 576, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    mla.kv_append(x, kv, table, torch.tensor([62], dtype=torch.int32, device="cuda"),
                  angle_table(64).cuda(), 0.05)
    assert (kv[-1, 62:] != 9).any(-1).all() and (kv[-1, :62] == 9).all()


def test_captured_replay_on_another_stream():
    """One graph replayed with new inputs in its buffers, on a side stream."""
    x, kv, table = _small()
    rope = angle_table(300).cuda()
    starts = torch.zeros(2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mla.kv_append(x, kv.clone(), table, starts, rope, 0.05)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            mla.kv_append(x, kv, table, starts, rope, 0.05)
            starts += 3
        for _ in range(3):
            x.copy_(torch.randn_like(x))
            g.replay()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    changed = (kv != 9).any(-1).cpu()
    assert starts.tolist() == [9, 9]
    assert changed[0, :9].all() and changed[2, :9].all() and int(changed.sum()) == 18
