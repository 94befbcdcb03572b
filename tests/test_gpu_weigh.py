"""Attention weights per cached key (mla_kv_weigh) against the oracle's sums, within the
bound of FP32 arithmetic that the oracle derives with them."""
import math

import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.cache as oc
from workloads import make_batch_from_lengths

pytestmark = pytest.mark.gpu

BAD = 1 << 30


def _lse(b, bmm1):
    """Base-2 LSEs of the batch's rows, rounded to FP32 (each request on the GPU in 64 bits)."""
    out = torch.full((b.R, b.M), -math.inf, dtype=torch.float64)
    val = lambda c: c.cuda().view(torch.float8_e4m3fn).double()  # noqa: E731
    for r, n in enumerate(b.seq_lens.tolist()):
        if n > 0:
            pages = b.block_table[r, :-(-n // 64)].long()
            keys = val(b.kv[pages]).reshape(-1, 576)[:n]
            x = val(b.q[r * b.k:(r + 1) * b.k]).reshape(-1, 576) @ keys.T * bmm1
            out[r] = (torch.logsumexp(x, 1) / math.log(2)).cpu()
    return out.float()


def _case(lens, k, H, seed=0, std=1.0):
    b = make_batch_from_lengths(lens, k, H, seed=seed, value_std=std, scaling="amax", fill=BAD)
    return b, float(np.float32(b.sm_scale * b.q_scale * b.kv_scale))


def _run(b, bmm1, lse, starts, *, decay=1.0, ahead=None, positions=True, seed=0, kv=None, stream=None,
         table=None, fault=0):
    rng = np.random.default_rng(seed)
    S = b.block_table.shape[1] * 64
    w0 = np.exp(rng.normal(size=(b.R, S))).astype(np.float32)
    p0 = rng.integers(0, 1000, (b.R, S)).astype(np.int32)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    w, p = torch.from_numpy(w0).cuda(), torch.from_numpy(p0).cuda()
    status = i32([0])
    torch.cuda.synchronize()
    mla.kv_weigh(b.q.cuda(), (b.kv if kv is None else kv).cuda(),
                 (b.block_table if table is None else table).cuda(), b.seq_lens.cuda(), lse.cuda(), bmm1,
                 w, i32(starts), decay=decay, positions=p if positions else None,
                 rope_starts=None if ahead is None else i32(ahead), status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status.item()) == fault
    return w.cpu().numpy(), p.cpu().numpy(), w0, p0


def _check(b, bmm1, lse, starts, got, *, decay=1.0, ahead=None, positions=True):
    w, p, w0, p0 = got
    sums, bounds = oc.key_weights(b.q.numpy(), b.kv.numpy(), np.where(b.block_table.numpy() == BAD, 0,
                                                                      b.block_table.numpy()),
                                  [0 if s < 0 else n for n, s in zip(b.seq_lens.tolist(), starts)],
                                  lse.numpy(), b.k, bmm1)
    for r in range(b.R):
        n = len(sums[r])
        j = np.arange(n)
        old = np.where(j < starts[r], np.float64(np.float32(decay)) * w0[r, :n], 0.0)
        want = old + sums[r]
        off = np.abs(w[r, :n] - want)
        tol = bounds[r] + want * 2.0 ** -22          # the product, the sum
        assert (off <= tol).all(), f"request {r}: {(off / tol).max()} of the bound at {(off / tol).argmax()}"
        assert np.array_equal(w[r, n:], w0[r, n:]), "entries behind the keys changed"
        new = (np.arange(p.shape[1]) >= starts[r]) & (np.arange(p.shape[1]) < n)
        first = starts[r] if ahead is None else ahead[r]
        pos = np.where(new & positions, first + np.arange(p.shape[1]) - starts[r], p0[r])
        assert np.array_equal(p[r], pos)


@pytest.mark.parametrize("k,H", [(1, 1), (1, 8), (4, 8), (7, 8), (1, 64), (1, 96), (5, 26), (7, 64)])
@pytest.mark.parametrize("lens", [(1,), (100, 37), (0, 63, 64, 65, 0, 127, 128, 129, 1, 0), (1024, 1100)])
def test_shapes(lens, k, H):
    b, bmm1 = _case(lens, k, H, seed=k * H + len(lens))
    starts = [max(0, n - k) for n in lens]
    lse = _lse(b, bmm1)
    _check(b, bmm1, lse, starts, _run(b, bmm1, lse, starts))


def test_more_rows_than_one_token_group():
    b, bmm1 = _case([200, 40], 32, 128, seed=5)
    lse = _lse(b, bmm1)
    _check(b, bmm1, lse, [200, 0], _run(b, bmm1, lse, [200, 0]))


def test_long_requests_are_cut_among_the_ctas():
    lens = [40000, 3, 9000, 0, 17]
    b, bmm1 = _case(lens, 2, 8, seed=6, std=0.7)
    lse = _lse(b, bmm1)
    starts = [n // 2 for n in lens]
    ahead = [70000 + n for n in lens]
    got = _run(b, bmm1, lse, starts, decay=0.5, ahead=ahead)
    _check(b, bmm1, lse, starts, got, decay=0.5, ahead=ahead)


def test_many_requests():
    rng = np.random.default_rng(7)
    lens = [int(v) for v in rng.integers(0, 200, 1024)]
    b, bmm1 = _case(lens, 1, 4, seed=7)
    lse = _lse(b, bmm1)
    starts = [n - n // 3 for n in lens]
    _check(b, bmm1, lse, starts, _run(b, bmm1, lse, starts))


def test_decay_and_no_positions():
    b, bmm1 = _case([300, 200], 3, 8, seed=8)
    lse = _lse(b, bmm1)
    for decay in (0.0, 0.9, 2.0):
        got = _run(b, bmm1, lse, [150, 200], decay=decay, positions=False)
        _check(b, bmm1, lse, [150, 200], got, decay=decay, positions=False)


def test_padding_requests_are_skipped():
    b, bmm1 = _case([100, 70, 129], 2, 8, seed=9)
    lse = _lse(b, bmm1)
    _check(b, bmm1, lse, [-1, 70, -5], _run(b, bmm1, lse, [-1, 70, -5]))


def test_rows_without_a_finite_lse_add_nothing():
    b, bmm1 = _case([100, 140], 4, 40, seed=10)
    lse = _lse(b, bmm1)
    lse[0, 3], lse[0, 159], lse[1, 0], lse[1, 81] = -math.inf, math.nan, math.inf, math.nan
    lse[0, 100:110] = -math.inf
    _check(b, bmm1, lse, [0, 0], _run(b, bmm1, lse, [0, 0]))


def test_nan_codes():
    """NaN codes behind a request's keys and in a row of queries reach no weight; a key of NaN
    codes gets no weight itself."""
    b, bmm1 = _case([100, 70], 2, 8, seed=11)
    lse = _lse(b, bmm1)
    want = _run(b, bmm1, lse, [0, 0])[0]
    kv = b.kv.clone()
    for r, n in enumerate((100, 70)):
        kv[b.block_table[r, n // 64], n % 64:] = 0x7F
    assert np.array_equal(_run(b, bmm1, lse, [0, 0], kv=kv)[0], want)
    kv[b.block_table[0, 0], 5] = 0x7F
    got = _run(b, bmm1, lse, [0, 0], kv=kv)[0]
    assert got[0, 5] == 0
    want[0, 5] = 0
    assert np.array_equal(got, want)
    b.q[1, 3] = 0xFF                               # row 11 of request 0
    cut = lse.clone()
    cut[0, 11] = -math.inf
    got = _run(b, bmm1, lse, [0, 0])[0]
    assert np.array_equal(got, _run(b, bmm1, cut, [0, 0])[0]) and np.isfinite(got).all()


def test_pages_outside_the_cache_are_zeros():
    b, bmm1 = _case([200, 70], 2, 8, seed=12)
    lse = _lse(b, bmm1)
    table = b.block_table.clone()
    table[0, 1] = b.kv.shape[0]
    got = _run(b, bmm1, lse, [0, 0], table=table, fault=mla.FAULT_PAGE_RANGE)
    zero = b.kv.clone()
    zero[b.block_table[0, 1]] = 0
    b.kv = zero
    _check(b, bmm1, lse, [0, 0], got)


def test_lengths_past_the_table_are_cut():
    b, bmm1 = _case([128], 1, 8, seed=13)
    lse = _lse(b, bmm1)
    want = _run(b, bmm1, lse, [0])
    b.seq_lens = torch.tensor([129], dtype=torch.int32)
    assert np.array_equal(_run(b, bmm1, lse, [0])[0], want[0])


def test_same_bits_every_time_and_on_another_stream():
    b, bmm1 = _case([5000, 333, 64], 7, 64, seed=14)
    lse = _lse(b, bmm1)
    starts = [4000, 0, 60]
    want = _run(b, bmm1, lse, starts)[0]
    assert np.array_equal(_run(b, bmm1, lse, starts)[0], want)
    assert np.array_equal(_run(b, bmm1, lse, starts, stream=torch.cuda.Stream())[0], want)


@pytest.mark.parametrize("k,H", [(4, 8), (7, 64)])
def test_weights_of_the_decodes_own_lse_sum_to_the_rows(k, H):
    b, bmm1 = _case([3000, 77, 640], k, H, seed=15)
    lens = b.seq_lens.cuda()
    eng = mla.FoldedMla(b.R, k, H, b.block_table.shape[1], b.kv.shape[0], "cuda")
    q, kv, table = b.q.cuda(), b.kv.cuda(), b.block_table.cuda()
    eng.plan(lens)
    _, lse = eng.decode(q, kv, table, lens, bmm1, b.kv_scale)
    w = torch.zeros((b.R, table.shape[1] * 64), device="cuda")
    mla.kv_weigh(q, kv, table, lens, lse, bmm1, w, torch.zeros_like(lens))
    # The decode's LSEs are within 1e-3 (base 2), its tests' bound: a row gives 1 within 7e-4.
    assert (w.double().sum(1) / (k * H) - 1).abs().max() < 7.1e-4


def test_a_wait_that_runs_out_is_reported():
    for k, H in ((4, 8), (7, 64)):
        b, bmm1 = _case([2000, 333], k, H, seed=16)
        lse = _lse(b, bmm1).cuda()
        S = b.block_table.shape[1] * 64
        q, kv, table, lens = b.q.cuda(), b.kv.cuda(), b.block_table.cuda(), b.seq_lens.cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        starts = torch.zeros_like(lens)
        w = torch.full((2, S), -1.0, device="cuda")
        mla.kv_weigh_wait_test(q, kv, table, lens, lse, bmm1, w, starts, status, 20_000_000)
        torch.cuda.synchronize()
        assert int(status.item()) == mla.FAULT_WAIT_TIMEOUT
        assert (w[0, :64] == -1).all() and (w[1, 200:333] > 0).all()   # CTA 0 wrote nothing
        mla.kv_weigh(q, kv, table, lens, lse, bmm1, w, starts)
        assert (w.double().sum(1)[0] - k * H - (S - 2000) * -1.0).abs() < 1e-2 * k * H


def test_a_captured_call():
    b, bmm1 = _case([700, 64], 4, 8, seed=17)
    lse = _lse(b, bmm1)
    want = _run(b, bmm1, lse, [0, 0])[0]
    q, kv, table, lens, l = (t.cuda() for t in (b.q, b.kv, b.block_table, b.seq_lens, lse))
    w, starts = torch.zeros((2, table.shape[1] * 64), device="cuda"), torch.zeros_like(lens)
    g = torch.cuda.CUDAGraph()
    mla.kv_weigh(q, kv, table, lens, l, bmm1, w, starts)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mla.kv_weigh(q, kv, table, lens, l, bmm1, w, starts)
    w.zero_()
    g.replay()
    torch.cuda.synchronize()
    got = w.cpu().numpy()
    assert np.array_equal(got[0, :700], want[0, :700]) and np.array_equal(got[1, :64], want[1, :64])
