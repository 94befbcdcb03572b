"""Eviction by accumulated weight (mla_kv_evict) against the oracle: every value exact."""
import math

import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.cache as oc

pytestmark = pytest.mark.gpu


def _weights(rng, shape, kind):
    w = np.exp(2 * rng.normal(size=shape)).astype(np.float32)
    if kind == "ties":
        w = np.float32(2.0) ** rng.integers(-2, 2, shape).astype(np.float32)
    elif kind == "equal":
        w = np.full(shape, 0.25, dtype=np.float32)
    elif kind == "odd":                       # NaN, infinities, both zeros, negatives, subnormals
        pick = np.array([math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, -1.5, 1e-42, -1e-42, 3.0],
                        dtype=np.float32)
        w = np.where(rng.random(shape) < 0.7, pick[rng.integers(0, len(pick), shape)], w)
    elif kind == "close":                     # neighbours in FP32
        w = (np.float32(1.0).view(np.int32) + rng.integers(0, 40, shape).astype(np.int32)).view(np.float32)
    return w


def _run(lens, keep, *, recent=0, sinks=0, kind="plain", mixed=False, positions=True, in_place=False,
         seed=0, width=None, bad=(), spare=0, workspace=False, stream=None):
    """Evicts and compares everything; returns nothing."""
    rng = np.random.default_rng(seed)
    R = len(lens)
    need = [-(-max(n, 0) // 64) for n in lens]
    width = width or max(1, max(need))
    need = [min(v, width) for v in need]
    pages = sum(need) + 3 + spare
    perm = rng.permutation(pages)
    table = np.full((R, width), 1 << 30, dtype=np.int32)
    at = 0
    for r in range(R):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
    S = width * 64
    w0 = _weights(rng, (R, S), kind)
    p0 = np.tile(np.arange(S, dtype=np.int32), (R, 1))
    if mixed:
        for r in range(R):
            p0[r] = rng.permutation(S) * 3 - 5
    kv0 = torch.randint(0, 256, (pages, 64, 576), generator=torch.Generator().manual_seed(seed),
                        dtype=torch.uint8).numpy()
    true_table = table.copy()
    for r, page in bad:
        table[r, page] = -7
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv, w, p, n, status = dev(kv0), dev(w0), dev(p0), i32(lens), i32([0])
    wo, po, no = torch.full_like(w, -3.0), torch.full_like(p, -9), torch.full_like(n, -2)
    args = dict(positions=p if positions else None, recent=recent, sinks=sinks, status=status)
    if workspace:
        args["workspace"] = torch.randint(0, 255, (mla.kv_evict_workspace_bytes(R, width),),
                                          dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    if in_place:
        got = mla.kv_evict(kv, dev(table), n, w, i32(keep), lens_out=n, stream=stream, **args)
        assert got is n
        wo, po, no, wb, pb = w, p, n, w0, p0
    else:
        no = mla.kv_evict(kv, dev(table), n, w, i32(keep), weights_out=wo,
                          positions_out=po if positions else None, stream=stream, **args)
        wb, pb = np.full_like(w0, -3.0), np.full_like(p0, -9)
    torch.cuda.synchronize()
    if not in_place:
        assert np.array_equal(w.cpu().numpy(), w0, equal_nan=True) and np.array_equal(p.cpu().numpy(), p0)
        assert n.cpu().tolist() == list(lens)
    want_w, want_p, want_kv, want_n, moved_bad = wb.copy(), pb.copy(), kv0.copy(), [], False
    for r in range(R):
        m = min(max(lens[r], 0), S)
        kept, moves = oc.evict(m, w0[r], p0[r] if positions else range(S), keep[r], recent, sinks)
        new = len(kept)
        want_n.append(new)
        to = dict(moves)
        for j in kept:
            want_w[r, to.get(j, j)], want_p[r, to.get(j, j)] = w0[r, j], p0[r, j]
        want_w[r, new:m], want_p[r, new:m] = 0.0, -1
        for a, b in moves:
            if table[r, a // 64] < 0 or table[r, b // 64] < 0:
                moved_bad = True
                continue
            want_kv[true_table[r, b // 64], b % 64] = kv0[true_table[r, a // 64], a % 64]
    assert no.cpu().tolist() == want_n
    assert np.array_equal(wo.cpu().numpy().view(np.int32), want_w.view(np.int32)), "weights"
    if positions:
        assert np.array_equal(po.cpu().numpy(), want_p), "positions"
    assert np.array_equal(kv.cpu().numpy(), want_kv), "cache rows"
    over = any(n > S for n in lens)
    assert int(status.item()) == (mla.FAULT_PAGE_RANGE if moved_bad or over else 0)


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd", "close"])
@pytest.mark.parametrize("in_place", [False, True])
def test_ragged_batch(kind, in_place):
    lens = [100, 0, 1, 64, 65, 700, 37, 500, 128, 333]
    keep = [60, 5, 1, 63, 64, 100, 40, 499, 0, 1]
    for mixed in (False, True):
        _run(lens, keep, recent=7, sinks=3, kind=kind, mixed=mixed, in_place=in_place, seed=len(kind))


@pytest.mark.parametrize("recent,sinks", [(0, 0), (1, 0), (0, 1), (50, 50), (400, 4), (1 << 30, 0),
                                          (0, 1 << 30), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_held_keys(recent, sinks):
    for mixed in (False, True):
        _run([300, 20, 301], [100, 50, 150], recent=recent, sinks=sinks, mixed=mixed, seed=recent % 97)
    _run([300, 20, 301], [100, 50, 150], recent=recent, sinks=sinks, positions=False)


def test_keep_all_none_and_negative():
    _run([200, 200, 200, 0, -4, 200], [200, 0, -5, 0, 3, 2 ** 31 - 1], recent=5, sinks=5)
    _run([200, 200, 200], [199, 1, 2], recent=5, sinks=5, in_place=True)


def test_a_decode_steps_few_keys():
    _run([2055] * 40, [2048] * 40, recent=64, sinks=4, mixed=True, seed=2)
    _run([2055] * 40, [2048] * 40, recent=64, sinks=4, mixed=True, seed=3, in_place=True)


@pytest.mark.parametrize("n", [4096, 4097, 8192, 9000, 30000, 131072])
def test_long_requests_on_clusters(n):
    _run([n, n // 3], [n // 2, n // 9], recent=100, sinks=4, mixed=True, seed=n, width=-(-n // 64))
    _run([n], [n // 2], kind="ties", seed=n + 1, in_place=True)


@pytest.mark.parametrize("R,width", [(3, 2048), (100, 700), (5, 12000)])
def test_short_requests_in_wide_tables(R, width):
    rng = np.random.default_rng(width)
    lens = [int(v) for v in rng.integers(0, 300, R)]
    _run(lens, [v // 2 for v in lens], recent=9, sinks=1, kind="ties", seed=R, width=width, mixed=True)


def test_clusters_of_every_size():
    for R, width in ((80, 130), (70, 70), (38, 130), (19, 300), (9, 600), (4, 1100)):
        rng = np.random.default_rng(R)
        lens = [int(v) for v in rng.integers(0, width * 64 + 1, R)]
        _run(lens, [n // 2 + 1 for n in lens], recent=33, sinks=2, kind="ties", seed=R, width=width)


def test_more_keys_than_shared_memory_holds():
    """Beyond 655,360 slots the codes are made anew in every pass."""
    n = 700_001
    rng = np.random.default_rng(1)
    S = -(-n // 64) * 64
    w0 = np.exp(rng.normal(size=(1, S))).astype(np.float32)
    p0 = rng.permutation(S).astype(np.int32)[None]
    table = rng.permutation(S // 64).astype(np.int32)[None]
    kv = torch.randint(0, 256, (S // 64, 64, 576), dtype=torch.uint8, device="cuda")
    before = kv.clone()
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    w, p, lens = dev(w0.copy()), dev(p0.copy()), torch.tensor([n], dtype=torch.int32, device="cuda")
    keep = torch.tensor([300_000], dtype=torch.int32, device="cuda")
    new = mla.kv_evict(kv, dev(table), lens, w, keep, positions=p, recent=1000, sinks=10)
    torch.cuda.synchronize()
    kept, moves = oc.evict(n, w0[0], p0[0], 300_000, 1000, 10)
    assert new.tolist() == [300_000]
    want = w0[0].copy()
    want[300_000:n] = 0
    src, dst = (np.array(v) for v in zip(*moves))
    want[dst] = w0[0][src]
    assert np.array_equal(w.cpu().numpy()[0], want)
    rows = lambda j: dev(table[0].astype(np.int64)[j // 64] * 64 + j % 64)  # noqa: E731
    flat = before.view(-1, 576)
    flat[rows(dst)] = before.view(-1, 576)[rows(src)]
    assert torch.equal(kv.view(-1, 576), flat)


def test_bad_pages_are_reported_and_not_touched():
    _run([400, 400], [100, 100], seed=5, bad=[(0, 1), (1, 4)])
    _run([400, 400], [100, 100], seed=6, bad=[(0, 0), (0, 5)], in_place=True)


def test_lengths_past_the_table():
    _run([400, 130], [100, 100], seed=7, width=2)


def test_workspace_of_the_callers():
    _run([400, 90, 1000], [100, 100, 10], seed=8, workspace=True, recent=9)


def test_another_stream():
    _run([3000, 90, 1000], [100, 100, 10], seed=9, stream=torch.cuda.Stream())


def test_many_requests():
    rng = np.random.default_rng(10)
    lens = [int(v) for v in rng.integers(0, 130, 1024)]
    _run(lens, [int(v) for v in rng.integers(0, 130, 1024)], recent=5, sinks=1, seed=11)


def test_a_captured_call_replayed():
    rng = np.random.default_rng(12)
    S = 320
    kv = torch.randint(0, 256, (10, 64, 576), dtype=torch.uint8, device="cuda")
    table = torch.randperm(10, device="cuda").int().view(2, 5)
    w, p = torch.zeros((2, S), device="cuda"), torch.zeros((2, S), dtype=torch.int32, device="cuda")
    lens, keep = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([50, 70], dtype=torch.int32,
                                                                              device="cuda")
    mla.kv_evict(kv, table, lens, w, keep, positions=p, recent=3, lens_out=lens)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.kv_evict(kv, table, lens, w, keep, positions=p, recent=3, lens_out=lens)
    for turn in range(3):
        w0 = np.exp(rng.normal(size=(2, S))).astype(np.float32)
        p0 = np.stack([rng.permutation(S), rng.permutation(S)]).astype(np.int32)
        n0 = [int(v) for v in rng.integers(0, S, 2)]
        w.copy_(torch.from_numpy(w0))
        p.copy_(torch.from_numpy(p0))
        lens.copy_(torch.tensor(n0, dtype=torch.int32))
        before = kv.clone()
        g.replay()
        torch.cuda.synchronize()
        want = before.view(-1, 576).clone()
        for r in range(2):
            kept, moves = oc.evict(n0[r], w0[r], p0[r], [50, 70][r], 3, 0)
            assert int(lens[r]) == len(kept)
            for a, b in moves:
                t = table[r].tolist()
                want[t[b // 64] * 64 + b % 64] = before.view(-1, 576)[t[a // 64] * 64 + a % 64]
        assert torch.equal(kv.view(-1, 576), want)
