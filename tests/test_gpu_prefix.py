"""The decode of a batch behind a shared prefix (mla_prefix_decode) against the
oracle.

Tolerance per output, with A = softmax-weighted mean of |v| and Z the sum of
the row's weights over its largest: the weights enter the PV product in two
8-bit terms, within 2^-7 relative and 2^-13 absolute of FP32 weights that are
at least 4 at the largest (so 2^-13 sum |v| / (4 Z)); scores and sums in FP32
move a weight by less than 2^-11; the result is rounded to BF16 once (2^-8 of
it at most):
    |err| <= (2^-7 + 2^-11) A + 2^-15 sum |v| / Z + 2^-8 |ref| + 1e-6.
A and Z are taken from the exact weights. The LSE moves by less
than 2^-11 base-2 units through the scores: 1e-3.
"""
import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.step as st
from tests.gpu_util import bmm_scales, to_device
from tests.step_util import prefix_batch

pytestmark = pytest.mark.gpu


def _decode(b, table, prefix, *, num_ctas=None, extra_prefix_pages=0, return_lse=True):
    d = to_device(b)
    pt = torch.cat([table, torch.full((extra_prefix_pages,), 1 << 30, dtype=torch.int32)]).cuda()
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], pt.numel(), d["kv"].shape[0], "cuda",
                        num_ctas=num_ctas)
    bmm1, bmm2 = bmm_scales(b)
    eng.plan(d["lens"])
    out, lse = eng.decode(d["q"], d["kv"], pt, torch.tensor([prefix], dtype=torch.int32).cuda(),
                          d["bt"], d["lens"], bmm1, bmm2, return_lse=return_lse)
    torch.cuda.synchronize()
    assert int(eng.status.item()) == 0
    return out, lse


def _check(out, lse, b, table, prefix, what=""):
    ro, rl, spread, reach = st.prefix_decode(b.q.numpy(), b.kv.numpy(), table.numpy(), prefix,
                                     b.block_table.numpy(), b.seq_lens.numpy(), b.k, b.sm_scale,
                                     b.q_scale, b.kv_scale)
    bound = (2.0 ** -7 + 2.0 ** -11) * spread + 2.0 ** -15 * reach + \
        2.0 ** -8 * np.abs(ro) + 1e-6
    o = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(o).all(), what
    excess = np.abs(o - ro) - bound
    assert excess.max() <= 0, f"{what}: out over its bound by {excess.max():.3e}"
    if lse is not None:
        l = lse.cpu().numpy().astype(np.float64)
        inf = np.isneginf(rl)
        assert np.array_equal(np.isneginf(l), inf) and np.abs(l[~inf] - rl[~inf]).max(initial=0) <= 1e-3


@pytest.mark.parametrize("k,H", [(1, 1), (4, 8), (7, 8), (1, 64), (4, 64), (3, 5)])
@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 128, 129, 300, 1000])
def test_against_the_oracle(prefix, k, H):
    b, table, n = prefix_batch((100, 0, 37, 64), k, H, prefix, seed=prefix + k * H,
                               fill=1 << 30)
    out, lse = _decode(b, table, n, extra_prefix_pages=prefix % 3)
    _check(out, lse, b, table, n)


@pytest.mark.parametrize("lens", [(0, 0, 0), (0,), (1,), (700,), (5, 0, 1, 400, 64, 63, 65, 129),
                                  (5000, 2048, 0, 1793, 2304)])
def test_own_keys_of_any_length(lens):
    b, table, n = prefix_batch(lens, 4, 8, 333, seed=sum(lens))
    for ctas in (None, 6):
        _check(*_decode(b, table, n, num_ctas=ctas), b, table, n, f"{ctas} CTAs")


def test_empty_prefix_and_rows_without_keys():
    b, table, _ = prefix_batch((0, 70, 0, 500), 4, 8, 64, seed=9)
    out, lse = _decode(b, table, 0)
    _check(out, lse, b, table, 0)
    assert not out[0].any() and torch.isneginf(lse[0]).all() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 20, 151, 152, 500])
@pytest.mark.parametrize("R,k,H,prefix", [(3, 4, 8, 5000), (9, 7, 8, 2500), (5, 1, 64, 1500)])
def test_any_number_of_ctas(R, k, H, prefix, num_ctas):
    rng = np.random.default_rng(num_ctas)
    b, table, n = prefix_batch([int(v) for v in rng.integers(0, 600, R)], k, H, prefix,
                               seed=num_ctas * R)
    _check(*_decode(b, table, n, num_ctas=num_ctas), b, table, n)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    R, k = int(rng.integers(1, 12)), int(rng.integers(1, 8))
    H = int(rng.choice([1, 2, 3, 8, 12, 16, 33, 64]))
    prefix = int(np.exp(rng.uniform(0, np.log(4000))))
    lens = [int(v) for v in rng.integers(0, int(rng.choice([2, 70, 900])), R)]
    std = float(rng.choice([0.5, 1.0]))
    b, table, n = prefix_batch(lens, k, H, prefix, seed=seed, std=std,
                               scaling="unit" if seed % 3 == 0 else "amax")
    what = f"R={R} k={k} H={H} prefix={prefix} lens={lens}"
    out, lse = _decode(b, table, n, num_ctas=[None, 5, 40][seed % 3],
                       return_lse=seed % 4 != 0)
    _check(out, lse, b, table, n, what)


def test_scores_far_apart():
    """Prefix keys that dominate, then own keys that dominate: the other side's
    weights vanish without a trace."""
    for big in ("prefix", "own"):
        b, table, n = prefix_batch((200, 130), 2, 8, 400, seed=11)
        kv = b.kv.view(torch.float8_e4m3fn).float()
        pages = table.long() if big == "prefix" else b.block_table[b.block_table >= 0].long()
        kv[pages] = (kv[pages] * 6).clamp(-448, 448)
        b.kv = kv.to(torch.float8_e4m3fn).view(torch.uint8)
        _check(*_decode(b, table, n), b, table, n, big)


@pytest.mark.parametrize("k,H", [(4, 8), (1, 64), (7, 33)])
def test_scores_that_grow_from_tile_to_tile(k, H):
    """Every few pages the keys double: the running max moves in the middle of a
    piece, again and again, and the sums follow."""
    b, table, n = prefix_batch((700, 0, 1500), k, H, 3000, seed=21 + H)
    kv = b.kv.view(torch.float8_e4m3fn).float() / 64
    for row in [table] + list(b.block_table):
        for i, page in enumerate(row.tolist()):
            kv[page] = kv[page] * 2.0 ** min(6, i // 7)
    b.kv = kv.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for ctas in (None, 2, 7):
        _check(*_decode(b, table, n, num_ctas=ctas), b, table, n, f"{ctas} CTAs")


@pytest.mark.parametrize("spots", [(261,), (390,), (261, 390), (390, 520), (767, 768), (900, 130)])
@pytest.mark.parametrize("k,H", [(4, 8), (3, 64)])
def test_one_key_that_tops_all_before_it(spots, k, H):
    """A key along some rows' queries, each later one longer, in the first or the second
    128 keys of a tile: the maximum of a few rows moves there, in one half or in both."""
    b, table, n = prefix_batch((700, 0, 300), k, H, 1000, seed=31)
    kv = b.kv.view(torch.float8_e4m3fn).float() / 16
    q = b.q.view(torch.float8_e4m3fn).float()
    for i, j in enumerate(sorted(spots)):
        kv[table[j // 64], j % 64] = q[i % q.shape[0], i % H] * 0.25 * 2 ** i
        for r in range(3):
            if j < int(b.seq_lens[r]):
                kv[b.block_table[r, j // 64], j % 64] = q[k * r, i % H] * 0.25 * 2 ** i
    b.kv = kv.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for ctas in (None, 2):
        _check(*_decode(b, table, n, num_ctas=ctas), b, table, n, f"{ctas} CTAs")


def test_a_row_of_nan_stays_alone():
    b, table, n = prefix_batch((100, 300), 4, 8, 600, seed=22)
    clean = b.q.clone()
    b.q[2, 3] = 0x7F
    out, lse = _decode(b, table, n)
    bad = 2 * 8 + 3                              # row of request 0
    assert out[0, bad].isnan().all() and not lse[0, bad].isfinite()
    b.q = clean
    good = torch.ones(b.R, b.M, dtype=torch.bool)
    good[0, bad] = False
    again, lse2 = _decode(b, table, n)
    assert torch.equal(out.cpu()[good], again.cpu()[good]) and torch.equal(lse.cpu()[good], lse2.cpu()[good])


def test_pages_past_2_31_bytes_of_cache():
    b, table, n = prefix_batch((100, 300), 4, 8, 600, seed=23)
    used, far = b.kv.shape[0], (1 << 31) // (64 * 576) + 7
    d = to_device(b)
    kv = torch.empty((far + used, 64, 576), dtype=torch.uint8, device="cuda")
    kv[far:] = d["kv"]
    bmm1, bmm2 = bmm_scales(b)
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), far + used, "cuda")
    eng.plan(d["lens"])
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = eng.decode(d["q"], kv, table.cuda() + far, plen, d["bt"] + far, d["lens"], bmm1, bmm2)
    assert int(eng.status.item()) == 0
    _check(out, lse, b, table, n)


def test_two_batches_on_two_streams():
    """Two engines, each on its own stream, many times over: neither disturbs the other."""
    jobs = []
    for seed, (lens, prefix) in enumerate((((100, 700, 0), 900), ((64, 5), 2500))):
        b, table, n = prefix_batch(lens, 4, 8, prefix, seed=24 + seed)
        d = to_device(b)
        eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda")
        jobs.append((b, table, n, d, eng, table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    results = []
    for _ in range(20):
        results = []
        for b, table, n, d, eng, pt, plen, stream in jobs:
            bmm1, bmm2 = bmm_scales(b)
            eng.plan(d["lens"], stream)
            results.append(eng.decode(d["q"], d["kv"], pt, plen, d["bt"], d["lens"], bmm1, bmm2,
                                      stream=stream))
    torch.cuda.synchronize()
    for (b, table, n, _, eng, *_), (out, lse) in zip(jobs, results):
        assert int(eng.status.item()) == 0
        _check(out, lse, b, table, n)


def test_many_short_requests():
    """More segments than parts, pieces of one tile, requests without keys between."""
    rng = np.random.default_rng(3)
    lens = [int(v) if rng.random() < 0.7 else 0 for v in rng.integers(1, 70, 300)]
    b, table, n = prefix_batch(lens, 1, 8, 100, seed=26)
    _check(*_decode(b, table, n), b, table, n)


@pytest.mark.parametrize("num_ctas", [None, 2])
def test_a_plan_of_other_lengths_stays_in_bounds(num_ctas):
    """Keys beyond the plan are not attended to, planned keys that are gone are masked,
    whole pieces of several tiles without a key among them."""
    b, table, n = prefix_batch((800, 40, 0), 4, 8, 200, seed=27)
    d = to_device(b)
    bmm1, bmm2 = bmm_scales(b)
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda",
                        num_ctas=num_ctas)
    eng.plan(torch.tensor([820, 820, 820], dtype=torch.int32, device="cuda"))
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"], bmm1, bmm2)
    assert int(eng.status.item()) == 0
    _check(out, lse, b, table, n)


@pytest.mark.parametrize("plan,fault", [          # one: the places of a request with one tile
    (lambda one: [0, 0, 0, 0], False),            # a plan: nobody has keys
    (lambda one: [0, one, 2 * one, 2 * one], False),             # a plan of other lengths
    (lambda one: [-1, -1, -1, -1], True),
    (lambda one: [0, one + 1, 2 * one + 1, 1 << 30], True),
    (lambda one: [2147483647, -2147483648, 7, 3 * one], True),
    (lambda one: [0, 2147483647, one, 3 * one], True),
    (lambda one: [one, one, 2 * one, 2 * one], True),            # does not begin at 0
    (lambda one: [0, one - 1, 2 * one - 1, 2 * one - 1], True),  # no tile
    (lambda one: [0, one + 1, one - 1, 3 * one], True),          # descends
    (lambda one: [0, one + 2, one + 2, one + 2], True),          # more tiles than the table holds
    (lambda one: [0, one + 2, 2 * one + 2, 2 * one + 2], True),
])
def test_a_plan_that_is_none_is_reported_without_a_fault(plan, fault):
    """Places that lead out of the line, its tables or its slots are not followed; the
    canary behind the workspace and the outputs stays, and a true plan works after it."""
    b, table, n = prefix_batch((300, 40, 0), 4, 8, 200, seed=27)
    d = to_device(b)
    bmm1, bmm2 = bmm_scales(b)
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda")
    assert d["bt"].shape[1] * 64 <= 512           # at most two tiles a request
    size = eng.workspace.numel()
    eng.workspace = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    eng.plan(torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda"))
    eng.places.copy_(torch.tensor(plan(int(eng.places[-1])), dtype=torch.int32))
    eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"], bmm1, bmm2)
    assert int(eng.status.item()) == (mla.FAULT_WORK_ITEM if fault else 0)
    assert bool((eng.workspace[size:] == 0xA5).all())
    eng.status.zero_()
    eng.plan(d["lens"])
    out, lse = eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"], bmm1, bmm2)
    assert int(eng.status.item()) == 0
    _check(out, lse, b, table, n)


def test_garbage_behind_the_last_keys_is_not_read():
    """NaN codes in the unused slots of the last pages, prefix and own."""
    b, table, n = prefix_batch((100, 37, 1), 4, 8, 333, seed=12)
    clean = b.kv.clone()
    b.kv[table[-1], n % 64:] = 0x7F
    for r in range(3):
        L = int(b.seq_lens[r])
        b.kv[b.block_table[r, L // 64], L % 64:] = 0xFF
    out, lse = _decode(b, table, n)
    b.kv = clean
    _check(out, lse, b, table, n)


def test_two_calls_of_one_plan_agree_and_match_the_whole_decode():
    """The same keys as one sequence per request (prefix copied into each) give
    the same attention through the plain decode."""
    b, table, n = prefix_batch((64, 128, 70), 4, 8, 640, seed=13)
    d = to_device(b)
    bmm1, bmm2 = bmm_scales(b)
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda")
    eng.plan(d["lens"])
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    first = eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"], bmm1, bmm2)
    second = eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"], bmm1, bmm2)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    joined = torch.cat([table.repeat(3, 1), b.block_table], 1).contiguous().cuda()
    whole = mla.FoldedMla(b.R, b.k, b.H, joined.shape[1], d["kv"].shape[0], "cuda")
    lens = (d["lens"] + n).int()
    whole.plan(lens)
    out, lse = whole.decode(d["q"], d["kv"], joined, lens, bmm1, bmm2)
    assert (lse - first[1]).abs().max() <= 2e-3
    assert (out.float() - first[0].float()).abs().max() <= 4e-2


def test_bad_pages_are_reported_without_a_fault():
    b, table, n = prefix_batch((100, 37), 4, 8, 333, seed=14)
    d = to_device(b)
    bmm1, bmm2 = bmm_scales(b)
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda")
    eng.plan(d["lens"])
    bad = table.clone()
    bad[2] = d["kv"].shape[0]
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    eng.decode(d["q"], d["kv"], bad.cuda(), plen, d["bt"], d["lens"], bmm1, bmm2)
    assert int(eng.status.item()) == mla.FAULT_PAGE_RANGE
    eng.status.zero_()                           # a prefix longer than its table is cut off
    long = torch.tensor([64 * table.numel() + 1], dtype=torch.int32, device="cuda")
    out, lse = eng.decode(d["q"], d["kv"], table.cuda(), long, d["bt"], d["lens"], bmm1, bmm2)
    assert int(eng.status.item()) == mla.FAULT_PAGE_RANGE
    eng.status.zero_()
    full = 64 * table.numel()
    _check(out, lse, b, table, full)


def test_captured_replay_with_a_growing_prefix():
    """Plan and decode in one graph; lengths change in place between replays."""
    b, table, n = prefix_batch((100, 37, 260), 7, 8, 700, seed=15)
    d = to_device(b)
    bmm1, bmm2 = bmm_scales(b)
    side = torch.cuda.Stream()
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda")
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.empty((b.R, b.M, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b.R, b.M), device="cuda")
    pt = table.cuda()
    step = lambda: (eng.plan(d["lens"]), eng.decode(  # noqa: E731
        d["q"], d["kv"], pt, plen, d["bt"], d["lens"], bmm1, bmm2, out=out, lse=lse))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        for prefix, lens in ((700, (100, 37, 260)), (65, (1, 0, 200)), (0, (100, 5, 0))):
            plen.fill_(prefix)
            d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            g.replay()
            side.synchronize()
            assert int(eng.status.item()) == 0
            b.seq_lens = torch.tensor(lens, dtype=torch.int32)
            _check(out, lse, b, table, prefix, f"prefix {prefix}")


def test_whole_step():
    """Absorb, append, shared-prefix decode as a step runs them, two steps: the
    codes each call leaves are what the next one reads."""
    R, k, H, P, base = 3, 2, 8, 130, (20, 63, 0)
    g = torch.Generator().manual_seed(16)
    pages, width = 12, 2
    kv = torch.zeros((pages, 64, 576), dtype=torch.uint8, device="cuda")
    perm = torch.randperm(pages, generator=g).int()
    ptable, table = perm[:3].cuda(), perm[3:3 + R * width].view(R, width).cuda()
    rope = mla.rope_table(P + 200)
    weight = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    qs, ks = 6 / 448, 6 / 448
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.kv_append(rand(P, 576), kv, ptable[None].contiguous(), zero, rope, ks, norm_weight=weight)
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")
    starts = torch.zeros(R, dtype=torch.int32, device="cuda")
    new = torch.tensor((0,) + base).cumsum(0).int().cuda()
    mla.kv_append(rand(sum(base), 576), kv, table, starts, rope, ks, norm_weight=weight,
                  cu_tokens=new, rope_starts=starts + P)
    lens = torch.tensor(base, dtype=torch.int32, device="cuda")
    w = (torch.randn((H, 128, 512), generator=g) / 128 ** 0.5).to(torch.bfloat16).cuda()
    eng = mla.PrefixMla(R, k, H, width, 3, pages, "cuda")
    sm = 1 / 192 ** 0.5
    for _ in range(2):
        q = mla.query_absorb(rand(R * k, H, 192), w, rope, lens + P, qs)
        mla.kv_append(rand(R * k, 576), kv, table, lens, rope, ks, norm_weight=weight,
                      rope_starts=lens + P)
        lens += k
        eng.plan(lens)
        out, lse = eng.decode(q, kv, ptable, plen, table, lens, sm * qs * ks, ks)
        torch.cuda.synchronize()
        assert int(eng.status.item()) == 0
        ro, rl, spread, reach = st.prefix_decode(q.cpu().numpy(), kv.cpu().numpy(), ptable.cpu().numpy(), P,
                                         table.cpu().numpy(), lens.cpu().numpy(), k, sm, qs, ks)
        bound = (2.0 ** -7 + 2.0 ** -11) * spread + 2.0 ** -15 * reach + 2.0 ** -8 * np.abs(ro) + 1e-6
        assert (np.abs(out.float().cpu().numpy() - ro) <= bound).all()
        assert np.abs(lse.cpu().numpy() - rl).max() <= 1e-3
