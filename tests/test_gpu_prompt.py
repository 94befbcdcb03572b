"""Attention of packed prompts (mla_prompt_attention) against 64-bit values, within the tolerance that
tests/prompt_util.py derives."""
import math

import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.prompt_util import check, reference

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(192.0)


def _cu(n, start=0):
    c = [start]
    for v in n:
        c.append(c[-1] + v)
    return c


def _inputs(cu, ck, H, Hkv, seed, *, behind=0, fused=True, wide=0, gain=1.0):
    """Inputs with `behind` rows behind the last request's, which hold NaN, as do the rows before the
    first; `wide` elements between heads and rows that are not the call's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    T, Tk = cu[-1] + behind, ck[-1] + behind
    q = (gain * rand(T, H, 192 + wide)).to(torch.bfloat16)[..., :192]
    if fused:
        kv = rand(Tk, Hkv, 256 + wide).to(torch.bfloat16)
        kn, v = kv[..., :128], kv[..., 128:256]
    else:
        kn, v = rand(Tk, Hkv, 128).to(torch.bfloat16), rand(Tk, Hkv, 128).to(torch.bfloat16)
    kr = rand(Tk, 64 + 8 * (wide > 0)).to(torch.bfloat16)[:, :64]
    for t, c in ((q, cu), (kn, ck), (kr, ck), (v, ck)):
        t[:c[0]] = math.nan
        t[c[-1]:] = math.nan
    return q, kn, kr, v


def _run(n, m=None, *, H=2, Hkv=None, causal=True, seed=0, start=0, **kw):
    Hkv = Hkv or H
    cu = _cu(n, start)
    ck = None if m is None else _cu(m, start)
    q, kn, kr, v = _inputs(cu, ck or cu, H, Hkv, seed, **kw)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((q.shape[0], H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], H), 7.0, device="cuda")
    status = i32([0])
    got = mla.prompt_attention(q, kn, kr, v, i32(cu), SCALE, cu_keys=None if ck is None else i32(ck),
                               causal=causal, out=out, lse=lse, status=status)
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is lse and int(status.item()) == 0
    ref = reference(q, kn, kr, v, cu, ck, SCALE, causal)
    rows = check(out, lse, ref, f"{n} {m} H{H}")
    assert (out[~rows] == 7).all() and (lse[~rows] == 7).all(), "rows of no request were written"
    return out, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [(1,), (127,), (128, 129), (0, 255, 0, 256, 1, 257, 0), (100, 37),
                               (511, 64, 3), (640,)])
def test_prompts(n, causal):
    _run(n, H=3, causal=causal, seed=sum(n), behind=5, start=3)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m", [((1,), (1000,)), ((1, 1, 1), (1, 128, 129)), ((16,), (2000,)),
                                 ((100, 300), (700, 301)), ((130, 5), (0, 7)), ((300,), (40,)),
                                 ((600, 257, 256), (100, 1, 200)), ((3, 0, 2), (0, 50, 0))])
def test_cached_keys_and_rows_without_keys(n, m, causal):
    _run(n, m, H=2, causal=causal, seed=sum(m), behind=70)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 2), (8, 1), (6, 3), (15, 5), (64, 64), (40, 8)])
def test_heads(H, Hkv):
    _run((150, 70), H=H, Hkv=Hkv, seed=H)


@pytest.mark.parametrize("fused,wide", [(True, 0), (False, 0), (True, 8), (True, 64)])
def test_layouts(fused, wide):
    _run((140, 9), (200, 140), H=3, seed=wide, fused=fused, wide=wide)


def test_token_strides_below_a_heads():
    """Heads outside, tokens inside: the strides may come in any order."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kn, v, kr = rand(4, 300, 192).transpose(0, 1), rand(2, 300, 128).transpose(0, 1), \
        rand(2, 300, 128).transpose(0, 1), rand(300, 64)
    cu = [0, 170, 300]
    out, lse = mla.prompt_attention(q, kn, kr, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), SCALE)
    check(out, lse, reference(q, kn, kr, v, cu, None, SCALE, True))


@pytest.mark.parametrize("n", [2048, 3000, 5000])
def test_long_prompts_cut_into_parts(n):
    _run((n,), H=1, seed=n, behind=1)
    _run((n // 3, n), H=3, Hkv=1, seed=n + 1, causal=False)


def test_chunks_of_long_prompts():
    _run((512,), (9001,), H=4, seed=1)
    _run((1, 40, 300), (6000, 4000, 2000), H=2, seed=2)
    _run((1,), (20000,), H=1, seed=3)


def test_whole_items_claimed_by_the_ctas():
    """Enough work of few long items that none is cut: 64 heads of prompts of five tiles and more."""
    _run((640, 700, 650, 900, 1100), H=64, Hkv=8, seed=4)


@pytest.mark.parametrize("R", [31, 32, 33, 70])
def test_one_long_prompt_among_short_ones(R):
    """Up to 32 requests the CTAs plan for themselves, beyond a kernel does; the long one is cut."""
    n = [(7 * i) % 50 for i in range(R)]
    n[R // 2] = 3500
    _run(n, H=2, seed=R, behind=3)
    _run([1] * R, [40 + i if i != 5 else 5000 for i in range(R)], H=2, Hkv=1, seed=R + 1)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (3, 3), (5, 1), (9, 3), (15, 5), (8, 2), (7, 7)])
def test_two_heads_to_an_item(H, Hkv, causal):
    """Requests of up to 256 rows have a head in each half of an item: on the same keys or each on its
    own, an odd head left over, whole and cut, beside requests that are longer."""
    _run((1, 256, 0, 100, 257, 200), (900, 256, 20, 1500, 300, 0), H=H, Hkv=Hkv, causal=causal, seed=H, behind=2)
    _run((5,), (9000,), H=H, Hkv=Hkv, causal=causal, seed=H + 1)
    _run((130, 20), (3000, 2500), H=H, Hkv=Hkv, causal=causal, seed=H + 2, start=4)


@pytest.mark.parametrize("R,H,Hkv,n,m", [(30, 32, 32, 9, 10), (30, 32, 8, 40, 700), (40, 21, 3, 33, 650),
                                         (40, 64, 64, 2, 300)])
def test_many_short_items(R, H, Hkv, n, m):
    """More items than pairs of CTAs, by turns and claimed, two heads each."""
    _run([n + i % 7 for i in range(R)], [m + 5 * i for i in range(R)], H=H, Hkv=Hkv, seed=R)


def test_many_requests():
    g = torch.Generator().manual_seed(5)
    n = torch.randint(0, 40, (1024,), generator=g).tolist()
    _run(n, H=1, seed=5)


@pytest.mark.parametrize("gain", [0.0, 1e-3, 20.0, 300.0])
def test_flat_and_peaked_scores(gain):
    _run((400, 130), H=2, seed=6, gain=gain)
    _run((30,), (1500,), H=2, seed=7, gain=gain)


def test_growing_scores_move_the_maximum():
    """Keys whose scores grow from tile to tile by far more than 2^8, and shrink again."""
    n = 900
    g = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn(n, 2, 192, generator=g, device="cuda").abs().to(torch.bfloat16)
    up = torch.cat([torch.linspace(-3, 3, 600), torch.linspace(3, -3, 300)]).cuda()
    kn = (up[:, None, None] * torch.ones(n, 2, 128, device="cuda")).to(torch.bfloat16)
    kr = torch.randn(n, 64, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(n, 2, 128, generator=g, device="cuda").to(torch.bfloat16)
    cu = [0, n]
    for causal in (True, False):
        out, lse = mla.prompt_attention(q, kn, kr, v, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                        1.0, causal=causal)
        check(out, lse, reference(q, kn, kr, v, cu, None, 1.0, causal))


def test_nan_and_infinities_stay_in_their_request():
    """Requests full of NaN and infinities beside finite ones; within a request a key's NaN reaches
    the rows that see it and no row before its tile."""
    n = (100, 300, 65, 200)
    cu = _cu(n)
    q, kn, kr, v = _inputs(cu, cu, 2, 2, 9, fused=False)
    want, want_l = mla.prompt_attention(q, kn, kr, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), SCALE)
    for t in (q, kn, kr, v):
        t[400:465] = math.nan
    v[0:100] = math.inf
    kn[465 + 150] = math.nan
    v[465 + 199] = math.nan
    out, lse = mla.prompt_attention(q, kn, kr, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), SCALE)
    same = lambda a, b: torch.equal(a, b)  # noqa: E731
    assert same(out[100:400], want[100:400]) and same(lse[100:400], want_l[100:400])
    assert same(lse[0:100], want_l[0:100])
    assert torch.isnan(out[400:465]).all() and torch.isnan(lse[400:465]).all()
    assert same(lse[465:615], want_l[465:615]) and torch.isnan(lse[615:]).all()
    assert same(out[465:465 + 128], want[465:465 + 128]) and torch.isnan(out[615:]).all()


@pytest.mark.parametrize("n,m,H", [(700, 700, 2), (300, 900, 1), (1500, 1500, 1), (2048, 2048, 4),
                                   (256, 900, 2), (200, 700, 3), (150, 6000, 4), (129, 129, 96)])
def test_values_that_are_no_numbers_reach_only_rows_that_see_them(n, m, H):
    """Other rows, and other dims of the rows that do, keep their bits; cut items too."""
    q, kn, kr, v = _inputs([0, n], [0, m], H, H, 21)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want, want_l = mla.prompt_attention(q, kn, kr, v, i32(0, n), SCALE, cu_keys=i32(0, m))
    spots = [(m - n + i, d, x) for i, d, x in
             [(0, 3, math.nan), (5, 64, math.inf), (127, 127, -math.inf), (128, 0, math.nan), (n - 1, 63, math.nan),
              (n // 2, 77, math.inf), (n // 2 + 1, 77, -math.inf)]]
    for j, d, x in spots:
        v[j, H - 1, d] = x
    out, lse = mla.prompt_attention(q, kn, kr, v, i32(0, n), SCALE, cu_keys=i32(0, m))
    assert torch.equal(lse, want_l)
    hit = torch.zeros(n, H, 128, dtype=torch.bool, device="cuda")
    for j, d, _ in spots:
        hit[max(0, j - (m - n)):, H - 1, d] = True
    assert torch.equal(out[~hit], want[~hit]) and not torch.isfinite(out[hit]).any()


def test_a_row_of_nan_queries_stays_alone():
    q, kn, kr, v = _inputs([0, 300], [0, 300], 2, 2, 10)
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    want, want_l = mla.prompt_attention(q, kn, kr, v, cu, SCALE)
    q[17, 1] = math.nan
    out, lse = mla.prompt_attention(q, kn, kr, v, cu, SCALE)
    assert torch.isnan(out[17, 1]).all() and torch.isnan(lse[17, 1])
    out[17, 1], lse[17, 1] = want[17, 1], want_l[17, 1]
    assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("cu,ck,live", [
    ([0, 50, 30, 100], None, [0, 2]), ([-5, 50, 100, 100], None, [1]), ([0, 50, 100, 101], None, [0, 1]),
    ([0, 50, 75, 100], [0, 60, 40, 100], [0, 2]), ([0, 2 ** 31 - 1, 75, 100], None, [2])])
def test_offsets_that_are_none_skip_their_request(cu, ck, live):
    q, kn, kr, v = _inputs([0, 100], [0, 100], 2, 2, 11)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    status = i32([0])
    out = torch.full((100, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mla.prompt_attention(q, kn, kr, v, i32(cu), SCALE, cu_keys=None if ck is None else i32(ck), out=out,
                         status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == mla.FAULT_WORK_ITEM
    owners = torch.zeros(100, dtype=torch.int32, device="cuda")
    for r in live:
        owners[cu[r]:cu[r + 1]] += 1
    for r in live:
        a, b = cu[r], cu[r + 1]
        c, d = (ck or cu)[r], (ck or cu)[r + 1]
        ref = reference(q[a:b], kn[c:d], kr[c:d], v[c:d], [0, b - a], [0, d - c], SCALE, True)
        alone = owners[a:b] == 1                   # rows that two requests share may be either's
        check(out[a:b][alone], None, [x[alone] for x in ref])
    assert (out[owners == 0] == 7).all()


def test_no_tokens_and_no_keys():
    q, kn, kr, v = _inputs([0, 10], [0, 10], 2, 2, 12)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = mla.prompt_attention(q[:0], kn[:0], kr[:0], v[:0], i32([0, 0]), SCALE)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)
    out, lse = mla.prompt_attention(q, kn[:0], kr[:0], v[:0], i32([0, 10]), SCALE, cu_keys=i32([0, 0]))
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = mla.prompt_attention(q, kn, kr, v, i32([0, 0]), SCALE, out=torch.ones_like(q[..., :128]).contiguous())
    torch.cuda.synchronize()
    assert (out == 1).all()


def test_without_lse_same_bits_and_another_stream():
    n = (700, 1500)
    q, kn, kr, v = _inputs(_cu(n), _cu(n), 4, 4, 13)
    cu = torch.tensor(_cu(n), dtype=torch.int32, device="cuda")
    out, lse = mla.prompt_attention(q, kn, kr, v, cu, SCALE)
    again, none = mla.prompt_attention(q, kn, kr, v, cu, SCALE, return_lse=False)
    assert none is None and torch.equal(again, out)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other, _ = mla.prompt_attention(q, kn, kr, v, cu, SCALE, stream=s)
    s.synchronize()
    assert torch.equal(other, out)


def test_a_captured_call_with_other_lengths():
    """One captured graph, replayed for batches that are cut, that are not, and that are empty."""
    T, H = 3000, 4
    q, kn, kr, v = _inputs([0, T], [0, T], H, H, 14)
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")
    ws = torch.randint(0, 255, (mla.prompt_workspace_bytes(2),), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, device="cuda")
    mla.prompt_attention(q, kn, kr, v, cu, SCALE, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.prompt_attention(q, kn, kr, v, cu, SCALE, out=out, lse=lse, workspace=ws)
    for c in ([0, 100, T], [0, 0, 0], [0, 400, 800], [0, T, T], [5, 30, 2777]):
        cu.copy_(torch.tensor(c, dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        rows = check(out, lse, reference(q, kn, kr, v, c, None, SCALE, True), str(c))
        assert (out[~rows] == 7).all()


def test_two_workspaces_on_two_streams():
    n = (2000, 900)
    ins = [_inputs(_cu(n), _cu(n), 4, 4, 20 + i) for i in range(2)]
    cu = torch.tensor(_cu(n), dtype=torch.int32, device="cuda")
    want = [mla.prompt_attention(*x, cu, SCALE)[0] for x in ins]
    ws = [torch.empty(mla.prompt_workspace_bytes(2), dtype=torch.uint8, device="cuda") for _ in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(mla.prompt_attention(*ins[i], cu, SCALE, workspace=ws[i], stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


def test_a_wait_that_runs_out_is_reported_and_the_workspace_stays_usable():
    for n, H in (((1500,), 2), ((640, 700, 650, 900, 1100), 64)):
        q, kn, kr, v = _inputs(_cu(n), _cu(n), H, H, 15)
        cu = torch.tensor(_cu(n), dtype=torch.int32, device="cuda")
        ws = torch.empty(mla.prompt_workspace_bytes(len(n)), dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want, want_l = mla.prompt_attention(q, kn, kr, v, cu, SCALE)
        out, lse = torch.zeros_like(want), torch.zeros_like(want_l)
        mla.prompt_attention_wait_test(q, kn, kr, v, cu, SCALE, out, lse, ws, status, 20_000_000)
        torch.cuda.synchronize()
        assert int(status.item()) == mla.FAULT_WAIT_TIMEOUT
        status.zero_()
        mla.prompt_attention(q, kn, kr, v, cu, SCALE, out=out, lse=lse, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and torch.equal(out, want) and torch.equal(lse, want_l)
