"""Bounded waits of the kernels around the decode: they count from the end of the kernel
before, and one that runs out stops its CTA, is reported, and leaves the next call whole."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.gpu_util import bmm_scales, to_device
from tests.step_util import angle_table, prefix_batch
from tests.test_gpu_prefix import _check

pytestmark = pytest.mark.gpu

MS = 1_000_000


def _absorb_inputs(R, k, H, seed=71):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((R * k, H, 192), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((H, 128, 512), generator=g) / 128 ** 0.5).to(torch.bfloat16).cuda()
    starts = torch.randint(0, 50, (R,), generator=g).int().cuda()
    return q, w, angle_table(60).cuda(), starts, 6 / 448


@pytest.mark.parametrize("R,k,H", [(2, 4, 8), (64, 7, 8), (128, 7, 64)])
def test_absorb_wait_that_runs_out(R, k, H):
    """One band, one job and three jobs of four bands per CTA: the CTA without its first
    weights stops after 20 ms; the others have written theirs, and the next call is whole."""
    args = _absorb_inputs(R, k, H)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = mla.query_absorb(*args, status=status)
    assert int(status.item()) == 0
    got = torch.full_like(want, 9)
    mla.query_absorb_wait_test(*args, got, status, 20 * MS)
    torch.cuda.synchronize()
    assert int(status.item()) == mla.FAULT_WAIT_TIMEOUT
    late = (got != want).any(-1)
    assert late.any()
    if R > 2:                                     # CTA 0 has few of the (head, 128 tokens) blocks
        assert late.float().mean() < 0.5
    status.zero_()
    again = mla.query_absorb(*args, status=status)
    assert int(status.item()) == 0 and torch.equal(again, want)


def test_absorb_behind_a_kernel_that_outlasts_its_limit():
    """A decode on one CTA lets its successor start at once and then runs for tens of ms;
    the absorb's CTAs are on other SMs by then, with 2 ms for any of their waits."""
    keys = 1 << 23
    shape = mla.make_shape(1, 4, 8, keys // 64, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros((4, 8, 576), dtype=torch.uint8, device="cuda")
    kv = torch.zeros((1, 64, 576), dtype=torch.uint8, device="cuda")
    table, lens = torch.zeros((1, keys // 64), **i32), torch.full((1,), keys, **i32)
    counts, work = torch.zeros(1, **i32), torch.full((mla.plan_list_len(shape),), -1, **i32)
    ws = torch.empty(max(mla.workspace_bytes(shape), 256), dtype=torch.uint8, device="cuda")
    out = torch.empty((1, 32, 512), dtype=torch.bfloat16, device="cuda")
    lse, status = torch.empty((1, 32), device="cuda"), torch.zeros(2, **i32)
    args = _absorb_inputs(5, 3, 8)
    want = mla.query_absorb(*args)
    got = torch.empty_like(want)
    mla.plan_splits(shape, lens, counts, work)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

    def decode():
        mla.folded_decode(shape, q, kv, table, lens, 0.1, 1.0, counts, work, ws, out, lse, status[:1])

    decode()
    begin.record()
    decode()
    end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) > 20.0         # ms: ten times the limit below
    decode()                                      # no event between the two
    mla.query_absorb_wait_test(*args, got, status[1:], 2 * MS, withhold=False)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    assert torch.equal(got, want)


@pytest.mark.parametrize("lens,k,H,prefix,num_ctas", [
    ((100, 300), 4, 8, 600, None),                # a tile or two per pair, most pairs without any
    ((100, 300), 4, 8, 600, 2),                   # all on the pair that stops
    ((700, 0, 1500), 3, 64, 3000, 6),             # pieces of several tiles, in three pairs
    ((5,) * 40, 1, 64, 0, 4),                     # own keys alone, many pieces of one tile
])
def test_prefix_wait_that_runs_out(lens, k, H, prefix, num_ctas):
    """The pair without its first queries stops after 20 ms; the same plan and workspace serve
    the next call."""
    b, table, _ = prefix_batch(lens, k, H, max(prefix, 1), seed=72)
    d = to_device(b)
    eng = mla.PrefixMla(b.R, k, H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda",
                        num_ctas=num_ctas)
    eng.plan(d["lens"])
    pt, plen = table.cuda(), torch.tensor([prefix], dtype=torch.int32, device="cuda")
    bmm1, bmm2 = bmm_scales(b)
    out = torch.empty((b.R, b.M, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b.R, b.M), device="cuda")
    mla.prefix_decode_wait_test(eng.shape, d["q"], d["kv"], pt, plen, d["bt"], d["lens"], bmm1, bmm2,
                                eng.places, eng.workspace, out, lse, eng.status, 20 * MS)
    torch.cuda.synchronize()
    assert int(eng.status.item()) == mla.FAULT_WAIT_TIMEOUT
    eng.status.zero_()
    out, lse = eng.decode(d["q"], d["kv"], pt, plen, d["bt"], d["lens"], bmm1, bmm2)
    torch.cuda.synchronize()
    assert int(eng.status.item()) == 0
    _check(out, lse, b, table, prefix)
