"""Pages outside the cache in the decode behind a shared prefix: reported, and read as
pages of zeros, so that no row sees what an earlier tile left in shared memory."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.gpu_util import bmm_scales, to_device
from tests.step_util import prefix_batch
from tests.test_gpu_prefix import _check

pytestmark = pytest.mark.gpu


def _run(b, table, n, *, num_ctas=None, kv=None, fault=0):
    d = to_device(b)
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda",
                        num_ctas=num_ctas)
    eng.plan(d["lens"])
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = eng.decode(d["q"], d["kv"] if kv is None else kv, table.cuda(), plen, d["bt"],
                          d["lens"], *bmm_scales(b))
    torch.cuda.synchronize()
    assert int(eng.status.item()) == fault
    return out, lse


@pytest.mark.parametrize("num_ctas", [None, 2])
@pytest.mark.parametrize("k,H", [(4, 8), (3, 64)])
@pytest.mark.parametrize("prefix_at,own_at", [((0,), ()), ((2, 3), ()), ((9,), ()), ((), (0,)),
                                              ((), (3, 4)), ((), (10,)), (range(10), range(11)),
                                              ((1, 5, 8), (1, 2, 5))])
def test_pages_outside_the_cache_are_zeros(prefix_at, own_at, k, H, num_ctas):
    """First, middle and last pages of the prefix (10, the last of 24 keys) and of request 0
    (11, the last of 60), alone, side by side and all. A decode on a cache of NaN codes goes
    before, so that stale shared memory would show."""
    b, table, n = prefix_batch((700, 300), k, H, 600, seed=51)
    nan = torch.full(b.kv.shape, 0x7F, dtype=torch.uint8, device="cuda")
    used = set(table.tolist()) | set(b.block_table[0].tolist()) | set(b.block_table[1, :5].tolist())
    zero = min(set(range(b.kv.shape[0])) - used)  # a page that nobody has
    b.kv[zero] = 0
    outside = [b.kv.shape[0], -1, -2, -(1 << 31), (1 << 31) - 1]
    bad_table, bad_own = table.clone(), b.block_table.clone()
    for i in prefix_at:
        bad_table[i], table[i] = outside[i % 5], zero
    for i in own_at:
        bad_own[0, i], b.block_table[0, i] = outside[i % 5], zero
    want = b.block_table
    b.block_table = bad_own
    _run(b, bad_table, n, num_ctas=num_ctas, kv=nan, fault=mla.FAULT_PAGE_RANGE)
    out, lse = _run(b, bad_table, n, num_ctas=num_ctas, fault=mla.FAULT_PAGE_RANGE)
    b.block_table = want
    _check(out, lse, b, table, n)
