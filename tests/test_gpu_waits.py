"""Bounded waits of the kernels around the decode: they count from the end of the kernel
before, and one that runs out stops its CTA, is reported, and leaves the next call whole."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.step_util import angle_table

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
