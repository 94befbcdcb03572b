"""NaN through the merge of partial decodes by their LSEs (mla_lse_merge): a source whose
LSE is NaN had keys, so its NaN stays; -inf is for rows whose sources are all empty."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.gpu_util import bmm_scales, to_device
from tests.step_util import prefix_batch

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def _merge(outs, lses):
    out = torch.empty(outs.shape[1:], dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(lses.shape[1:], device="cuda")
    mla.lse_merge(outs.contiguous(), lses.contiguous(), out, lse)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("sources", [1, 2, 3, 33, 40])
def test_sources_of_nan(sources):
    """Rows: no NaN; one NaN source among finite ones; all NaN; NaN among empty ones; all
    empty. The NaN source is the last, past the first 32 where there are as many."""
    g = torch.Generator().manual_seed(sources)
    outs = torch.randn((sources, 5, 512), generator=g).to(torch.bfloat16)
    lses = torch.randn((sources, 5), generator=g)
    lses[:, 2] = NAN
    lses[:, 3:] = -INF
    for row in (1, 3):
        lses[-1, row], outs[-1, row] = NAN, NAN
    outs[:, 2] = NAN
    out, lse = _merge(outs.cuda(), lses.cuda())
    assert out[0].isfinite().all() and lse[0].isfinite()
    for row in (1, 2, 3):
        assert out[row].isnan().all() and lse[row].isnan(), row
    assert not out[4].any() and torch.isneginf(lse[4])


def test_a_row_of_nan_of_two_prefix_decodes():
    """The row's LSE is NaN on both shards: the merged row is NaN, not 0; the others are
    as without it."""
    parts = []
    for seed in (44, 45):
        b, table, n = prefix_batch((100, 300), 4, 8, 300, seed=seed)
        b.q[2, 3] = 0x7F
        d = to_device(b)
        eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda")
        eng.plan(d["lens"])
        plen = torch.tensor([n], dtype=torch.int32, device="cuda")
        parts.append(eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"],
                                *bmm_scales(b)))
    outs, lses = (torch.stack(p).flatten(1, 2) for p in zip(*parts))
    out, lse = _merge(outs, lses)
    assert out[19].isnan().all() and lse[19].isnan()
    live = torch.arange(64) != 19
    assert out[live].isfinite().all() and lse[live].isfinite().all()
