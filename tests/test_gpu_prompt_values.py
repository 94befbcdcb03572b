"""Values that are no numbers in mla_prompt_attention, where they are easily lost."""
import math

import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.prompt_util import check, reference

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(192)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n,m,H,Hkv", [(300, 900, 1, 1), (64, 5000, 2, 2), (200, 6000, 3, 1), (2048, 2048, 1, 1)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_piece_of_no_weight_keeps_its_nan(n, m, H, Hkv, causal, bad):
    """The first keys' scores are 200 (base 2) below the others': in FP32 their weights are 0, but 0 times
    NaN or an infinity is NaN, whether the request's keys are cut into pieces or not."""
    g = torch.Generator(device="cuda").manual_seed(n)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kn, kr, v = rand(n, H, 192), rand(m, Hkv, 128), rand(m, 64), rand(m, Hkv, 128)
    low = m // 4
    q[:, :, 0], kn[:, :, 0] = 8, 0
    kn[:low, :, 0] = -200 * math.log(2) / SCALE / 8
    args = (_i32(0, n), SCALE, _i32(0, m), causal)
    want, want_l = mla.prompt_attention(q, kn, kr, v, *args)
    check(want, want_l, reference(q, kn, kr, v, [0, n], [0, m], SCALE, causal))
    v[5, Hkv - 1, 3] = bad
    out, lse = mla.prompt_attention(q, kn, kr, v, *args)
    hit = torch.zeros(n, H, 128, dtype=torch.bool, device="cuda")
    first = max(0, 5 - (m - n)) if causal else 0
    hit[first:, H - H // Hkv:, 3] = True
    if causal and m == n:                          # rows that see low keys alone: an infinity stays one
        assert not torch.isfinite(out[hit]).any() and torch.isnan(out[low + 1:, H - 1, 3]).all()
    else:
        assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse, want_l)


@pytest.mark.parametrize("n,m,H,Hkv", [(5, 100, 2, 2), (300, 900, 1, 1), (64, 5000, 2, 2), (200, 6000, 3, 1),
                                       (1000, 1000, 1, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_whose_scores_are_all_minus_infinity(n, m, H, Hkv, causal):
    """0 / 0: NaN, not the zeros of a row without keys. Some rows by their query, and by the first keys all
    rows that see no others; the rest are as if those keys were not there."""
    g = torch.Generator(device="cuda").manual_seed(m)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kn, kr, v = rand(n, H, 192), rand(m, Hkv, 128), rand(m, 64), rand(m, Hkv, 128)
    low = m // 4
    q[:, :, 0], q[:, :, 1], kn[:, :, 0], kn[:, :, 1] = 1, 1, 0, 1
    kn[:low, :, 0] = -math.inf
    mine = torch.arange(1, n, 7, device="cuda")
    q[mine, H - 1, 1] = -math.inf
    status = _i32(0)
    out, lse = mla.prompt_attention(q, kn, kr, v, _i32(0, n), SCALE, _i32(0, m), causal, status=status)
    alone = torch.zeros(n, H, dtype=torch.bool, device="cuda")
    alone[mine, H - 1] = True
    if causal:
        alone[:max(0, low - (m - n))] = True
    assert torch.isnan(out[alone]).all() and (lse[alone] == -math.inf).all()
    q[mine, H - 1, 1] = 1
    ref = reference(q, kn[low:], kr[low:], v[low:], [0, n], [0, m - low], SCALE, causal)
    check(out[~alone], lse[~alone], [x[~alone] for x in ref])
    assert int(status.item()) == 0


def test_minus_infinity_beside_nan_scores():
    """Pieces of a cut item that have NaN, and others with -infinity alone."""
    n, m = 40, 6000
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kn, kr, v = rand(n, 1, 192), rand(m, 1, 128), rand(m, 64), rand(m, 1, 128)
    q[:, :, 0], kn[:, :, 0] = 1, -math.inf
    kn[m // 2, 0, 5] = math.nan
    out, lse = mla.prompt_attention(q, kn, kr, v, _i32(0, n), SCALE, _i32(0, m))
    assert torch.isnan(out).all() and torch.isnan(lse).all()
