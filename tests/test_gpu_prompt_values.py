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
