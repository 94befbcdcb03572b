"""NaN in the decode of a batch behind a shared prefix: a row that NaN reaches has NaN
in out and in its LSE, however the keys are cut; -inf is for rows without keys alone."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.gpu_util import bmm_scales, to_device
from tests.step_util import prefix_batch
from tests.test_gpu_prefix import _check

pytestmark = pytest.mark.gpu

NAN = 0x7F


def _decode(b, table, n, num_ctas=None):
    d = to_device(b)
    eng = mla.PrefixMla(b.R, b.k, b.H, d["bt"].shape[1], table.numel(), d["kv"].shape[0], "cuda",
                        num_ctas=num_ctas)
    eng.plan(d["lens"])
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"], *bmm_scales(b))
    torch.cuda.synchronize()
    assert int(eng.status.item()) == 0
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("num_ctas", [None, 2, 7])
@pytest.mark.parametrize("lens,prefix", [((100, 300), 600), ((100, 300), 0), ((0, 300), 1000),
                                         ((1, 0), 1)])
def test_a_query_row_of_nan(lens, prefix, num_ctas):
    b, table, _ = prefix_batch(lens, 4, 8, max(prefix, 1), seed=41)
    clean = _decode(b, table, prefix, num_ctas)
    b.q[2, 3] = NAN                               # row 19 of request 0
    b.q[6, 5, 575] = NAN                          # one rope dim of row 21 of request 1
    out, lse = _decode(b, table, prefix, num_ctas)
    bad = torch.zeros(2, 32, dtype=torch.bool)
    bad[0, 19], bad[1, 21] = True, True
    for r in range(2):
        if lens[r] + prefix == 0:                 # no keys: nothing meets the NaN
            bad[r] = False
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("num_ctas", [None, 2, 7])
def test_a_key_of_nan(num_ctas):
    """In the prefix it reaches every row, in a request's own keys the request's rows,
    whichever pieces it shares them with; a request without keys has none."""
    b, table, n = prefix_batch((700, 300, 0), 4, 8, 900, seed=42)
    clean = _decode(b, table, n, num_ctas)
    kv = b.kv.clone()
    b.kv[b.block_table[1, 3], 17, 40] = NAN
    out, lse = _decode(b, table, n, num_ctas)
    assert out[1, :, 40].isnan().all() and lse[1].isnan().all()
    assert torch.equal(out[::2], clean[0][::2]) and torch.equal(lse[::2], clean[1][::2])
    out, lse = _decode(b, table, 0, num_ctas)     # behind no prefix
    assert lse[1].isnan().all() and lse[0].isfinite().all() and torch.isneginf(lse[2]).all()
    assert not out[2].any()
    b.kv = kv
    b.kv[table[7], 3, 560] = 0xFF
    out, lse = _decode(b, table, n, num_ctas)
    assert out.isnan().all() and lse.isnan().all()


def test_rows_without_keys_beside_nan():
    b, table, _ = prefix_batch((0, 70), 2, 8, 64, seed=43)
    b.q[:] = NAN
    out, lse = _decode(b, table, 0)
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    assert out[1].isnan().all() and lse[1].isnan().all()
    b, table, n = prefix_batch((0, 70), 2, 8, 64, seed=43)
    _check(*_decode(b, table, n), b, table, n)
