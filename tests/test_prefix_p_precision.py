"""How P's second term is rounded where requests share a prefix: E5M2 there, E4M3 in the
decode of every request on its own. Bounds of both for any weight, and what each leaves in
an output of broad and of peaked rows. No GPU; PyTorch's casts round as the kernels do."""
import numpy as np
import pytest
import torch

import oracle.attention as att
from workloads import make_batch_from_lengths

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def _two_terms(p, second):
    """p (float64, up to 2^8) as E4M3 plus a second term, back in float64."""
    hi = p.float().to(E4M3).float()
    return hi.double() + (p.float() - hi).to(second).double()


@pytest.mark.parametrize("second,rel,small", [(E5M2, 2.0 ** -8, 2.0 ** -14),
                                              (E4M3, 2.0 ** -9, 2.0 ** -10)])
def test_bounds_of_a_weight(second, rel, small):
    """hi = e4m3(p) leaves at most half a step, 2^-4 of p's power of two (2^-10 below 2^-6);
    what is less than that lies in the binade below it, where half a step of E5M2 is 2^-3 of
    the binade's lower end: 2^-8 of p's power of two, or 2^-14. E4M3's is 2^-4 of it, 2^-9,
    but never less than half of its smallest step, 2^-10."""
    p = torch.exp2(torch.linspace(-30, 8, 2_000_001, dtype=torch.float64))
    err = (_two_terms(p, second) - p.float().double()).abs()
    assert bool((err <= rel * p + small).all())
    # Neither part can be halved.
    assert bool((err > rel * p / 2).logical_and(p > 1).any())
    assert bool((err[p < 2.0 ** -7] > small / 2).any())


def _output_errors(std, seed):
    """Root mean square error of an output relative to the output's, from P's terms alone:
    (E4M3 + E5M2, E4M3 + E4M3). 4 x 8 rows of one request of 4,096 keys, all against a
    maximum 2 below the row's largest score, as the kernels keep it."""
    b = make_batch_from_lengths((4096,), 4, 8, seed=seed, value_std=std, scaling="amax")
    q = att.e4m3.decode(b.q.numpy()).reshape(32, 576) * b.q_scale
    keys = att.request_keys(b.kv.numpy(), b.block_table.numpy()[0], 0, 4096, b.kv_scale)
    x = torch.from_numpy((q @ keys.T) * b.sm_scale / np.log(2.0))
    p = torch.exp2(x - x.amax(1, keepdim=True) + 2.0)
    v = torch.from_numpy(keys[:, :512])
    out = p @ v
    return [float((((_two_terms(p, t) - p) @ v) ** 2).mean().sqrt() / (out ** 2).mean().sqrt())
            for t in (E5M2, E4M3)]


def test_broad_rows():
    """Values of deviation 0.5: scores within a few units of each other, most weights where
    E4M3's second term is finer."""
    e5m2, e4m3 = _output_errors(0.5, 91)
    assert e4m3 < e5m2 < 2.0 * e4m3 and e5m2 < 2.0 ** -9, (e5m2, e4m3)


def test_peaked_rows():
    """Deviation 1: a few keys lead, most weights lie below E4M3's normal range."""
    e5m2, e4m3 = _output_errors(1.0, 92)
    assert 1.5 * e5m2 < e4m3 and e5m2 < 2.0 ** -9, (e5m2, e4m3)
