"""The oracle of the cache's books: closed forms and worked examples."""
import math

import numpy as np

import oracle.attention as att
import oracle.cache as oc
from workloads import make_batch_from_lengths


def test_weights_of_a_row_sum_to_one():
    b = make_batch_from_lengths([5, 0, 70], 2, 3, seed=3)
    out, lse = att.mla_decode(b.q.numpy(), b.kv.numpy(), b.block_table.numpy(), b.seq_lens.numpy(),
                              b.k, b.sm_scale, b.q_scale, b.kv_scale)
    bmm1 = b.sm_scale * b.q_scale * b.kv_scale
    w, e = oc.key_weights(b.q.numpy(), b.kv.numpy(), b.block_table.numpy(), b.seq_lens.numpy(),
                          np.asarray(lse).reshape(3, 6), b.k, bmm1)
    assert [len(x) for x in w] == [5, 0, 70]
    assert abs(w[0].sum() - 6) < 1e-4 and abs(w[2].sum() - 6) < 1e-4
    assert all((x >= 0).all() and (y > 0).all() for x, y in zip(w, e))


def test_one_key_gets_every_row_and_rows_without_an_lse_add_nothing():
    b = make_batch_from_lengths([1], 1, 4, seed=4)
    _, lse = att.mla_decode(b.q.numpy(), b.kv.numpy(), b.block_table.numpy(), b.seq_lens.numpy(),
                            1, b.sm_scale, 1.0, 1.0)
    lse = np.array(lse).reshape(1, 4)
    lse[0, 1], lse[0, 2] = -math.inf, math.nan
    w, _ = oc.key_weights(b.q.numpy(), b.kv.numpy(), b.block_table.numpy(), b.seq_lens.numpy(), lse,
                          1, b.sm_scale)
    assert abs(w[0][0] - 2) < 1e-5


def test_evict_worked_examples():
    w = [5, 1, 4, 1, 3, 9]
    slots = range(6)
    # The three largest: 9, 5, 4 (slots 5, 0, 2); slot 5 moves into slot 1.
    assert oc.evict(6, w, slots, 3, 0, 0) == ([0, 2, 5], [(5, 1)])
    # Ties to the lower slot: of the two ones slot 1 stays.
    assert oc.evict(6, w, slots, 5, 0, 0) == ([0, 1, 2, 4, 5], [(5, 3)])
    # Slots 0 and 1 and the newest are held.
    assert oc.evict(6, [0] * 6, slots, 4, 1, 2) == ([0, 1, 2, 5], [(5, 3)])
    # By position, not by slot.
    assert oc.evict(4, w, [7, 0, 9, 3], 2, 1, 1) == ([1, 2], [(2, 0)])
    # More held than places: the lower slots.
    assert oc.evict(6, w, slots, 2, 6, 0) == ([0, 1], [])
    assert oc.evict(6, w, slots, 0, 2, 2) == ([], [])
    assert oc.evict(2, w, slots, 3, 0, 0) == ([0, 1], [])
    # NaN weighs less than anything.
    assert oc.evict(3, [math.nan, -math.inf, 0.0], slots, 2, 0, 0) == ([1, 2], [(2, 0)])
