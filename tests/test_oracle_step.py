"""Pins of the oracle's step functions to things other than themselves."""
import cmath

import numpy as np
import pytest

import oracle.attention as att
import oracle.step as st
from workloads import make_batch_from_lengths


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("position", [0, 1, 77, 131071])
def test_rotation_is_multiplication_by_a_unit_complex_number(interleaved, position):
    x = np.random.default_rng(position).normal(size=64)
    y = st.rotate(x, position, interleaved)
    for i in range(32):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        z = complex(x[p], x[q]) * cmath.exp(1j * position * 10000.0 ** (-i / 32))
        assert abs(complex(y[p], y[q]) - z) < 1e-9
    if position == 0:
        assert np.array_equal(y, x)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotated_products_depend_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(3)
    a, b = rng.normal(size=64), rng.normal(size=64)
    want = st.rotate(a, 11, interleaved) @ st.rotate(b, 4, interleaved)
    got = st.rotate(a, 1011, interleaved) @ st.rotate(b, 1004, interleaved)
    assert abs(want - got) < 1e-9


def test_cache_row_norm():
    x = np.random.default_rng(0).normal(size=576)
    y = st.cache_row(x, np.ones(512), 0.0, 0, True, 1.0)
    assert abs((y[:512] ** 2).mean() - 1) < 1e-12          # unit mean square
    assert np.allclose(st.cache_row(5 * x, np.ones(512), 0.0, 0, True, 1.0)[:512], y[:512])
    assert np.allclose(st.cache_row(x, None, 0.0, 0, True, 0.5), 2 * x)


def test_absorbed_query_selects_columns():
    q = np.random.default_rng(1).normal(size=192)
    w = np.zeros((128, 512))
    w[np.arange(128), np.arange(128) + 300] = 1.0
    y = st.absorbed_query(q, w, 0, True, 0.25)
    assert np.allclose(y[300:428], 4 * q[:128]) and not y[:300].any() and not y[428:512].any()
    assert np.allclose(y[512:], 4 * q[128:])


def test_prefix_decode_is_the_decode_of_the_joined_keys():
    """One request holding all keys, split at a page edge into prefix and own."""
    b = make_batch_from_lengths((200,), 2, 3, seed=5, scaling="amax")
    o, l = att.mla_decode(b.q.numpy(), b.kv.numpy(), b.block_table.numpy(), b.seq_lens.numpy(), 2,
                          b.sm_scale, b.q_scale, b.kv_scale)
    bt = b.block_table.numpy()
    po, pl, spread, reach = st.prefix_decode(b.q.numpy(), b.kv.numpy(), bt[0, :2], 128, bt[:, 2:],
                                             [72], 2, b.sm_scale, b.q_scale, b.kv_scale)
    assert np.allclose(po.reshape(o.shape), o, atol=1e-12) and np.allclose(pl.reshape(l.shape), l)
    assert (spread >= np.abs(po)).all() and (reach >= spread - 1e-12).all()
    no, nl, _, _ = st.prefix_decode(b.q.numpy(), b.kv.numpy(), bt[0], 0, bt, [0], 2, b.sm_scale,
                                    b.q_scale, b.kv_scale)
    assert not no.any() and np.isneginf(nl).all()
