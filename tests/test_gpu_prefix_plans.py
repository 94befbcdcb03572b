"""Plans of other lengths than the decode's: the shared-prefix decode attends to every key
of the lengths that it is given, whatever the plan was made for."""
import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.gpu_util import bmm_scales, to_device
from tests.step_util import prefix_batch
from tests.test_gpu_prefix import _check

pytestmark = pytest.mark.gpu


def _engine(b, table, num_ctas=None):
    return mla.PrefixMla(b.R, b.k, b.H, b.block_table.shape[1], table.numel(), b.kv.shape[0], "cuda",
                         num_ctas=num_ctas)


def _decode(eng, b, table, n, fault=0):
    d = to_device(b)
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = eng.decode(d["q"], d["kv"], table.cuda(), plen, d["bt"], d["lens"], *bmm_scales(b))
    torch.cuda.synchronize()
    assert int(eng.status.item()) == fault
    _check(out, lse, b, table, n)


@pytest.mark.parametrize("num_ctas", [None, 2, 7, 500])
@pytest.mark.parametrize("planned,lens", [
    ((250, 40, 0), (260, 40, 0)),                 # a request grew past a tile's edge
    ((0, 0, 0), (300, 40, 513)),                  # nobody had keys
    ((820, 820, 0), (800, 40, 900)),              # some have fewer tiles, one has more
    ((256, 512, 768), (257, 513, 769)),
    ((1, 1, 1), (0, 0, 1500)),
])
@pytest.mark.parametrize("prefix,k,H", [(200, 4, 8), (0, 4, 8), (700, 3, 64)])
def test_longer_than_planned(planned, lens, prefix, k, H, num_ctas):
    b, table, _ = prefix_batch(lens, k, H, max(prefix, 1), seed=61)
    eng = _engine(b, table, num_ctas)
    eng.plan(torch.tensor(planned, dtype=torch.int32, device="cuda"))
    _decode(eng, b, table, prefix)


def test_many_requests_longer_than_planned():
    """More requests than a CTA of the merge has threads, one of them short of a tile, the
    last or one in the middle; then a plan of the right lengths."""
    rng = np.random.default_rng(62)
    lens = [int(v) if rng.random() < 0.8 else 0 for v in rng.integers(1, 600, 700)]
    for r in (699, 300):
        lens[r] = 257
        b, table, n = prefix_batch(lens, 1, 2, 100, seed=62)
        planned = b.seq_lens.clone()
        planned[r] = 256
        eng = _engine(b, table)
        eng.plan(planned.cuda())
        _decode(eng, b, table, n)
        eng.plan(b.seq_lens.cuda())
        _decode(eng, b, table, n)


@pytest.mark.parametrize("num_ctas", [None, 2])
def test_words_that_are_no_plan(num_ctas):
    """Reported, and the answer is that of the lengths."""
    b, table, n = prefix_batch((300, 40, 0), 4, 8, 200, seed=63)
    eng = _engine(b, table, num_ctas)
    eng.plan(torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda"))
    one = int(eng.places[-1])                     # places of a request with one tile
    for words in ([-1] * 4, [2147483647, -2147483648, 7, 3 * one], [0, one + 1, one - 1, 3 * one],
                  [0, 3 * one, 3 * one, 3 * one], [one] * 4,
                  [one, one + 1, 2 * one + 1, 2 * one + 1]):
        eng = _engine(b, table, num_ctas)
        eng.plan(b.seq_lens.cuda())
        eng.places.copy_(torch.tensor(words, dtype=torch.int32))
        for _ in range(2):
            _decode(eng, b, table, n, fault=mla.FAULT_WORK_ITEM)
            eng.status.zero_()


def test_one_plan_for_a_graph_whose_lengths_grow():
    """The decode alone is captured, behind a plan of its first lengths."""
    b, table, n = prefix_batch((700, 300, 1), 4, 8, 130, seed=64)
    d = to_device(b)
    eng = _engine(b, table)
    plen = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.empty((3, 32, 512), dtype=torch.bfloat16, device="cuda")
    lse, pt = torch.empty((3, 32), device="cuda"), table.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d["lens"].copy_(torch.tensor((250, 300, 0), dtype=torch.int32))
        eng.plan(d["lens"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            eng.decode(d["q"], d["kv"], pt, plen, d["bt"], d["lens"], *bmm_scales(b), out=out, lse=lse)
        for lens in ((250, 300, 0), (256, 300, 0), (257, 300, 1), (700, 300, 1), (0, 0, 0)):
            d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            g.replay()
            side.synchronize()
            assert int(eng.status.item()) == 0
            b.seq_lens = torch.tensor(lens, dtype=torch.int32)
            _check(out, lse, b, table, n, str(lens))


def test_decode_before_any_plan():
    """The first decode plans its lengths itself, on its own stream."""
    b, table, n = prefix_batch((300, 40, 0), 4, 8, 200, seed=65)
    _decode(_engine(b, table), b, table, n)
    d = to_device(b)
    eng, side = _engine(b, table), torch.cuda.Stream()
    eng.places.fill_(-7)                          # what an allocation may hold
    plen, pt = torch.tensor([n], dtype=torch.int32, device="cuda"), table.cuda()
    torch.cuda.synchronize()
    out, lse = eng.decode(d["q"], d["kv"], pt, plen, d["bt"], d["lens"], *bmm_scales(b), stream=side)
    side.synchronize()
    assert int(eng.status.item()) == 0 and eng.planned
    _check(out, lse, b, table, n)


def test_a_new_engine_leaves_no_fill_behind():
    """A plan on another stream is not overwritten by what the constructor put on its own:
    that stream is kept busy until after the plan."""
    b, table, n = prefix_batch((300, 40, 0), 4, 8, 200, seed=66)
    d = to_device(b)
    plen, pt = torch.tensor([n], dtype=torch.int32, device="cuda"), table.cuda()
    side, x = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    _engine(b, table).plan(d["lens"], side)       # its memory is there to take afterwards
    x @ x
    torch.cuda.synchronize()
    for _ in range(60):                           # some tens of ms on the current stream
        x = x @ x * 1e-2
    eng = _engine(b, table)
    eng.plan(d["lens"], side)
    side.synchronize()
    torch.cuda.synchronize()
    places = eng.places.tolist()
    assert places[0] == 0 and places[-1] > places[1] > 0
    _decode(eng, b, table, n)
