"""The documented recipe of a bounded cache, run as it stands with the calls' contracts in place of the
kernels: after a prompt, the first and the newest tokens and the keys of most weight stay."""
import os
import re
import types

import numpy as np
import pytest
import torch

import oracle.cache as oc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
R, PAGES, KEEP, NEW = 2, 17, 512, 4


def _recipe():
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "kv_evict" in b]
    assert len(blocks) == 1
    books, step = blocks[0].replace('"cuda"', '"cpu"').split("# ... a step", 1)
    return books, "# ... a step" + step


def _kv_weigh(q, kv, table, lens, lse, bmm1, weights, starts, decay=1.0, positions=None, rope_starts=None):
    for r in range(R):
        at, n = int(starts[r]), int(lens[r])
        weights[r, :at] *= decay
        weights[r, at:n] = 0
        weights[r, :n] += q[r, :n]                 # here: what the step gives each key
        positions[r, at:n] = int(rope_starts[r]) + torch.arange(n - at, dtype=torch.int32)


def _kv_evict(kv, table, lens, weights, keep, positions=None, recent=0, sinks=0):
    new = lens.clone()
    for r in range(R):
        n = int(lens[r])
        kept, moves = oc.evict(n, weights[r].numpy(), positions[r].numpy(), int(keep[r]), recent, sinks)
        for a, b in moves:
            weights[r, b], positions[r, b] = weights[r, a], positions[r, a]
        new[r] = len(kept)
        weights[r, len(kept):n], positions[r, len(kept):n] = 0, -1
    return new


@pytest.mark.parametrize("prefix", [0, 300])
def test_newest_and_heaviest_keys_stay_after_a_prompt(prefix):
    books, step = _recipe()
    rng = np.random.default_rng(prefix)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    env = dict(torch=torch, mla=types.SimpleNamespace(kv_weigh=_kv_weigh, kv_evict=_kv_evict), R=R,
               max_pages=PAGES, prefix=prefix, kv=None, block_table=None, lse=None, bmm1_scale=1.0,
               keep=i32(KEEP, KEEP), cached=i32(1000, 700))
    exec(books, env)
    ends = [prefix + 1000, prefix + 700]
    for turn in range(3):
        given = torch.from_numpy(rng.random((R, PAGES * 64)).astype(np.float32))
        env.update(qc=given, starts=i32(*ends), lens=env["cached"] + NEW)
        before, had = env["positions"].clone(), env["cached"].tolist()
        exec(step, env)
        for r in range(R):
            ends[r] += NEW
            assert int(env["cached"][r]) == KEEP
            now = set(env["positions"][r, :KEEP].tolist())
            assert now.issuperset(range(ends[r] - 64, ends[r])), "the newest tokens"
            assert len(now) == KEEP
            if prefix == 0:
                assert now.issuperset(range(4)), "the first tokens"
            if turn == 0:                          # one step's weights: the largest of the rest
                rest = [j for j in range(had[r]) if int(before[r, j]) >= 4 and
                        int(before[r, j]) < ends[r] - 64]
                want = sorted(rest, key=lambda j: (-float(given[r, j]), j))[:KEEP - 64 - 4 * (prefix == 0)]
                assert now.issuperset(int(before[r, j]) for j in want)
