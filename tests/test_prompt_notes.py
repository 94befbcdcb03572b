"""Notes of values that are no numbers (mla_prompt_attention): four pieces have places for them, and no
reader may lose one. Shown on a model of the pair of CTAs; on the GPU, batches in which a half has no tiles in many pieces on end."""
import itertools
import math
import os
import re

import pytest
import torch

from mla_decode_attention_folded_gb300 import build

PLACES = 4


def _kernel():
    text = open(os.path.join(build.CSRC, "prompt.cu")).read()
    return re.sub(r"//[^\n]*", "", text)


def _waits():
    """Whether whoever notes waits for the other CTA's V warp to have taken the piece before, as the
    source has it."""
    body = _kernel().split("uint32_t odd = 0;", 1)[1].split("red.relaxed.cluster", 1)[0]
    return "wait_v_piece(ctl, seq, a)" in body


def _run(pieces, waits, held=None):
    """Two CTAs over a line of pieces (tiles, 0 or 1, of each half), every warp as far as it gets; `held`
    (CTA, half, piece): that softmax does not leave the piece. Each step waits only for others to be far
    enough, so no other order of steps gets any warp further. Returns how many pieces each CTA's V warp
    has left, and the softmaxes."""
    n = len(pieces)
    tiles = [max(p) for p in pieces]
    before = [sum(tiles[:i]) for i in range(n + 1)]
    given, copied, v_taken, v_left = [0, 0], [0, 0], [0, 0], [0, 0]
    taken, made, left = ([[0, 0], [0, 0]] for _ in range(3))     # [CTA][half]: softmax: piece, weights, output
    m_taken, m_left = [0, 0], [0, 0]                             # MMA warps of the first CTA
    moved = True
    while moved:
        moved = False

        def step(row, at, ok):
            nonlocal moved
            if ok:
                row[at] += 1
                moved = True

        for c in (0, 1):
            # A piece is handed on once all have taken the one two before it, its predecessor's tiles under way.
            slow = min([v_taken[c], *taken[c]] + (m_taken if c == 0 else []))
            step(given, c, given[c] < n and slow >= given[c] - 1 and copied[c] >= before[given[c]])
            # Three tiles of V in flight; a place is free once both halves' MMAs have left the piece.
            step(copied, c, copied[c] < before[given[c]] and copied[c] - 3 < before[min(m_left)])
            step(v_taken, c, v_taken[c] == v_left[c] < given[c])
            x = v_left[c]
            step(v_left, c, v_taken[c] > x and copied[c] >= before[x + 1] and
                 (not waits or not tiles[x] or v_taken[1 - c] >= x))
            for h in (0, 1):
                step(taken[c], h, taken[c][h] == left[c][h] < given[c])
                x = made[c][h]
                step(made[c], h, taken[c][h] > x and (not pieces[x][h] or m_taken[h] > x))
                x = left[c][h]
                step(left[c], h, made[c][h] > x and (not pieces[x][h] or m_left[h] > x) and (c, h, x) != held)
        for h in (0, 1):
            step(m_taken, h, m_taken[h] == m_left[h] < given[0])
            x = m_left[h]
            # Left with both CTAs' V, and where the half has tiles both CTAs' weights.
            step(m_left, h, m_taken[h] > x and (not tiles[x] or min(v_left) > x) and
                 (not pieces[x][h] or min(made[0][h], made[1][h]) > x))
    return v_left, left


def _lost(pieces, waits):
    """Whether a note can be written over before its reader has read it."""
    assert _run(pieces, waits) == ([len(pieces)] * 2, [[len(pieces)] * 2] * 2), "stuck"
    for c, h, x in itertools.product((0, 1), (0, 1), range(len(pieces) - PLACES)):
        v_left, _ = _run(pieces, waits, (c, h, x))
        if pieces[x][h] and any(v > x + PLACES and max(pieces[x + PLACES]) for v in v_left):
            return True
    return False


KINDS = [(1, 1), (1, 0), (0, 1), (0, 0)]


def test_the_model_loses_notes_without_the_wait():
    assert not _lost([(1, 1)] * 9, False)
    assert _lost([(1, 1), (1, 0), (1, 1), (1, 0), (1, 1), (1, 0)], False)
    assert _lost([(1, 1), (0, 0), (0, 0), (0, 0), (1, 1)], False)


def test_no_note_is_written_over_before_it_is_read():
    waits = _waits()
    for n in (5, 6):
        for batch in itertools.product(KINDS, repeat=n):
            assert not _lost(list(batch), waits), batch


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_notes_of_many_short_pieces(seed):
    """Short requests on an odd number of heads, many without keys: every NaN reaches the rows and dims
    that see it, in every run."""
    import mla_decode_attention_folded_gb300 as mla
    g = torch.Generator().manual_seed(seed)
    R, H = 300, (1, 3, 5, 2)[seed]
    n = torch.randint(1, 257, (R,), generator=g).tolist()
    m = [0 if x < 0.5 else int(1 + 400 * x * x) for x in torch.rand(R, generator=g).tolist()]
    cu, ck = list(itertools.accumulate(n, initial=0)), list(itertools.accumulate(m, initial=0))
    dev = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=dev, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kn, kr, v = rand(cu[-1], H, 192), rand(ck[-1], H, 128), rand(ck[-1], 64), rand(ck[-1], H, 128)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32(cu), 1 / math.sqrt(192), i32(ck))
    want, want_l = mla.prompt_attention(q, kn, kr, v, *args)
    hit = torch.zeros(cu[-1], H, 128, dtype=torch.bool, device="cuda")
    for r in range(R):
        for h in range(H):
            for _ in range(2 if m[r] else 0):
                j = int(torch.randint(max(0, m[r] - n[r]), m[r], (1,), generator=g))
                d = int(torch.randint(0, 128, (1,), generator=g))
                v[ck[r] + j, h, d] = math.nan
                hit[cu[r] + max(0, j - (m[r] - n[r])):cu[r + 1], h, d] = True
    status = i32([0])
    for _ in range(20):
        out, lse = mla.prompt_attention(q, kn, kr, v, *args, status=status)
        assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], want[~hit]) and torch.equal(lse, want_l)
    assert int(status.item()) == 0
