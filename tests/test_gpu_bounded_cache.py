"""The operators as they are used together: prompts attended to and cached, decode steps whose weights
are summed, a cache that stays within its budget; eager against the oracle, and as one captured
graph against the eager calls, bit for bit."""
import math

import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.attention as att
import oracle.cache as oc
import oracle.e4m3 as e4m3
from tests.gpu_util import ATOL, LSE_TOL, RTOL
from tests.prompt_util import check, reference
from tests.step_util import angle_table

pytestmark = pytest.mark.gpu

SM = 1 / math.sqrt(192)
R, k, H, PAGES = 3, 2, 8, 4                       # pages of a request
BUDGET, RECENT, SINKS, DECAY = 150, 20, 4, 0.75
SCALE = 6 / 448


class Run:
    """A model's layer in small: projections drawn at random, prompts, then steps."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.kv = torch.zeros((R * PAGES + 1, 64, 576), dtype=torch.uint8, device="cuda")
        self.table = torch.randperm(R * PAGES, generator=g, device="cuda").int().view(R, PAGES).contiguous()
        self.weights = torch.full((R, PAGES * 64), 9.0, device="cuda")
        self.positions = torch.full((R, PAGES * 64), -1, dtype=torch.int32, device="cuda")
        self.rope, self.w_uk = angle_table(1024).cuda(), (self.rand(H, 128, 512) / 128 ** 0.5)
        self.w_norm = (1 + 0.1 * self.rand(512)).to(torch.bfloat16)
        self.lens, self.ends = self.i32([0] * R), self.i32([0] * R)      # cached keys, next positions
        self.keep, self.status = self.i32([BUDGET] * R), self.i32([0])
        self.eng = mla.FoldedMla(R, k, H, PAGES, self.kv.shape[0], "cuda")
        self.bmm1 = float(np.float32(SM * SCALE * SCALE))
        self.q, self.new = self.rand(R * k, H, 192), self.rand(R * k, 576)

    def step(self):
        """One decode step of k tokens a request (self.q, self.new); all state in place."""
        q = mla.query_absorb(self.q, self.w_uk, self.rope, self.ends, SCALE, status=self.status)
        mla.kv_append(self.new, self.kv, self.table, self.lens, self.rope, SCALE, norm_weight=self.w_norm,
                      rope_starts=self.ends, status=self.status)
        starts = self.lens.clone()
        self.lens += k
        self.eng.plan(self.lens)
        out, lse = self.eng.decode(q, self.kv, self.table, self.lens, self.bmm1, SCALE)
        mla.kv_weigh(q, self.kv, self.table, self.lens, lse, self.bmm1, self.weights, starts, decay=DECAY,
                     positions=self.positions, rope_starts=self.ends, status=self.status)
        self.ends += k
        before = self.lens.clone()
        mla.kv_evict(self.kv, self.table, self.lens, self.weights, self.keep, positions=self.positions,
                     recent=RECENT, sinks=SINKS, lens_out=self.lens, status=self.status)
        return q, out, lse, starts, before

    def faults(self):
        torch.cuda.synchronize()
        return int(self.status.item()), int(self.eng.status.item())

    def state(self):
        return [t.clone() for t in (self.kv, self.weights, self.positions, self.lens, self.ends)]


def _prompts(run, n):
    cu = [0]
    for v in n:
        cu.append(cu[-1] + v)
    T = cu[-1]
    q, kv, kr = run.rand(T, H, 192), run.rand(T, H, 256), run.rand(T, 64)
    out, lse = mla.prompt_attention(q, kv[..., :128], kr, kv[..., 128:], run.i32(cu), SM, status=run.status)
    check(out, lse, reference(q, kv[..., :128], kr, kv[..., 128:], cu, None, SM, True))
    mla.kv_append(run.rand(T, 576), run.kv, run.table, run.lens, run.rope, SCALE, norm_weight=run.w_norm,
                  cu_tokens=run.i32(cu), status=run.status)
    run.lens.copy_(run.i32(list(n)))
    run.ends.copy_(run.lens)
    # The books of what the prompt brought: the positions, and no weight yet.
    run.weights.zero_()
    run.positions.copy_(torch.arange(PAGES * 64, device="cuda", dtype=torch.int32).expand(R, -1))


def test_steps_of_a_bounded_cache():
    run = Run()
    n = [160, 37, 149]
    _prompts(run, n)
    books = [{j: 0.0 for j in range(v)} for v in n]          # position -> weight, by the oracle
    rows = {}                                                # (request, position) -> codes
    for s in range(4):
        run.q, run.new = run.rand(R * k, H, 192), run.rand(R * k, 576)
        kv0, w0, p0 = run.kv.cpu().numpy(), run.weights.cpu().numpy(), run.positions.cpu().numpy()
        lens0, ends0 = run.lens.tolist(), run.ends.tolist()
        q, out, lse, starts, before = run.step()
        assert run.faults() == (0, 0)
        table = run.table.cpu().numpy()
        assert starts.tolist() == lens0 and before.tolist() == [v + k for v in lens0]
        kv1, w1, p1 = run.kv.cpu().numpy(), run.weights.cpu().numpy(), run.positions.cpu().numpy()
        for r in range(R):
            old = {int(p0[r, j]): kv0[table[r, j // 64], j % 64] for j in range(lens0[r])}
            held = lens0[r] + k
            new_len = min(held, BUDGET)
            assert run.lens.tolist()[r] == new_len
            now = {int(p1[r, j]): (kv1[table[r, j // 64], j % 64], float(w1[r, j])) for j in range(new_len)}
            assert len(now) == new_len and (p1[r, new_len:held] == -1).all() and (w1[r, new_len:held] == 0).all()
            # Rows stay their positions' rows.
            for p, (codes, _) in now.items():
                if p in old:
                    assert np.array_equal(codes, old[p])
            # What was dropped weighs no more than what stayed, but for the held ones.
            gone = [p for p in old if p not in now]
            assert all(ends0[r] + i in now for i in range(k)) and all(p in now for p in range(SINKS))
            assert all(p in now for p in range(ends0[r] + k - RECENT, ends0[r] + k))
            # The decode, and every key's weight, over the keys as they were before the eviction.
            codes = np.stack([old[p] if p in old else now[p][0] for p in [*old, *range(ends0[r], ends0[r] + k)]])
            keys = e4m3.decode(codes) * float(SCALE)
            qd = e4m3.decode(q.cpu().numpy()[r * k:(r + 1) * k]).reshape(-1, 576) * float(SCALE)
            ref_o, ref_l = att.attend(qd, keys, SM)
            o = out.float().cpu().numpy().reshape(R, k * H, 512)[r]
            assert (np.abs(o - ref_o) <= ATOL + RTOL * np.abs(ref_o)).all()
            l = lse.cpu().numpy().reshape(R, k * H)[r]
            assert np.abs(l - ref_l).max() <= LSE_TOL
            got = np.exp2(SM / math.log(2) * (qd @ keys.T) - l[:, None].astype(np.float64)).sum(0)
            for i, p in enumerate([*old, *range(ends0[r], ends0[r] + k)]):
                books[r][p] = books[r].get(p, 0.0) * DECAY + got[i]
                if p in now:
                    assert abs(now[p][1] - books[r][p]) <= 1e-4 * books[r][p] + 1e-6
            free = [p for p in now if SINKS <= p < ends0[r] + k - RECENT]
            if gone and free:
                assert max(books[r][p] for p in gone) <= min(books[r][p] for p in free) * (1 + 1e-3)


def test_a_captured_step_equals_the_eager_one():
    eager, graph = Run(5), Run(5)
    for run in (eager, graph):
        _prompts(run, [100, 149, 120])
    assert all(torch.equal(a, b) for a, b in zip(eager.state(), graph.state()))
    saved = graph.state()
    graph.step()                                    # warm up, then back
    torch.cuda.synchronize()
    for t, v in zip((graph.kv, graph.weights, graph.positions, graph.lens, graph.ends), saved):
        t.copy_(v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = graph.step()
    for t, v in zip((graph.kv, graph.weights, graph.positions, graph.lens, graph.ends), saved):
        t.copy_(v)
    for s in range(30):                             # past the budget of every request
        q, new = eager.rand(R * k, H, 192), eager.rand(R * k, 576)
        for run in (eager, graph):
            run.q.copy_(q)
            run.new.copy_(new)
        want = eager.step()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), f"step {s}"
    assert eager.faults() == (0, 0) and graph.faults() == (0, 0)
    assert all(torch.equal(a, b) for a, b in zip(eager.state(), graph.state()))
    assert eager.lens.tolist() == [BUDGET] * R and eager.ends.tolist() == [160, 209, 180]


def test_a_prompts_cache_cut_down_by_its_last_tokens_attention():
    """The weights that the last tokens of a prompt give decide what stays; decoding over what stays is
    the oracle's over those keys."""
    run = Run(7)
    _prompts(run, [250, 200, 180])
    lens = run.lens.clone()
    q = mla.query_absorb(run.rand(R * k, H, 192), run.w_uk, run.rope, run.ends - k, SCALE)
    run.eng.plan(lens)
    _, lse = run.eng.decode(q, run.kv, run.table, lens, run.bmm1, SCALE)
    mla.kv_weigh(q, run.kv, run.table, lens, lse, run.bmm1, run.weights, torch.zeros_like(lens),
                 positions=run.positions)
    kv0, w0, table = run.kv.cpu().numpy(), run.weights.cpu().numpy(), run.table.cpu().numpy()
    keep = run.i32([64, 100, 180])
    new = mla.kv_evict(run.kv, run.table, lens, run.weights, keep, positions=run.positions, recent=16, sinks=2)
    run.eng.plan(new)
    out, _ = run.eng.decode(q, run.kv, run.table, new, run.bmm1, SCALE)
    for r, n in enumerate([250, 200, 180]):
        kept, _ = oc.evict(n, w0[r], range(256), int(keep[r]), 16, 2)
        keys = e4m3.decode(np.stack([kv0[table[r, j // 64], j % 64] for j in kept])) * float(SCALE)
        qd = e4m3.decode(q.cpu().numpy()[r * k:(r + 1) * k]).reshape(-1, 576) * float(SCALE)
        ref, _ = att.attend(qd, keys, SM)
        o = out.float().cpu().numpy().reshape(R, k * H, 512)[r]
        assert (np.abs(o - ref) <= ATOL + RTOL * np.abs(ref)).all()
        assert sorted(run.positions[r, :len(kept)].tolist()) == kept
