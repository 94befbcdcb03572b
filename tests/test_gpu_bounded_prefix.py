"""A cache of bounded length behind a shared prefix: weights of the requests' own keys from the LSEs over
both, positions that go on from the prefix, an eviction, and decodes over what stays."""
import math

import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.attention as att
import oracle.cache as oc
import oracle.e4m3 as e4m3
from tests.gpu_util import ATOL, LSE_TOL, RTOL, bmm_scales
from tests.step_util import prefix_batch

pytestmark = pytest.mark.gpu


def _attend(out, lse, b, shared, own):
    """out and lse of a decode against the oracle's over the prefix's keys and each request's own."""
    for r in range(b.R):
        qd = e4m3.decode(b.q.numpy()[r * b.k:(r + 1) * b.k].reshape(b.M, 576)) * float(b.q_scale)
        ref_o, ref_l = att.attend(qd, np.concatenate([shared, own[r]]), b.sm_scale)
        o, l = out[r].float().cpu().numpy(), lse[r].cpu().numpy()
        assert (np.abs(o - ref_o) <= ATOL + RTOL * np.abs(ref_o)).all()
        assert np.abs(l - ref_l).max() <= LSE_TOL


@pytest.mark.parametrize("own,k,H,prefix", [((100, 37, 64), 4, 8, 300), ((700, 5, 333, 64), 7, 8, 64),
                                            ((600, 4, 130), 4, 64, 1000), ((65,), 1, 3, 1), ((90, 41), 2, 16, 0)])
def test_weights_eviction_and_decodes(own, k, H, prefix):
    b, table, prefix = prefix_batch(own, k, H, prefix, seed=sum(own) + prefix, fill=1 << 30)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rng = np.random.default_rng(prefix)
    bmm1, bmm2 = bmm_scales(b)
    q, kv, pt, bt, lens = b.q.cuda(), b.kv.cuda(), table.cuda(), b.block_table.cuda(), b.seq_lens.cuda()
    S = bt.shape[1] * 64
    starts = [n - k for n in own]                            # the step's k keys are the last; < 0: skipped
    positions = (prefix + torch.arange(S, dtype=torch.int32)).repeat(b.R, 1)
    for r, s in enumerate(starts):
        positions[r, s:] = -7                                # to be written
    w0, p0 = np.exp(rng.normal(size=(b.R, S))).astype(np.float32), positions.numpy().copy()
    positions = positions.cuda()
    weights, status = torch.from_numpy(w0).cuda(), i32([0])
    eng = mla.PrefixMla(b.R, k, H, bt.shape[1], pt.numel(), kv.shape[0], "cuda")
    eng.plan(lens)
    out, lse = eng.decode(q, kv, pt, i32([prefix]), bt, lens, bmm1, bmm2)
    shared = att.request_keys(b.kv.numpy(), table.numpy(), 0, prefix, b.kv_scale)
    keys = [att.request_keys(b.kv.numpy(), b.block_table[r].numpy(), 0, n, b.kv_scale) for r, n in enumerate(own)]
    _attend(out, lse, b, shared, keys)

    mla.kv_weigh(q, kv, bt, lens, lse, bmm1, weights, i32(starts), decay=0.5, positions=positions,
                 rope_starts=i32([prefix + s for s in starts]), status=status)
    got, at = weights.cpu().numpy(), positions.cpu().numpy()
    _, off = oc.key_weights(b.q.numpy(), b.kv.numpy(), np.where(b.block_table.numpy() == 1 << 30, 0, b.block_table),
                            own, lse.cpu().numpy(), k, bmm1)
    for r, n in enumerate(own):
        if starts[r] < 0:
            assert np.array_equal(got[r], w0[r]) and np.array_equal(at[r], p0[r])
            continue
        qd = e4m3.decode(b.q.numpy()[r * k:(r + 1) * k].reshape(b.M, 576)) * float(b.q_scale)
        x = b.sm_scale / math.log(2) * (qd @ np.concatenate([shared, keys[r]]).T)
        top = x.max(1, keepdims=True)
        p = np.exp2(x - top)
        sums = (p / p.sum(1, keepdims=True))[:, prefix:].sum(0)
        old = np.where(np.arange(n) < starts[r], 0.5 * w0[r, :n].astype(np.float64), 0.0)
        # The kernel's own bound around its LSE, and what that LSE may be off by (the decode's bound). bmm1 is
        # the scales' product in FP32, two roundings: 2^-23 of each score, in ln 2 of 2^x.
        scale = math.log(2) * np.abs(x).max() * 2.0 ** -23
        tol = off[r] + sums * np.expm1(math.log(2) * LSE_TOL + 2 * scale) + (old + sums) * 2.0 ** -22
        assert (np.abs(got[r, :n] - (old + sums)) <= tol).all(), f"request {r}"
        assert np.array_equal(got[r, n:], w0[r, n:])
        assert at[r, :n].tolist() == list(range(prefix, prefix + n)) and (at[r, n:] == -7).all()

    keep, recent, sinks = [max(1, n * 2 // 3) for n in own], k + 5, prefix + 3
    new = mla.kv_evict(kv, bt, lens, weights, i32(keep), positions=positions, recent=recent, sinks=sinks,
                       status=status)
    assert new.tolist() == keep
    kept = [oc.evict(n, got[r], at[r], keep[r], recent, sinks)[0] for r, n in enumerate(own)]
    for r, n in enumerate(own):
        slots = positions[r, :keep[r]].cpu().numpy() - prefix
        assert sorted(slots) == kept[r]
        assert np.array_equal(weights[r, :keep[r]].cpu().numpy(), got[r, slots])
        if keep[r] >= recent + 3:
            assert set(kept[r]).issuperset([0, 1, 2, *range(n - recent, n)])
    eng.plan(new)
    out, lse = eng.decode(q, kv, pt, i32([prefix]), bt, new, bmm1, bmm2)
    _attend(out, lse, b, shared, [keys[r][kept[r]] for r in range(b.R)])
    pages = table[:-(-prefix // 64)].long()
    assert torch.equal(kv.cpu()[pages], b.kv[pages]), "the prefix's keys changed"
    assert int(status.item()) == 0 and int(eng.status.item()) == 0


def test_captured_steps_behind_a_prefix_equal_eager_ones():
    """Append, decode, weigh and evict as one graph, replayed past the budget."""
    R, k, H, prefix, budget, scale = 3, 2, 8, 130, 60, 6 / 448
    sm = 1 / math.sqrt(192)

    class Side:
        def __init__(self):
            g = torch.Generator(device="cuda").manual_seed(3)
            rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
            i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
            self.kv = torch.zeros((8, 64, 576), dtype=torch.uint8, device="cuda")
            self.pt, self.bt, self.prefix = i32(6, 1, 4), i32(0, 2, 3).view(3, 1), i32(prefix)
            self.rope, self.w_uk = mla.rope_table(512, device="cuda"), rand(H, 128, 512) / 128 ** 0.5
            self.lens, self.ends = i32(40, 0, 7), i32(40, 0, 7) + prefix
            self.keep, self.status = i32(budget, 20, budget), i32(0)
            self.weights = torch.zeros((R, 64), device="cuda")
            self.positions = (prefix + torch.arange(64, dtype=torch.int32, device="cuda")).repeat(R, 1)
            self.q, self.new = rand(R * k, H, 192), rand(R * k, 576)
            self.eng = mla.PrefixMla(R, k, H, 1, 3, 8, "cuda")
            mla.kv_append(rand(prefix, 576), self.kv, self.pt[None], i32(0), self.rope, scale)
            mla.kv_append(rand(47, 576), self.kv, self.bt, i32(0, 0, 0), self.rope, scale, cu_tokens=i32(0, 40, 40, 47),
                          rope_starts=i32(prefix, prefix, prefix))

        def step(self):
            q = mla.query_absorb(self.q, self.w_uk, self.rope, self.ends, scale)
            mla.kv_append(self.new, self.kv, self.bt, self.lens, self.rope, scale, rope_starts=self.ends,
                          status=self.status)
            starts = self.lens.clone()
            self.lens += k
            self.eng.plan(self.lens)
            out, lse = self.eng.decode(q, self.kv, self.pt, self.prefix, self.bt, self.lens, sm * scale * scale, scale)
            mla.kv_weigh(q, self.kv, self.bt, self.lens, lse, sm * scale * scale, self.weights, starts, decay=0.9,
                         positions=self.positions, rope_starts=self.ends, status=self.status)
            self.ends += k
            mla.kv_evict(self.kv, self.bt, self.lens, self.weights, self.keep, positions=self.positions, recent=8,
                         sinks=prefix + 2, lens_out=self.lens, status=self.status)
            return out, lse

        def state(self):
            return self.kv, self.weights, self.positions, self.lens, self.ends

    eager, graph = Side(), Side()
    saved = [t.clone() for t in graph.state()]
    graph.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = graph.step()
    for t, v in zip(graph.state(), saved):
        t.copy_(v)
    rand = torch.Generator(device="cuda").manual_seed(4)
    for s in range(20):
        q = torch.randn((R * k, H, 192), generator=rand, device="cuda").to(torch.bfloat16)
        new = torch.randn((R * k, 576), generator=rand, device="cuda").to(torch.bfloat16)
        for side in (eager, graph):
            side.q.copy_(q)
            side.new.copy_(new)
        want = eager.step()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), f"step {s}"
    assert all(torch.equal(a, b) for a, b in zip(eager.state(), graph.state()))
    assert eager.lens.tolist() == [47 + 13, 20, 47] and int(eager.status.item()) == int(graph.status.item()) == 0
    for r, n in enumerate(eager.lens.tolist()):
        now = set(eager.positions[r, :n].tolist())
        end = int(eager.ends[r])
        assert len(now) == n and now.issuperset(range(end - 8, end)) and now.issuperset([prefix, prefix + 1])
