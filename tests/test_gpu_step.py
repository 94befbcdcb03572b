"""A step around the decode as one captured graph: absorbed queries, new tokens into the
cache, plan and decode, replayed with a cache that grows and inputs that change. Every
replay is compared with the oracle and with the same calls made eagerly."""
import numpy as np
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
import oracle.step as st
from tests.gpu_util import assert_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [130, 0])
@pytest.mark.parametrize("k,H,base", [(2, 8, (20, 63, 0)), (7, 3, (250, 0, 511, 5))])
def test_captured_step(k, H, base, prefix):
    """prefix 0: the regular decode on the same cache and queries."""
    R, steps, ks, qs, sm = len(base), 3, 6 / 448, 6 / 448, 1 / 192 ** 0.5
    g = torch.Generator().manual_seed(81 + k)
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    width = -(-(max(base) + (steps + 1) * k) // 64)
    shared = -(-prefix // 64)
    pages = R * width + shared + 2
    perm = torch.randperm(pages, generator=g).int()
    ptable, table = perm[:max(1, shared)].cuda(), perm[shared:shared + R * width].view(R, width).cuda()
    rope = mla.rope_table(prefix + max(base) + (steps + 1) * k + 1)
    weight = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda()
    w = (torch.randn((H, 128, 512), generator=g) / 128 ** 0.5).to(torch.bfloat16).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = torch.zeros((pages, 64, 576), dtype=torch.uint8, device="cuda")
    plen, status = torch.tensor([prefix], **i32), torch.zeros(1, **i32)
    if prefix:
        mla.kv_append(rand(prefix, 576).cuda(), kv, ptable[None].contiguous(), torch.zeros(1, **i32),
                      rope, ks, norm_weight=weight, status=status)
    zero, cu = torch.zeros(R, **i32), torch.tensor((0,) + base).cumsum(0).int().cuda()
    mla.kv_append(rand(sum(base), 576).cuda(), kv, table, zero, rope, ks, norm_weight=weight,
                  cu_tokens=cu, rope_starts=zero + prefix, status=status)
    q_in, new = rand(R * k, H, 192).cuda(), rand(R * k, 576).cuda()
    lens = torch.tensor(base, **i32)
    if prefix:
        eng = mla.PrefixMla(R, k, H, width, shared, pages, "cuda")
    else:
        eng = mla.FoldedMla(R, k, H, width, pages, "cuda", min_split_tokens=64)
    qc = torch.empty((R * k, H, 576), dtype=torch.uint8, device="cuda")
    out = torch.empty((R, k * H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((R, k * H), device="cuda")

    def step(cache, lens):
        starts = lens + prefix
        mla.query_absorb(q_in, w, rope, starts, qs, out=qc, status=status)
        mla.kv_append(new, cache, table, lens, rope, ks, norm_weight=weight, rope_starts=starts,
                      status=status)
        lens += k
        eng.plan(lens)
        if prefix:
            eng.decode(qc, cache, ptable, plen, table, lens, sm * qs * ks, ks, out=out, lse=lse)
        else:
            eng.decode(qc, cache, table, lens, sm * qs * ks, ks, out=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kv.clone(), lens.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(kv, lens)
        for i in range(steps):
            q_in.copy_(rand(R * k, H, 192))
            new.copy_(rand(R * k, 576))
            eager_kv, eager_lens = kv.clone(), lens.clone()
            graph.replay()
            got = [t.clone() for t in (qc, kv, lens, out, lse)]
            step(eager_kv, eager_lens)
            side.synchronize()
            assert int(status.item()) == 0 and int(eng.status.item()) == 0
            for a, b in zip(got, (qc, eager_kv, eager_lens, out, lse)):
                assert torch.equal(a, b)
            assert lens.tolist() == [n + (i + 1) * k for n in base]
            ro, rl, spread, reach = st.prefix_decode(
                qc.cpu().numpy(), kv.cpu().numpy(), ptable.cpu().numpy(), prefix, table.cpu().numpy(),
                lens.cpu().numpy(), k, sm, qs, ks)
            o, l = out.float().cpu().numpy(), lse.cpu().numpy()
            if prefix:                            # the bound of tests/test_gpu_prefix.py
                bound = (2.0 ** -7 + 2.0 ** -11) * spread + 2.0 ** -15 * reach + \
                    2.0 ** -8 * np.abs(ro) + 1e-6
                assert (np.abs(o - ro) <= bound).all() and np.abs(l - rl).max() <= 1e-3
            else:
                assert_close(o, l, ro, rl, f"step {i}")
