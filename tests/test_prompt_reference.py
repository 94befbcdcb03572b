"""The tests' 64-bit attention of packed prompts against scalar loops."""
import math

import torch

from tests.prompt_util import reference


def test_against_scalar_loops():
    g = torch.Generator().manual_seed(0)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    cu, ck = [0, 3, 3, 5, 7], [0, 4, 6, 6, 7]          # m = 4, 2, 0, 1 keys for n = 3, 0, 2, 2 tokens
    q, kn, kr, v = bf(8, 4, 192), bf(7, 2, 128), bf(7, 64), bf(7, 2, 128)
    for causal in (True, False):
        out, lse, _, _ = reference(q, kn, kr, v, cu, ck, 0.1, causal)
        for r in range(4):
            n, m = cu[r + 1] - cu[r], ck[r + 1] - ck[r]
            for i in range(n):
                for h in range(4):
                    seen = [j for j in range(m) if not causal or j <= i + m - n]
                    e, o = [], [0.0] * 128
                    for j in seen:
                        k = ck[r] + j
                        s = sum(float(q[cu[r] + i, h, d]) * float(kn[k, h // 2, d]) for d in range(128))
                        s += sum(float(q[cu[r] + i, h, 128 + d]) * float(kr[k, d]) for d in range(64))
                        e.append(math.exp(0.1 * s))
                    for x, j in zip(e, seen):
                        for d in range(128):
                            o[d] += x / sum(e) * float(v[ck[r] + j, h // 2, d])
                    row = cu[r] + i
                    want = math.log2(sum(e)) if e else -math.inf
                    assert want == lse[row, h] or abs(want - float(lse[row, h])) < 1e-12
                    assert max(abs(x - float(y)) for x, y in zip(o, out[row, h])) < 1e-12
        assert torch.isnan(out[7]).all()
