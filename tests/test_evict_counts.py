"""The counts of mla_kv_evict's select, which all CTAs of a cluster add to in the first one's shared
memory while that one adds its own: one width for all additions to a word, read from the source
(additions of two widths that overlap are a data race, which no run can be relied on to show); on
the GPU, keys that fall into neighbouring counts of every digit, on clusters of every size."""
import os
import re

import numpy as np
import pytest

from mla_decode_attention_folded_gb300 import build


def test_additions_to_a_count_have_one_width():
    text = open(os.path.join(build.CSRC, "evict.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    assert re.search(r"uint32_t hist\[3\]\[kBins\]", text)
    own = re.findall(r"atomicAdd\(&sh\.hist[^;]*;", text)
    assert own and all(a.endswith(", 1u);") for a in own)          # 32 bits
    remote = re.findall(r"\b(?:red|atom)\.[\w.:]*\.add\.(\w+)", text)
    assert remote and set(remote) == {"u32"}


# The code of a positive weight is its bits with the sign set; its digits are 11, 11 and 10 bits.
STEPS = {"first": 1 << 21, "second": 1 << 10, "third": 1}


@pytest.mark.gpu
@pytest.mark.parametrize("digit", STEPS)
@pytest.mark.parametrize("R,width", [(70, 70), (19, 300), (9, 300), (4, 600), (1, 1100)])
def test_neighbouring_counts(digit, R, width, monkeypatch):
    import tests.test_gpu_evict as base

    def weights(rng, shape, kind):
        at = rng.integers(0, 4, shape) * STEPS[digit]
        return (np.float32(1.0).view(np.int32) + at.astype(np.int32)).view(np.float32)

    monkeypatch.setattr(base, "_weights", weights)
    rng = np.random.default_rng(width + R)
    lens = [int(v) for v in rng.integers(width * 32, width * 64 + 1, R)]
    base._run(lens, [int(n * f) for n, f in zip(lens, rng.random(R))], recent=33, sinks=2, seed=R, width=width)
