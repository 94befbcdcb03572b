"""What the binding of kv_evict refuses before anything is launched, on CPU tensors that stand for
the device's."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla


class Launched(Exception):
    pass


@pytest.fixture
def evict(monkeypatch):
    """kv_evict with all checks of places passed and the library out of reach."""
    def load():
        raise Launched

    monkeypatch.setattr(mla.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mla, "_device", lambda name, t, dims: 0)
    monkeypatch.setattr(mla, "_check", lambda dev, name, t, dtypes, shape: None)
    monkeypatch.setattr(mla._lib, "load", load)

    def call(**change):
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        a = dict(kv=torch.zeros(8, 64, 576, dtype=torch.uint8), block_table=i32(4, 5, 6, 7).view(2, 2),
                 seq_lens=i32(3, 9), weights=torch.zeros(2, 128), keep=i32(2, 20),
                 workspace=torch.zeros(1 << 12, dtype=torch.uint8))
        a.update(change)
        return mla.kv_evict(**a)

    return call


def test_lens_out(evict):
    flat = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(Launched):
        evict()
    with pytest.raises(Launched):                  # seq_lens itself, or apart
        evict(seq_lens=flat[:2], lens_out=flat[:2], keep=flat[2:4])
    with pytest.raises(Launched):
        evict(seq_lens=flat[:2], lens_out=flat[2:4], keep=flat[4:6])
    for a, b in ((0, 1), (1, 0)):
        with pytest.raises(ValueError, match="lens_out"):
            evict(seq_lens=flat[a:a + 2], lens_out=flat[b:b + 2])
        with pytest.raises(ValueError, match="lens_out"):
            evict(keep=flat[a:a + 2], lens_out=flat[b:b + 2])
    with pytest.raises(ValueError, match="lens_out"):
        evict(keep=flat[:2], lens_out=flat[:2])


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, -2 ** 32 + 5, 2 ** 63])
def test_counts_beyond_32_bits(evict, value):
    """They would reach the library as other numbers: 2^32 + 5 as 5."""
    for name in ("recent", "sinks"):
        with pytest.raises(ValueError, match=name):
            evict(**{name: value})
        with pytest.raises(Launched):
            evict(**{name: 2 ** 31 - 1})
