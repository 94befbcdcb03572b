"""Tensors that the bindings of prompt_attention, kv_weigh and kv_evict refuse: their pointers would be
read or written wrongly."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla

pytestmark = pytest.mark.gpu


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16, device="cuda")


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8, device="cuda")


def _prompt(**change):
    a = dict(q=_bf(5, 4, 192), k_nope=_bf(7, 2, 128), k_rope=_bf(7, 64), v=_bf(7, 2, 128), cu_tokens=_i32(0, 2, 5),
             sm_scale=0.1, cu_keys=_i32(0, 3, 7))
    a.update(change)
    return mla.prompt_attention(**a)


def test_prompt_accepts():
    out, lse = _prompt()
    assert out.shape == (5, 4, 128) and lse.shape == (5, 4)
    assert _prompt(return_lse=False)[1] is None
    kv = _bf(7, 2, 264)
    _prompt(k_nope=kv[..., :128], v=kv[..., 128:256], k_rope=_bf(7, 72)[:, :64])


@pytest.mark.parametrize("change", [
    lambda: dict(q=_bf(5, 4, 192).float()), lambda: dict(q=_bf(5, 4, 128)), lambda: dict(q=_bf(5, 768)),
    lambda: dict(q=_bf(5, 4, 384)[..., ::2]), lambda: dict(q=None), lambda: dict(k_nope=_bf(7, 2, 192)),
    lambda: dict(k_nope=_bf(7, 2, 128).cpu()), lambda: dict(k_nope=_bf(6, 2, 128)), lambda: dict(k_rope=_bf(6, 64)),
    lambda: dict(k_rope=_bf(7, 2, 64)), lambda: dict(v=_bf(7, 1, 128)), lambda: dict(v=_bf(7, 2, 128).half()),
    lambda: dict(cu_tokens=_i32(0)), lambda: dict(cu_tokens=_i32(0, 2, 5).long()),
    lambda: dict(cu_tokens=_i32(0, 9, 2, 9, 5)[::2]), lambda: dict(cu_keys=_i32(0, 7)), lambda: dict(cu_keys=None),
    lambda: dict(out=_bf(5, 4, 64)), lambda: dict(out=_bf(5, 4, 128).float()),
    lambda: dict(lse=torch.zeros(4, 5, device="cuda")), lambda: dict(status=_i32(0, 0)),
    lambda: dict(workspace=torch.zeros(1 << 24, device="cuda")),
])
def test_prompt(change):
    with pytest.raises(ValueError):
        _prompt(**change())


@pytest.mark.parametrize("change,code", [
    (lambda: dict(q=_bf(5, 3, 192)), -2),                               # 3 heads over 2
    (lambda: dict(q=_bf(5, 4, 196)[..., :192]), -7),
    (lambda: dict(q=_bf(1, 4, 192).expand(5, 4, 192)), -2),
    (lambda: dict(k_nope=_bf(7, 1, 128).expand(7, 2, 128)), -2),
    (lambda: dict(k_rope=_bf(1, 64).expand(7, 64)), -2),
    (lambda: dict(workspace=_u8(256)), -3), (lambda: dict(sm_scale=0.0), -2)])
def test_prompt_by_the_library(change, code):
    with pytest.raises(mla.MlaError) as e:
        _prompt(**change())
    assert e.value.code == code


def _weigh(**change):
    a = dict(q=_u8(4, 3, 576), kv=_u8(8, 64, 576), block_table=_i32(4, 5, 6, 7).view(2, 2), seq_lens=_i32(3, 9),
             lse=torch.zeros(2, 6, device="cuda"), bmm1_scale=1.0, weights=torch.zeros(2, 128, device="cuda"),
             starts=_i32(0, 0))
    a.update(change)
    mla.kv_weigh(**a)


def test_weigh_accepts():
    _weigh()
    _weigh(positions=torch.zeros(2, 128, dtype=torch.int32, device="cuda"), rope_starts=_i32(1, 2),
           status=_i32(0), q=_u8(4, 3, 576).view(torch.float8_e4m3fn), kv=_u8(8, 64, 576).view(torch.float8_e4m3fn))


@pytest.mark.parametrize("change", [
    lambda: dict(q=_u8(5, 3, 576)), lambda: dict(q=_u8(4, 3, 512)), lambda: dict(q=_bf(4, 3, 576)),
    lambda: dict(kv=_u8(8, 32, 576)), lambda: dict(kv=_u8(8, 64, 640)[..., :576]),
    lambda: dict(block_table=_i32(4, 5, 6, 7).view(2, 2).t()), lambda: dict(seq_lens=_i32(3)),
    lambda: dict(lse=torch.zeros(4, 3, device="cuda")), lambda: dict(lse=_bf(2, 6)),
    lambda: dict(weights=torch.zeros(2, 64, device="cuda")), lambda: dict(weights=_bf(2, 128)),
    lambda: dict(starts=_i32(0, 0).long()), lambda: dict(rope_starts=_i32(0)), lambda: dict(status=_i32()),
    lambda: dict(positions=torch.zeros(2, 128, device="cuda")), lambda: dict(starts=_i32(0, 0).cpu()),
])
def test_weigh(change):
    with pytest.raises(ValueError):
        _weigh(**change())


@pytest.mark.parametrize("change,code", [
    (lambda: dict(bmm1_scale=0.0), -2), (lambda: dict(decay=-1.0), -2),
    (lambda: dict(q=_u8(2 * 2048, 3, 576), lse=torch.zeros(2, 6144, device="cuda")), -2)])
def test_weigh_by_the_library(change, code):
    with pytest.raises(mla.MlaError) as e:
        _weigh(**change())
    assert e.value.code == code


def _evict(**change):
    a = dict(kv=_u8(8, 64, 576), block_table=_i32(4, 5, 6, 7).view(2, 2), seq_lens=_i32(3, 9),
             weights=torch.zeros(2, 128, device="cuda"), keep=_i32(2, 20))
    a.update(change)
    return mla.kv_evict(**a)


def _books(dtype=torch.float32, n=128):
    return torch.zeros(2, n, dtype=dtype, device="cuda")


def test_evict_accepts():
    assert _evict().tolist() == [2, 9]
    lens = _i32(3, 9)
    w, p = _books(), _books(torch.int32)
    assert _evict(seq_lens=lens, lens_out=lens, weights=w, weights_out=w, positions=p, positions_out=p) is lens


@pytest.mark.parametrize("change", [
    lambda: dict(kv=_u8(8, 64, 512)), lambda: dict(kv=_u8(8, 64, 576).cpu()), lambda: dict(block_table=_i32(4, 5)),
    lambda: dict(seq_lens=_i32(3, 9, 1)), lambda: dict(weights=_books(n=64)), lambda: dict(weights=_books().double()),
    lambda: dict(keep=2), lambda: dict(keep=_i32(2)), lambda: dict(positions=_books()),
    lambda: dict(positions_out=_books(torch.int32)), lambda: dict(weights_out=_books(n=64)),
    lambda: dict(lens_out=_i32(0)), lambda: dict(status=_i32(0, 0)), lambda: dict(workspace=_books()),
])
def test_evict(change):
    with pytest.raises(ValueError):
        _evict(**change())


def test_evict_outputs_that_overlap_their_input():
    flat = torch.zeros(3 * 128, device="cuda")
    with pytest.raises(ValueError):
        _evict(weights=flat[:256].view(2, 128), weights_out=flat[128:].view(2, 128))
    flat = torch.zeros(3 * 128, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        _evict(positions=flat[128:].view(2, 128), positions_out=flat[:256].view(2, 128))


@pytest.mark.parametrize("change,code", [(lambda: dict(recent=-1), -2), (lambda: dict(sinks=-1), -2),
                                         (lambda: dict(workspace=_u8(256)), -3)])
def test_evict_by_the_library(change, code):
    with pytest.raises(mla.MlaError) as e:
        _evict(**change())
    assert e.value.code == code
