"""Tensors the binding of the calls around the decode refuses: their pointers
would be read or written wrongly."""
import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from tests.step_util import angle_table

pytestmark = pytest.mark.gpu


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _append(**change):
    a = dict(kv_new=torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda"),
             kv=torch.zeros(4, 64, 576, dtype=torch.uint8, device="cuda"),
             block_table=_i32(0, 1, 2, 3).view(2, 2), starts=_i32(0, 0),
             rope=angle_table(80).cuda(), kv_scale=1.0)
    a.update(change)
    mla.kv_append(**a)


@pytest.mark.parametrize("change", [
    lambda: dict(kv=torch.zeros(4, 64, 576, dtype=torch.int8, device="cuda")),
    lambda: dict(kv=torch.zeros(4, 32, 576, dtype=torch.uint8, device="cuda")),
    lambda: dict(kv=torch.zeros(4, 64, 640, dtype=torch.uint8, device="cuda")[:, :, :576]),
    lambda: dict(kv_new=torch.zeros(4, 576, device="cuda")),
    lambda: dict(kv_new=torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(kv_new=torch.zeros(4, 576, dtype=torch.bfloat16)),
    lambda: dict(kv_new=torch.zeros(576, 4, dtype=torch.bfloat16, device="cuda").t()),
    lambda: dict(block_table=_i32(0, 1, 2, 3)),
    lambda: dict(block_table=_i32(0, 1, 2, 3).view(2, 2).long()),
    lambda: dict(block_table=_i32(0, 1, 2, 3).view(2, 2).t()),
    lambda: dict(starts=_i32(0)),
    lambda: dict(starts=torch.zeros(2, dtype=torch.int64, device="cuda")),
    lambda: dict(rope=angle_table(80).cuda()[:, :32]),
    lambda: dict(rope=angle_table(80).cuda().double()),
    lambda: dict(norm_weight=torch.zeros(512, device="cuda")),
    lambda: dict(norm_weight=torch.zeros(576, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(cu_tokens=_i32(0, 4)),
    lambda: dict(rope_starts=_i32(0)),
    lambda: dict(status=_i32(0, 0)),
])
def test_append(change):
    with pytest.raises(ValueError):
        _append(**change())


@pytest.mark.parametrize("change,code", [
    (lambda: dict(kv_new=torch.zeros(5, 576, dtype=torch.bfloat16, device="cuda")), -2),
    (lambda: dict(kv_new=torch.zeros(4, 580, dtype=torch.bfloat16, device="cuda")[:, :576]), -7),
    (lambda: dict(kv_new=torch.zeros(4, 584, dtype=torch.bfloat16, device="cuda")[:, 4:580]), -7),
    (lambda: dict(kv_new=torch.zeros(1, 576, dtype=torch.bfloat16, device="cuda").expand(4, 576)), -2),
    (lambda: dict(kv_scale=0.0), -2)])
def test_append_by_the_library(change, code):
    with pytest.raises(mla.MlaError) as e:
        _append(**change())
    assert e.value.code == code


def _absorb(**change):
    a = dict(q=torch.zeros(4, 3, 192, dtype=torch.bfloat16, device="cuda"),
             w_uk=torch.zeros(3, 128, 512, dtype=torch.bfloat16, device="cuda"),
             rope=angle_table(80).cuda(), rope_starts=_i32(0, 0), q_scale=1.0)
    a.update(change)
    mla.query_absorb(**a)


@pytest.mark.parametrize("change", [
    lambda: dict(q=torch.zeros(4, 3, 192, device="cuda")),
    lambda: dict(q=torch.zeros(4, 3, 128, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(q=torch.zeros(5, 3, 192, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(q=torch.zeros(0, 3, 192, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(w_uk=torch.zeros(3, 512, 128, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(w_uk=torch.zeros(2, 128, 512, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(rope_starts=_i32(0, 0).long()),
    lambda: dict(rope_starts=_i32()),
    lambda: dict(rope=angle_table(80)),
    lambda: dict(out=torch.zeros(4, 3, 512, dtype=torch.uint8, device="cuda")),
    lambda: dict(out=torch.zeros(4, 3, 576, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(status=torch.zeros(1, device="cuda")),
])
def test_absorb(change):
    with pytest.raises(ValueError):
        _absorb(**change())


@pytest.mark.parametrize("change,code", [
    (lambda: dict(q=torch.zeros(4, 3, 196, dtype=torch.bfloat16, device="cuda")[:, :, :192]), -7),
    (lambda: dict(q=torch.zeros(4, 1, 192, dtype=torch.bfloat16, device="cuda").expand(4, 3, 192)), -2),
    (lambda: dict(q_scale=float("nan")), -2)])
def test_absorb_by_the_library(change, code):
    with pytest.raises(mla.MlaError) as e:
        _absorb(**change())
    assert e.value.code == code


def _prefix(**change):
    eng = mla.PrefixMla(2, 2, 3, 2, 4, 8, "cuda")
    a = dict(q=torch.zeros(4, 3, 576, dtype=torch.uint8, device="cuda"),
             kv=torch.zeros(8, 64, 576, dtype=torch.uint8, device="cuda"),
             prefix_table=_i32(0, 1, 2, 3), prefix_len=_i32(5),
             block_table=_i32(4, 5, 6, 7).view(2, 2), seq_lens=_i32(3, 9), bmm1_scale=1.0,
             bmm2_scale=1.0)
    a.update(change)
    eng.plan(_i32(3, 9))
    return eng.decode(**a)


def test_prefix_accepts():
    out, lse = _prefix()
    assert out.shape == (2, 6, 512) and lse.shape == (2, 6)
    assert _prefix(return_lse=False)[1] is None


@pytest.mark.parametrize("change", [
    lambda: dict(q=torch.zeros(4, 3, 576, device="cuda")),
    lambda: dict(q=torch.zeros(4, 4, 576, dtype=torch.uint8, device="cuda")),
    lambda: dict(kv=torch.zeros(7, 64, 576, dtype=torch.uint8, device="cuda")),
    lambda: dict(kv=torch.zeros(8, 64, 576, dtype=torch.uint8)),
    lambda: dict(prefix_table=_i32(0, 1, 2)),
    lambda: dict(prefix_table=_i32(0, 1, 2, 3).long()),
    lambda: dict(prefix_len=5),
    lambda: dict(prefix_len=_i32(5, 5)),
    lambda: dict(block_table=_i32(4, 5, 6, 7).view(2, 2).t()),
    lambda: dict(seq_lens=_i32(3)),
    lambda: dict(out=torch.zeros(2, 6, 512, device="cuda")),
    lambda: dict(out=torch.zeros(4, 3, 512, dtype=torch.bfloat16, device="cuda")),
    lambda: dict(lse=torch.zeros(2, 6, dtype=torch.bfloat16, device="cuda")),
])
def test_prefix(change):
    with pytest.raises(ValueError):
        _prefix(**change())


def test_prefix_by_the_library():
    with pytest.raises(mla.MlaError) as e:
        _prefix(bmm1_scale=0.0)
    assert e.value.code == -2
    with pytest.raises(ValueError):
        mla.PrefixMla(2, 2, 3, 2, 4, 8, "cuda").plan(torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(mla.MlaError):
        mla.PrefixMla(2000, 2, 3, 2, 4, 8, "cuda")
