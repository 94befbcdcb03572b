"""Refusals of mla_prompt_attention, mla_kv_weigh and mla_kv_evict, on the host: nothing here launches
a kernel. The C entries get aligned pointers that are never read; the binding's checks refuse
CPU tensors before anything else."""
import ctypes

import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from mla_decode_attention_folded_gb300 import _lib

P = ctypes.c_void_p(1 << 20)                       # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD2 = ctypes.c_void_p((1 << 20) + 2)
NULL, SHAPE, WORKSPACE, UNSUPPORTED, ALIGN = -1, -2, -3, -5, -7
BIG = 1 << 40


def _weigh(shape=None, *, ptr=None, bmm1=0.1, decay=1.0, **fields):
    s = _lib.CacheShape(2, 3, 8, 64, 4, 10)
    for name, value in fields.items():
        setattr(s, name, value)
    at = dict(q=P, kv=P, table=P, lens=P, lse=P, starts=P, rope_starts=None, weights=P, positions=None,
              status=None)
    at.update(ptr or {})
    return _lib.load().mla_kv_weigh(
        ctypes.byref(s) if shape is None else shape, at["q"], at["kv"], at["table"], at["lens"],
        at["lse"], bmm1, decay, at["starts"], at["rope_starts"], at["weights"], at["positions"],
        at["status"], None)


@pytest.mark.parametrize("fields,code", [
    (dict(page_size=32), UNSUPPORTED), (dict(R=0), SHAPE), (dict(R=1025), SHAPE), (dict(k=0), SHAPE),
    (dict(H=0), SHAPE), (dict(k=1025, H=4), SHAPE), (dict(k=1 << 20, H=1 << 20), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(max_pages=(1 << 20) + 1), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(num_pages=1 << 25), SHAPE)])
def test_weigh_shapes_refused(fields, code):
    assert _weigh(**fields) == code


@pytest.mark.parametrize("name", ["q", "kv", "table", "lens", "lse", "starts", "weights"])
def test_weigh_null_pointers_refused(name):
    assert _weigh(ptr={name: None}) == NULL


@pytest.mark.parametrize("name,at", [("q", ODD), ("kv", ODD), ("table", ODD2), ("lens", ODD2), ("lse", ODD2),
                                     ("starts", ODD2), ("rope_starts", ODD2), ("weights", ODD2),
                                     ("positions", ODD2), ("status", ODD2)])
def test_weigh_alignment_refused(name, at):
    assert _weigh(ptr={name: at}) == ALIGN


@pytest.mark.parametrize("kw", [dict(bmm1=0.0), dict(bmm1=-1.0), dict(bmm1=float("nan")),
                                dict(bmm1=float("inf")), dict(decay=-0.5), dict(decay=float("nan")),
                                dict(decay=float("inf"))])
def test_weigh_numbers_refused(kw):
    assert _weigh(**kw) == SHAPE


def test_weigh_wait_test_limits():
    f = _lib.load().mla_kv_weigh_wait_test
    s = _lib.CacheShape(2, 3, 8, 64, 4, 10)
    args = [ctypes.byref(s), P, P, P, P, P, 0.1, 1.0, P, None, P, None]
    assert f(*args, None, 10_000_000, None) == NULL
    assert f(*args, P, 999_999, None) == SHAPE and f(*args, P, 2_000_000_001, None) == SHAPE
    assert _lib.load().mla_kv_weigh(None, *args[1:], None, None) == NULL


def _evict(shape=None, *, ptr=None, recent=0, sinks=0, ws=BIG, **fields):
    s = _lib.CacheShape(2, 0, 0, 64, 4, 10)        # k and H are not looked at
    for name, value in fields.items():
        setattr(s, name, value)
    at = dict(kv=P, table=P, lens=P, weights=P, positions=None, keep=P, weights_out=P, positions_out=None,
              lens_out=P, workspace=P, status=None)
    at.update(ptr or {})
    return _lib.load().mla_kv_evict(
        ctypes.byref(s) if shape is None else shape, at["kv"], at["table"], at["lens"], at["weights"],
        at["positions"], at["keep"], recent, sinks, at["weights_out"], at["positions_out"],
        at["lens_out"], at["workspace"], ws, at["status"], None)


@pytest.mark.parametrize("fields,code", [
    (dict(page_size=128), UNSUPPORTED), (dict(R=0), SHAPE), (dict(R=1025), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(max_pages=(1 << 20) + 1), SHAPE), (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 25), SHAPE)])
def test_evict_shapes_refused(fields, code):
    assert _evict(**fields) == code


@pytest.mark.parametrize("name", ["kv", "table", "lens", "weights", "keep", "weights_out", "lens_out",
                                  "workspace"])
def test_evict_null_pointers_refused(name):
    assert _evict(ptr={name: None}) == NULL


def test_evict_positions_come_in_pairs():
    assert _evict(ptr=dict(positions=P)) == NULL and _evict(ptr=dict(positions_out=P)) == NULL


@pytest.mark.parametrize("name,at", [("kv", ODD), ("workspace", ODD), ("table", ODD2), ("lens", ODD2),
                                     ("weights", ODD2), ("keep", ODD2), ("weights_out", ODD2),
                                     ("lens_out", ODD2), ("status", ODD2)])
def test_evict_alignment_refused(name, at):
    assert _evict(ptr={name: at}) == ALIGN


def test_evict_numbers_and_workspace_refused():
    assert _evict(recent=-1) == SHAPE and _evict(sinks=-1) == SHAPE
    need = mla.kv_evict_workspace_bytes(2, 4)
    assert need >= 2 * 4 * 32 * 8 + 2 * 4
    assert _evict(ws=need - 1) == WORKSPACE
    n = ctypes.c_size_t(0)
    f = _lib.load().mla_kv_evict_workspace_bytes
    assert f(None, ctypes.byref(n)) == NULL
    assert f(ctypes.byref(_lib.CacheShape(2, 0, 0, 64, 4, 10)), None) == NULL
    assert f(ctypes.byref(_lib.CacheShape(0, 0, 0, 64, 4, 10)), ctypes.byref(n)) == SHAPE


def _prompt(shape=None, *, ptr=None, scale=0.1, ws=BIG, **fields):
    s = _lib.PromptShape(2, 10, 12, 8, 4, 1, 152, 8 * 192, 192, 4 * 256, 256, 4 * 256, 256, 64)
    for name, value in fields.items():
        setattr(s, name, value)
    at = dict(q=P, kn=P, kr=P, v=P, cu=P, ck=None, workspace=P, out=P, lse=None, status=None)
    at.update(ptr or {})
    return _lib.load().mla_prompt_attention(
        ctypes.byref(s) if shape is None else shape, at["q"], at["kn"], at["kr"], at["v"], at["cu"], at["ck"],
        scale, at["workspace"], ws, at["out"], at["lse"], at["status"], None)


@pytest.mark.parametrize("fields,code", [
    (dict(R=0), SHAPE), (dict(R=1025), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 24) + 1), SHAPE),
    (dict(keys=-1), SHAPE), (dict(keys=(1 << 24) + 1), SHAPE), (dict(H=0), SHAPE), (dict(H=4097), SHAPE),
    (dict(kv_heads=0), SHAPE), (dict(kv_heads=3), SHAPE), (dict(kv_heads=16), SHAPE), (dict(causal=2), SHAPE),
    (dict(causal=-1), SHAPE), (dict(num_ctas=0), SHAPE), (dict(num_ctas=2049), SHAPE),
    (dict(q_token_stride=184), SHAPE), (dict(q_head_stride=184), SHAPE), (dict(k_token_stride=120), SHAPE),
    (dict(k_head_stride=120), SHAPE), (dict(v_token_stride=120), SHAPE), (dict(v_head_stride=120), SHAPE),
    (dict(rope_stride=56), SHAPE), (dict(q_token_stride=1540), ALIGN), (dict(q_head_stride=196), ALIGN),
    (dict(k_token_stride=1028), ALIGN), (dict(v_head_stride=132), ALIGN), (dict(rope_stride=68), ALIGN)])
def test_prompt_shapes_refused(fields, code):
    assert _prompt(**fields) == code


@pytest.mark.parametrize("name", ["q", "kn", "kr", "v", "cu", "workspace", "out"])
def test_prompt_null_pointers_refused(name):
    assert _prompt(ptr={name: None}) == NULL


@pytest.mark.parametrize("name,at", [("q", ODD), ("kn", ODD), ("kr", ODD), ("v", ODD), ("out", ODD),
                                     ("out", ctypes.c_void_p((1 << 20) + 16)), ("workspace", ODD),
                                     ("cu", ODD2), ("ck", ODD2), ("lse", ODD2), ("status", ODD2)])
def test_prompt_alignment_refused(name, at):
    assert _prompt(ptr={name: at}) == ALIGN


def test_prompt_numbers_and_workspace_refused():
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _prompt(scale=scale) == SHAPE
    need = mla.prompt_workspace_bytes(2, num_ctas=152)
    assert _prompt(ws=need - 1) == WORKSPACE
    assert _prompt(tokens=0, ptr=dict(q=None, out=None, workspace=None)) == 0
    n = ctypes.c_size_t(0)
    f = _lib.load().mla_prompt_workspace_bytes
    assert f(None, ctypes.byref(n)) == NULL
    assert _lib.load().mla_prompt_attention(None, P, P, P, P, P, None, 0.1, P, BIG, P, None, None, None) == NULL
    s = _lib.PromptShape(2, 10, 12, 8, 4, 1, 152, 8 * 192, 192, 1024, 256, 1024, 256, 64)
    assert f(ctypes.byref(s), None) == NULL
    g = _lib.load().mla_prompt_attention_wait_test
    args = [ctypes.byref(s), P, P, P, P, P, None, 0.1, P, BIG, P, None]
    assert g(*args, None, 10_000_000, None) == NULL
    assert g(*args, P, 999_999, None) == SHAPE and g(*args, P, 2_000_000_001, None) == SHAPE


def test_the_binding_refuses_cpu_tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    kv, table = torch.zeros(4, 64, 576, dtype=torch.uint8), i32(0, 1, 2, 3).view(2, 2)
    with pytest.raises(ValueError):
        mla.prompt_attention(bf(4, 2, 192), bf(4, 2, 128), bf(4, 64), bf(4, 2, 128), i32(0, 4), 0.1)
    with pytest.raises(ValueError):
        mla.kv_weigh(torch.zeros(2, 3, 576, dtype=torch.uint8), kv, table, i32(3, 4), torch.zeros(2, 3), 1.0,
                     torch.zeros(2, 128), i32(0, 0))
    with pytest.raises(ValueError):
        mla.kv_evict(kv, table, i32(3, 4), torch.zeros(2, 128), i32(2, 2))
