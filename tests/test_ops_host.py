"""Refusals of the calls around the decode, on the host: nothing here launches a
kernel. The C entries get aligned pointers that are never read; the binding's
checks refuse CPU tensors before anything else."""
import ctypes

import pytest
import torch

import mla_decode_attention_folded_gb300 as mla
from mla_decode_attention_folded_gb300 import _lib

P = ctypes.c_void_p(1 << 20)                       # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
NULL, SHAPE, UNSUPPORTED, ALIGN = -1, -2, -5, -7


def _append(shape=None, *, ptr=None, eps=1e-6, scale=0.1, **fields):
    s = _lib.AppendShape(2, 8, 64, 4, 10, 100, 1, 576)
    for name, value in fields.items():
        setattr(s, name, value)
    at = dict(x=P, w=None, rope=P, cu=None, starts=P, rope_starts=None, table=P, kv=P, status=None)
    at.update(ptr or {})
    return _lib.load().mla_kv_append(
        ctypes.byref(s) if shape is None else shape, at["x"], at["w"], eps, at["rope"], at["cu"],
        at["starts"], at["rope_starts"], at["table"], scale, at["kv"], at["status"], None)


@pytest.mark.parametrize("fields,code", [
    (dict(page_size=32), UNSUPPORTED), (dict(R=0), SHAPE), (dict(R=(1 << 20) + 1), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(tokens=7), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(max_pages=1 << 25), SHAPE), (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 25), SHAPE),
    (dict(rope_rows=0), SHAPE), (dict(interleaved=2), SHAPE), (dict(row_stride=568), SHAPE),
    (dict(row_stride=580), ALIGN)])
def test_append_shapes_refused(fields, code):
    assert _append(**fields) == code


@pytest.mark.parametrize("name", ["x", "rope", "starts", "table", "kv"])
def test_append_null_pointers_refused(name):
    assert _append(ptr={name: None}) == NULL


@pytest.mark.parametrize("name", ["x", "w", "kv"])
def test_append_alignment_refused(name):
    assert _append(ptr={name: ODD}) == ALIGN


@pytest.mark.parametrize("kw", [dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(scale=1e-45), dict(eps=-1e-6),
                                dict(eps=float("nan")), dict(eps=float("inf"))])
def test_append_numbers_refused(kw):
    assert _append(**kw) == SHAPE


def test_append_without_tokens_needs_no_pointers():
    assert _append(tokens=0, ptr=dict(x=None, kv=None)) == 0
    assert _lib.load().mla_kv_append(None, P, None, 1e-6, P, None, P, None, P, 1.0, P, None,
                                     None) == NULL


def _absorb(*, ptr=None, scale=0.1, **fields):
    s = _lib.QueryShape(2, 4, 8, 100, 1, 8 * 192, 192)
    for name, value in fields.items():
        setattr(s, name, value)
    at = dict(q=P, w=P, rope=P, starts=P, out=P, status=None)
    at.update(ptr or {})
    return _lib.load().mla_query_absorb(ctypes.byref(s), at["q"], at["w"], at["rope"],
                                        at["starts"], scale, at["out"], at["status"], None)


@pytest.mark.parametrize("fields,code", [
    (dict(R=0), SHAPE), (dict(k=0), SHAPE), (dict(H=0), SHAPE), (dict(H=(1 << 16) + 1), SHAPE),
    (dict(R=1 << 23, k=4), SHAPE), (dict(R=1 << 22, k=1, H=1 << 12), SHAPE),
    (dict(rope_rows=0), SHAPE), (dict(interleaved=-1), SHAPE), (dict(token_stride=184), SHAPE),
    (dict(head_stride=184), SHAPE), (dict(token_stride=1540), ALIGN), (dict(head_stride=196), ALIGN)])
def test_absorb_shapes_refused(fields, code):
    assert _absorb(**fields) == code


@pytest.mark.parametrize("name", ["q", "w", "rope", "starts", "out"])
def test_absorb_pointers_refused(name):
    assert _absorb(ptr={name: None}) == NULL
    if name != "starts":
        assert _absorb(ptr={name: ODD}) == ALIGN


@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), float("inf"), 1e-45])
def test_absorb_scales_refused(scale):
    assert _absorb(scale=scale) == SHAPE


def _shape(**fields):
    s = mla.make_shape(4, 2, 8, 10, 100, 152)
    for name, value in fields.items():
        setattr(s, name, value)
    return s


def _prefix(shape=None, *, ptr=None, pages=3, bmm1=1.0, bmm2=1.0, plan_len=5, ws=1 << 40):
    s = shape or _shape()
    at = dict(q=P, kv=P, ptable=P, plen=P, table=P, lens=P, plan=P, ws=P, out=P, lse=None, status=None)
    at.update(ptr or {})
    return _lib.load().mla_prefix_decode(
        ctypes.byref(s), pages, at["q"], at["kv"], at["ptable"], at["plen"], at["table"], at["lens"],
        bmm1, bmm2, at["plan"], plan_len, at["ws"], ws, at["out"], at["lse"], at["status"], None)


@pytest.mark.parametrize("fields,code", [
    (dict(page_size=32), UNSUPPORTED), (dict(R=0), SHAPE), (dict(R=1025), SHAPE), (dict(H=5000), SHAPE),
    (dict(groups=2), SHAPE), (dict(max_pages=0), SHAPE), (dict(num_pages=1 << 25), SHAPE),
    (dict(num_ctas=0), SHAPE), (dict(R=1024, H=2048, max_pages=1 << 24), SHAPE)])
def test_prefix_shapes_refused(fields, code):
    assert _prefix(_shape(**fields)) == code
    lib, s = _lib.load(), _shape(**fields)
    size = ctypes.c_size_t(0)
    assert lib.mla_prefix_workspace_bytes(ctypes.byref(s), ctypes.byref(size)) == code
    assert lib.mla_prefix_plan(ctypes.byref(s), P, P, 2000, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(pages=0), SHAPE), (dict(pages=(1 << 24) + 1), SHAPE), (dict(bmm1=0.0), SHAPE),
    (dict(bmm1=float("nan")), SHAPE), (dict(bmm2=float("inf")), SHAPE), (dict(plan_len=4), -4),
    (dict(ws=1000), -3)])
def test_prefix_arguments_refused(kw, code):
    assert _prefix(**kw) == code


@pytest.mark.parametrize("name", ["q", "kv", "ptable", "plen", "table", "lens", "plan", "ws", "out"])
def test_prefix_pointers_refused(name):
    assert _prefix(ptr={name: None}) == NULL
    assert _prefix(ptr={name: ctypes.c_void_p((1 << 20) + 2)}) == ALIGN


def test_prefix_plan_arguments_refused():
    lib, s = _lib.load(), _shape()
    assert lib.mla_prefix_plan(ctypes.byref(s), None, P, 5, None) == NULL
    assert lib.mla_prefix_plan(ctypes.byref(s), P, None, 5, None) == NULL
    assert lib.mla_prefix_plan(ctypes.byref(s), P, P, 4, None) == -4
    assert lib.mla_prefix_plan(ctypes.byref(s), P, ctypes.c_void_p((1 << 20) + 2), 5, None) == ALIGN
    assert lib.mla_prefix_workspace_bytes(ctypes.byref(s), None) == NULL


@pytest.mark.parametrize("R,k,H,ctas", [(1, 1, 1, 1), (4, 2, 8, 152), (64, 7, 8, 152), (128, 7, 64, 152)])
def test_prefix_workspace(R, k, H, ctas):
    """One slot of 128 rows for every pair and segment but one: FP32 rows, then LSEs."""
    N, M = R * k * H, k * H
    slots = max(1, ctas // 2) + -(-N // 128) + R * -(-M // 128) - 1
    align = lambda x: (x + 255) // 256 * 256  # noqa: E731
    want = align(slots * 128 * 512 * 4) + align(slots * 128 * 4)
    assert mla.prefix_workspace_bytes(mla.make_shape(R, k, H, 10, 100, ctas)) == want


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 576, dtype=torch.bfloat16)
    kv = torch.zeros(1, 64, 576, dtype=torch.uint8)
    i32 = torch.zeros(1, dtype=torch.int32)
    rope = mla.rope_table(4, device="cpu")
    with pytest.raises(ValueError, match="kv is not a CUDA tensor"):
        mla.kv_append(x, kv, i32[None], i32, rope, 1.0)
    with pytest.raises(ValueError, match="q is not a CUDA tensor"):
        mla.query_absorb(torch.zeros(2, 1, 192, dtype=torch.bfloat16), x, rope, i32, 1.0)


@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_rope_table(base):
    t = mla.rope_table(131072, base, device="cpu")
    assert t.shape == (131072, 64) and t.dtype == torch.float32
    import math
    for p in (0, 1, 777, 131071):
        for i in (0, 7, 31):
            a = p * base ** (-i / 32)
            # 64-bit angles: their error is below 2^-53 * 2^17 * a few steps, FP32 rounding 2^-25.
            assert abs(float(t[p, i]) - math.cos(a)) < 2.0 ** -24
            assert abs(float(t[p, 32 + i]) - math.sin(a)) < 2.0 ** -24


def test_the_decode_profiles_are_of_this_source():
    """The operators around the decode leave its sources, and so its measured DRAM
    bytes, as they were."""
    import bench
    for name in ("R128_k7_H64_skewed128k", "R32_k4_H8_len1k-8k", "R64_k7_H8_lognormal2k",
                 "R16_k4_H64_len16k-64k"):
        assert bench.profiled_traffic(name) is not None


@pytest.mark.parametrize("withhold,limit,status,code", [
    (0, 999_999, P, SHAPE), (1, 0, P, SHAPE), (1, 2_000_000_001, P, SHAPE), (2, 2_000_000, P, SHAPE),
    (-1, 2_000_000, P, SHAPE), (1, 2_000_000, None, NULL)])
def test_absorb_wait_test_refuses(withhold, limit, status, code):
    """Other pointers are NULL: a working check answers first, and nothing launches."""
    s = _lib.QueryShape(2, 4, 8, 100, 1, 8 * 192, 192)
    assert _lib.load().mla_query_absorb_wait_test(ctypes.byref(s), None, None, None, None, 0.1, None,
                                                  status, withhold, limit, None) == code


@pytest.mark.parametrize("limit,status,code", [(999_999, P, SHAPE), (0, P, SHAPE),
                                               (2_000_000_001, P, SHAPE), (2_000_000, None, NULL)])
def test_prefix_wait_test_refuses(limit, status, code):
    s = _shape()
    assert _lib.load().mla_prefix_decode_wait_test(
        ctypes.byref(s), 3, None, None, None, None, None, None, 1.0, 1.0, None, 5, None, 0, None, None,
        status, limit, None) == code
