"""Refusals of the FP4 calls that need no GPU: nothing is enqueued (the pointers
below are never dereferenced)."""

import ctypes
import os
import re

import pytest
import torch

from moe_grouped_gemm_amd import dg, moe

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fp4", "dg_fp4.h")
A, B, C, D, E, F = (0x10000 * i for i in range(1, 7))
NULL, SHAPE, ALIGN, UNSUPPORTED, DEVICE = 1, 2, 3, 4, 6
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dg_[a-z0-9_]+)\s*\(", text)))
    assert sorted(n for n, _, _ in dg.FP4_SIGNATURES) == names
    for n in names:
        assert hasattr(dg.lib(), n)


def _dense(a=A, sfa=B, b=C, sfb=D, d=E, m=64, n=256, k=512):
    return dg.lib().dg_fp4_gemm_nt(a, sfa, b, sfb, d, m, n, k, None)


def _grouped(name):
    def call(a=A, sfa=B, b=C, sfb=D, d=E, rows=F, m=128, n=256, k=512, g=4):
        sizes = (g, m, n, k) if name == "masked" else (m, n, k, g)
        return getattr(dg.lib(), f"dg_m_grouped_fp4_gemm_nt_{name}")(a, sfa, b, sfb, d, rows, *sizes, None)
    return call


CALLS = {"dense": _dense, **{name: _grouped(name) for name in ("contiguous", "masked", "nopad")}}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_products_refuse(name):
    call = CALLS[name]
    for p in ("a", "sfa", "b", "sfb", "d"):
        assert call(**{p: None}) == NULL and call(**{p: A + 8}) == ALIGN
    for bad in ({"n": 0}, {"n": 200}, {"k": 0}, {"k": 192}, {"m": -1}, {"k": -128}):
        assert call(**bad) == SHAPE
    assert call(n=1 << 21) == UNSUPPORTED and call(k=1 << 21) == UNSUPPORTED
    assert call(m=1 << 30) == UNSUPPORTED
    if name != "dense":
        assert call(rows=None) == NULL and call(g=-1) == SHAPE and call(g=0) == 0
        assert call(m=1 << 20, n=1 << 20, k=128, g=4) == UNSUPPORTED        # more tiles than an int counts
    if name == "masked":
        assert call(m=0) == SHAPE and call(g=4097) == UNSUPPORTED and call(g=4096, m=1 << 18) == UNSUPPORTED
    else:
        assert call(m=0) == 0
    if name == "contiguous":
        assert call(m=100) == SHAPE
    if name == "nopad":
        assert call(g=2049) == UNSUPPORTED


@no_gpu
def test_valid_calls_need_a_device():
    for name, call in CALLS.items():
        assert call() == DEVICE, name
    assert _quantize() == DEVICE and _back() == DEVICE


@no_gpu
@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_largest_products_are_taken(name):
    """The limits as documented: rows below 2^30, groups as far as the layout's rows go."""
    g = {"dense": {}, "contiguous": {"g": 1 << 26}, "masked": {"g": 4096}, "nopad": {"g": 2048}}[name]
    m = {"masked": (1 << 18) - 1, "contiguous": (1 << 30) - 128}.get(name, (1 << 30) - 1)
    assert CALLS[name](m=m, n=128, k=128, **g) == DEVICE
    few = {k: min(v, 2048) for k, v in g.items()}     # b is 2^37 bytes, and d (masked) 2^39
    assert CALLS[name](m=128, n=1 << 20, k=128, **few) == DEVICE
    assert CALLS[name](m=128, n=128, k=1 << 20, **few) == DEVICE


def _quantize(x=A, kind=0, q=B, sf=C, groups=2, rows=5, k=256):
    return dg.lib().dg_quantize_fp4(x, kind, q, sf, groups, rows, k, None)


def _back(x=A, q=B, sf=C, groups=2, rows=5, k=256):
    return dg.lib().dg_dequantize_fp4(q, sf, x, groups, rows, k, None)


@pytest.mark.parametrize("call", [_quantize, _back])
def test_quantizer_refuses(call):
    for p in ("x", "q", "sf"):
        assert call(**{p: None}) == NULL and call(**{p: A + 4}) == ALIGN
    for bad in ({"rows": -1}, {"groups": -1}, {"k": 0}, {"k": 96}):
        assert call(**bad) == SHAPE
    assert call(k=1 << 21) == UNSUPPORTED and call(rows=1 << 30) == UNSUPPORTED
    assert call(groups=1 << 15, rows=1 << 15) == UNSUPPORTED and call(groups=1 << 10, rows=1 << 15, k=1 << 20) == UNSUPPORTED
    assert call(rows=0, x=None, q=None, sf=None) == 0 and call(groups=0, x=None, q=None, sf=None) == 0
    assert _quantize(kind=2) == SHAPE


def _dispatch(ids=D, x=A, q=B, sf=C, tokens=16, **change):
    sizes = {"layout": 2, "max_tokens": 64, "top_k": 4, "num_groups": 8, "rows": 128, "hidden": 256, "row_of": E,
             "group_rows": F, "grouped_layout": A, "workspace": B, "workspace_bytes": 1 << 30, **change}
    plan = moe._PlanStruct(*sizes.values())
    return moe.lib().dg_moe_dispatch_fp4(ctypes.byref(plan), ids, x, q, sf, tokens, None)


def test_dispatch_refuses():
    assert _dispatch(hidden=192) == SHAPE and _dispatch(layout=0) == SHAPE and _dispatch(workspace_bytes=0) == SHAPE
    assert _dispatch(tokens=-1) == SHAPE and _dispatch(tokens=65) == SHAPE
    assert _dispatch(rows=1 << 30, layout=3) == UNSUPPORTED and _dispatch(row_of=None) == NULL
    for p in ("x", "q", "sf"):
        assert _dispatch(**{p: None}) == NULL and _dispatch(**{p: A + 8}) == ALIGN
    assert _dispatch(ids=D + 2) == ALIGN
    assert _dispatch(tokens=0, ids=None, x=None, q=None, sf=None) == 0


def _glu(gu=A, q=B, sf=C, rows=D, layout=2, m=128, groups=8, inner=256):
    return moe.lib().dg_moe_swiglu_fp4(gu, q, sf, rows, layout, m, groups, inner, None)


def test_glu_refuses():
    for p in ("gu", "q", "sf"):
        assert _glu(**{p: None}) == NULL and _glu(**{p: A + 8}) == ALIGN
    assert _glu(rows=None) == NULL and _glu(rows=D + 2) == ALIGN
    assert _glu(inner=0) == SHAPE and _glu(inner=200) == SHAPE and _glu(inner=1 << 21) == UNSUPPORTED
    assert _glu(m=-1) == SHAPE and _glu(layout=7) == SHAPE and _glu(groups=0) == SHAPE and _glu(layout=1, m=100) == SHAPE
    assert _glu(groups=4097) == UNSUPPORTED and _glu(layout=0, rows=None, m=1 << 24) == UNSUPPORTED
    assert _glu(layout=0, m=0, rows=None, gu=None, q=None, sf=None) == 0


@no_gpu
def test_valid_steps_need_a_device():
    assert _dispatch() == DEVICE and _glu() == DEVICE


def test_binding_refuses():
    """The checks that come before the library: types, shapes, host tensors."""
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    q, sf, x = torch.zeros(4, 128, dtype=u8), torch.zeros(2, 4, dtype=i32), torch.zeros(4, 256, dtype=bf)
    with pytest.raises(ValueError):
        dg.quantize_fp4(x, q, sf)                        # host tensors
    with pytest.raises(TypeError):
        dg.quantize_fp4(x.half(), q, sf)
    with pytest.raises(TypeError):
        dg.quantize_fp4(x, None, sf)
    with pytest.raises(ValueError):
        dg.quantize_fp4(torch.zeros(256, dtype=bf), q, sf)
    with pytest.raises(ValueError):
        dg.dequantize_fp4(q, sf, x)
    with pytest.raises(ValueError):
        dg.fp4_gemm_nt(q, sf, q, sf, torch.zeros(4, 4, dtype=bf))
