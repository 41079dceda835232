"""C-ABI checks of the steps around the GEMMs that need no GPU: every declared
symbol is exported and bound, and invalid arguments are refused before
anything is enqueued (the pointers below are never dereferenced)."""

import ctypes
import os
import re

import pytest
import torch

from moe_grouped_gemm_amd import dg, moe

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe", "dg_moe.h")
A, B, C, D, E, F = (0x10000 * i for i in range(1, 7))
NULL, SHAPE, ALIGN, UNSUPPORTED, DEVICE = 1, 2, 3, 4, 6
# valid arguments reach the device check: refused for want of a device here, and not run where there is one
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dg_moe_[a-z0-9_]+)\s*\(", text)))
    assert sorted(n for n, _, _ in moe.SIGNATURES) == names
    for n in names:
        assert hasattr(moe.lib(), n)


def _plan(layout=2, max_tokens=64, top_k=4, num_groups=8, rows=128, hidden=256, row_of=A, group_rows=B, layout_ptr=C,
          ws=D, ws_bytes=1 << 30):
    return moe._PlanStruct(layout, max_tokens, top_k, num_groups, rows, hidden, row_of, group_rows, layout_ptr, ws,
                           ws_bytes)


def _calls(plan, tokens=16, x=A, y=B, w=C, ids=D, s=E):
    lib, p = moe.lib(), ctypes.byref(plan) if plan is not None else None
    return {
        "sort": lambda: lib.dg_moe_sort(p, ids, tokens, None),
        "dispatch": lambda: lib.dg_moe_dispatch(p, ids, x, y, tokens, None),
        "dispatch_fp8": lambda: lib.dg_moe_dispatch_fp8(p, ids, x, y, s, tokens, 0, None),
        "combine": lambda: lib.dg_moe_combine(p, x, w, y, tokens, None),
        "combine_bwd": lambda: lib.dg_moe_combine_bwd(p, x, s, w, y, F, tokens, None),
    }


BAD_PLANS = [
    ({"layout": 0}, SHAPE), ({"layout": 4}, SHAPE), ({"top_k": 0}, SHAPE), ({"top_k": 33}, UNSUPPORTED),
    ({"num_groups": 0}, SHAPE), ({"num_groups": 4097}, UNSUPPORTED), ({"layout": 3, "num_groups": 2049}, UNSUPPORTED),
    ({"rows": -1}, SHAPE), ({"rows": 0}, SHAPE), ({"layout": 1, "rows": 130}, SHAPE), ({"hidden": 192}, SHAPE),
    ({"hidden": 0}, SHAPE), ({"hidden": 1 << 21}, UNSUPPORTED), ({"max_tokens": -1}, SHAPE),
    ({"max_tokens": (1 << 20) + 1}, UNSUPPORTED), ({"num_groups": 4096, "rows": 1 << 19}, UNSUPPORTED),
    ({"layout": 3, "rows": 2 ** 31 - 1, "hidden": 512}, UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", BAD_PLANS)
def test_bad_plan_sizes(change, status):
    plan = _plan(**change)
    assert moe.lib().dg_moe_workspace_bytes(ctypes.addressof(plan)) == -1
    for name, call in _calls(plan).items():
        assert call() == status, name


@pytest.mark.parametrize("layout,rows", [(1, 2 ** 31 - 128), (3, 2 ** 31 - 1), (1, 2 ** 30), (3, 2 ** 30)])
def test_rows_past_the_kernels_indices(layout, rows):
    """Row numbers are int32 and the kernels step past the last one: 2^30 rows
    and more are refused, whatever the row length."""
    plan = _plan(layout=layout, rows=rows, hidden=128)
    assert moe.lib().dg_moe_workspace_bytes(ctypes.addressof(plan)) == -1
    for name, call in _calls(plan).items():
        assert call() == UNSUPPORTED, name
    assert moe.lib().dg_moe_workspace_bytes(ctypes.addressof(_plan(layout=layout, rows=2 ** 30 - 128, hidden=128))) > 0


def test_bad_plan_pointers():
    for name, call in _calls(None).items():
        assert call() == NULL, name
    assert moe.lib().dg_moe_workspace_bytes(None) == -1
    for change, status in (({"row_of": None}, NULL), ({"group_rows": None}, NULL), ({"ws": None}, NULL),
                           ({"layout": 1, "layout_ptr": None}, NULL), ({"row_of": A + 2}, ALIGN),
                           ({"group_rows": B + 1}, ALIGN), ({"ws": D + 8}, ALIGN), ({"ws_bytes": 0}, SHAPE)):
        for name, call in _calls(_plan(**change)).items():
            assert call() == status, (name, change)


def test_bad_call_arguments():
    plan = _plan()
    for tokens in (-1, 65):
        for name, call in _calls(plan, tokens=tokens).items():
            assert call() == SHAPE, name
    assert _calls(plan, ids=None)["sort"]() == NULL
    for name in ("dispatch", "dispatch_fp8", "combine", "combine_bwd"):
        assert _calls(plan, x=None)[name]() == NULL
        assert _calls(plan, y=None)[name]() == NULL
        assert _calls(plan, x=A + 8)[name]() == ALIGN
        assert _calls(plan, y=B + 2)[name]() == ALIGN
    assert _calls(plan, s=None)["dispatch_fp8"]() == NULL
    assert _calls(plan, s=None)["combine_bwd"]() == NULL       # dweights wanted, yp missing
    assert _calls(plan, w=None)["combine_bwd"]() == NULL
    assert _calls(plan, w=C + 1)["combine"]() == ALIGN
    for name in ("sort", "dispatch", "dispatch_fp8"):
        assert _calls(plan, ids=D + 2)[name]() == ALIGN
    for name in ("combine", "combine_bwd"):
        assert _calls(plan, tokens=0, x=None, y=None, w=None)[name]() == 0     # empty: a successful no-op
    for name in ("dispatch", "dispatch_fp8"):
        assert _calls(plan, tokens=0, ids=None, x=None, y=None)[name]() == 0


@no_gpu
def test_valid_calls_need_a_device():
    for layout in (1, 2, 3):
        for name, call in _calls(_plan(layout=layout)).items():
            assert call() == DEVICE, name
    assert _glu() == DEVICE and _glu_bwd() == DEVICE and _norm() == DEVICE and _norm_bwd() == DEVICE
    assert _norm_bwd(tokens=0) == DEVICE       # still clears the weight gradients


def _glu(gu=A, q=B, sfa=C, rows=D, layout=2, m=128, groups=8, inner=256):
    return moe.lib().dg_moe_swiglu_fp8(gu, q, sfa, rows, layout, m, groups, inner, 0, None)


def _glu_bwd(da=A, gu=B, dgu=C, rows=D, layout=2, m=128, groups=8, inner=256):
    return moe.lib().dg_moe_swiglu_bwd(da, gu, dgu, rows, layout, m, groups, inner, None)


@pytest.mark.parametrize("call", [_glu, _glu_bwd])
def test_glu_refusals(call):
    assert call(gu=None) == NULL and call(rows=None) == NULL
    assert call(gu=A + 8) == ALIGN and call(rows=D + 2) == ALIGN
    assert call(inner=0) == SHAPE and call(inner=200) == SHAPE and call(inner=1 << 21) == UNSUPPORTED
    assert call(m=-1) == SHAPE and call(m=0) == SHAPE and call(layout=1, m=100) == SHAPE and call(layout=7) == SHAPE
    assert call(groups=0) == SHAPE and call(groups=4097) == UNSUPPORTED and call(layout=3, groups=2049) == UNSUPPORTED
    assert call(layout=3, m=(1 << 22) + 1) == UNSUPPORTED and call(layout=0, rows=None, m=1 << 24) == UNSUPPORTED
    assert call(layout=0, m=-1) == SHAPE
    for layout in (0, 1, 3):
        assert call(layout=layout, m=0, rows=None if layout != 3 else D) == 0


def _norm(x=A, y=B, post=C, gate=D, kind=1, pre=E, h=F, n=A, r1=B, r2=C, rs=0.5, eps=1e-6, tokens=4, hidden=64):
    p = (0 if v is None else v for v in (x, y, post, gate, pre, h, n, r1, r2))
    return moe.lib().dg_moe_block_norm(moe._NORM.pack(*p, rs, eps, kind, tokens, hidden), None)


def _norm_bwd(dh=A, dn=B, h=C, y=D, post=E, gate=F, kind=1, pre=A, r1=B, r2=C, dx=D, dy=E, dpost=F, dgate=A, dpre=B,
              ws=C, ws_bytes=1 << 30, rs=0.5, tokens=4, hidden=64):
    p = (0 if v is None else v for v in (dh, dn, h, y, post, gate, pre, r1, r2, dx, dy, dpost, dgate, dpre, ws))
    return moe.lib().dg_moe_block_norm_bwd(moe._NORM_BWD.pack(*p, ws_bytes, rs, kind, tokens, hidden), None)


def test_argument_structs_have_the_headers_size():
    p, f, i = ctypes.sizeof(ctypes.c_void_p), 4, 4
    assert moe._NORM.size == 9 * p + 2 * f + 3 * i + 4           # padded to a multiple of a pointer
    assert moe._NORM_BWD.size == 15 * p + 8 + f + 3 * i
    assert moe.lib().dg_moe_block_norm(None, None) == NULL and moe.lib().dg_moe_block_norm_bwd(None, None) == NULL


def test_block_norm_refusals():
    assert _norm(x=None) == NULL and _norm(h=None) == NULL and _norm(pre=None) == NULL
    assert _norm(y=None) == NULL                               # h, gate, ... given without y
    assert _norm(n=None) == NULL and _norm(n=None, pre=None) == NULL
    assert _norm(post=None) == NULL                            # rstd_post without post_weight
    assert _norm(gate=None) == NULL and _norm(kind=0) == NULL
    assert _norm(kind=4) == SHAPE and _norm(kind=-1) == SHAPE
    assert _norm(hidden=0) == SHAPE and _norm(hidden=12) == SHAPE and _norm(hidden=16392) == UNSUPPORTED
    assert _norm(tokens=-1) == SHAPE and _norm(tokens=(1 << 21) + 1) == UNSUPPORTED
    assert _norm(eps=-1.0) == SHAPE and _norm(eps=float("nan")) == SHAPE
    assert _norm(x=A + 2) == ALIGN and _norm(gate=D + 4) == ALIGN and _norm(kind=2, gate=D + 2) == ALIGN
    assert _norm(r1=B + 2) == ALIGN
    assert _norm(tokens=0) == 0
    none = {"y": None, "post": None, "gate": None, "kind": 0, "h": None, "r1": None}
    assert _norm(**none) == NULL                               # residual_scale without a block output
    assert _norm(**none, rs=1.0, n=None, pre=None, r2=None) == NULL


def test_block_norm_bwd_refusals():
    assert _norm_bwd(dh=None, dn=None, pre=None, r2=None, dpre=None) == NULL
    for name in ("h", "pre", "r2", "dx", "dy", "r1", "ws", "gate"):
        assert _norm_bwd(**{name: None}) == NULL, name
    assert _norm_bwd(dn=None) == NULL and _norm_bwd(y=None) == NULL and _norm_bwd(post=None) == NULL
    assert _norm_bwd(kind=0) == NULL and _norm_bwd(kind=5) == SHAPE
    assert _norm_bwd(kind=0, gate=None) == NULL                # dgate without a gate
    assert _norm_bwd(hidden=20) == SHAPE and _norm_bwd(hidden=16392) == UNSUPPORTED and _norm_bwd(tokens=-2) == SHAPE
    assert _norm_bwd(dx=D + 8) == ALIGN and _norm_bwd(ws=C + 4) == ALIGN and _norm_bwd(dpre=B + 1) == ALIGN
    need = moe.lib().dg_moe_block_norm_workspace_bytes(4, 64)
    assert need > 0 and _norm_bwd(ws_bytes=need - 1) == SHAPE
    assert moe.lib().dg_moe_block_norm_workspace_bytes(-1, 64) == -1
    assert moe.lib().dg_moe_block_norm_workspace_bytes(4, 12) == -1


def test_plan_refuses_bad_sizes_and_layouts():
    with pytest.raises(ValueError):
        moe.Plan(8, 2, 4, "dense", 16, 256, "cpu")
    with pytest.raises(ValueError):
        moe.Plan(8, 2, 4, "contiguous", 100, 256, "cpu")
    with pytest.raises(ValueError):
        moe.Plan(8, 2, 4, "nopad", 16, 200, "cpu")
    with pytest.raises(ValueError):
        moe.block_norm_workspace(4, 12, "cpu")
    with pytest.raises(ValueError):        # there is no fallback
        moe.Plan(8, 2, 4, "nopad", 16, 256, "cpu")


def test_contiguous_rows_hold_any_split():
    assert moe.contiguous_rows(0, 8) == 0
    assert moe.contiguous_rows(1, 8) == 128
    assert moe.contiguous_rows(3, 2) == 384      # 3 + 2 * 127, rounded up; two segments of 128 at most are used
    assert dg.get_mk_alignment_for_contiguous_layout() == 128
