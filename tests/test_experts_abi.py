"""Refusals of the expert layer's calls that need no GPU: nothing is enqueued (the
pointers below are never dereferenced)."""

import ctypes

import pytest
import torch

from moe_grouped_gemm_amd import moe

P = [0x10000 * i for i in range(1, 10)]
NAMES = ("x", "topk_ids", "weights", "b1", "sfb1", "b2", "sfb2", "y", "workspace")
NULL, SHAPE, ALIGN, UNSUPPORTED, DEVICE = 1, 2, 3, 4, 6
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")


def _call(weight_type=0, tokens=4, top_k=2, num_groups=8, hidden=256, inner=128, workspace_bytes=1 << 30, **change):
    p = [0 if change.get(n, v) is None else change.get(n, v) for n, v in zip(NAMES, P)]
    args = moe._EXPERTS.pack(*p, workspace_bytes, weight_type, tokens, top_k, num_groups, hidden, inner)
    return moe.lib().dg_moe_experts(args, None)


def test_argument_struct_has_the_headers_size():
    assert moe._EXPERTS.size == 9 * ctypes.sizeof(ctypes.c_void_p) + 8 + 6 * 4
    assert moe.lib().dg_moe_experts(None, None) == NULL


def test_refusals():
    for n in NAMES:
        if n != "weights":
            assert _call(**{n: None}) == NULL, n
        assert _call(**{n: P[0] + 2}) == ALIGN, n
    for bad in ({"tokens": -1}, {"top_k": 0}, {"num_groups": 0}, {"hidden": 0}, {"hidden": 192}, {"inner": 0},
                {"inner": 64}, {"weight_type": 2}, {"weight_type": -1}):
        assert _call(**bad) == SHAPE, bad
    for big in ({"tokens": 129}, {"top_k": 33}, {"tokens": 128, "top_k": 9}, {"num_groups": 4097}, {"hidden": 1 << 17},
                {"inner": 1 << 17}, {"num_groups": 4096, "hidden": 1 << 16, "inner": 1 << 15}):
        assert _call(**big) == UNSUPPORTED, big
    need = moe.lib().dg_moe_experts_workspace_bytes(4, 2, 8, 128)
    assert need > 0 and _call(workspace_bytes=need - 1) == SHAPE
    assert _call(tokens=0, **dict.fromkeys(NAMES)) == 0
    for bad in ((-1, 2, 8, 128), (4, 0, 8, 128), (4, 2, 0, 128), (4, 2, 8, 100), (129, 2, 8, 128), (128, 9, 8, 128)):
        assert moe.lib().dg_moe_experts_workspace_bytes(*bad) == -1


@no_gpu
def test_valid_calls_need_a_device():
    assert _call() == DEVICE and _call(weight_type=1, weights=None) == DEVICE


def test_binding_refuses():
    with pytest.raises(ValueError):
        moe.experts_workspace(129, 1, 8, 128, "cpu")
    with pytest.raises(ValueError):
        moe.experts_workspace(2 ** 32 + 1, 1, 8, 128, "cpu")
    host = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                  # there is no fallback
        moe.experts(host, None, None, None, None, None, None, host, None)
