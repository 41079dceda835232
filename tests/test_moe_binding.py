"""Checks of the Python binding of the steps around the GEMMs that need no
GPU: what a call does before and around the library's entry point."""

import pytest
import torch

from moe_grouped_gemm_amd import moe


class _OnDevice1(torch.Tensor):
    """A host tensor that says it lives on the second GPU."""

    def get_device(self):
        return 1


def _there(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnDevice1)


class _Machine:
    """Two devices of which the first is current, and a library whose entry
    points note where and on which stream they were called."""

    def __init__(self, monkeypatch):
        self.current, self.calls = 0, []
        outer = self

        class Guard:
            def __init__(self, index):
                self.index = index

            def __enter__(self):
                self.before, outer.current = outer.current, self.index

            def __exit__(self, *exc):
                outer.current = self.before

        class Library:
            def __getattr__(self, name):
                def entry(*args):
                    outer.calls.append((name, outer.current, args[-1]))
                    return 0
                return entry

        monkeypatch.setattr(torch.cuda, "device", Guard)
        monkeypatch.setattr(moe, "_current_device", lambda: outer.current, raising=False)
        monkeypatch.setattr(moe, "_raw_stream", lambda index: 1000 * index)
        monkeypatch.setattr(moe, "lib", lambda: Library())


def _plan():
    plan = moe.Plan.__new__(moe.Plan)
    plan.layout, plan.max_tokens, plan.top_k, plan.num_groups, plan.rows, plan.hidden = "nopad", 4, 2, 3, 8, 128
    plan.device, plan._index, plan._ref = torch.device("cuda", 1), 1, 0
    plan.rows_shape, plan.scale_shape = torch.Size((8, 128)), torch.Size((1, 8))
    plan.row_of = _there(4, 2, dtype=torch.int32)
    plan.workspace = _there(64, dtype=torch.uint8)
    return plan


def _calls():
    bf16, f32, i32, fp8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
    plan = _plan()
    x, rows = _there(4, 128, dtype=bf16), _there(8, 128, dtype=bf16)
    ids, w = _there(4, 2, dtype=i32), _there(4, 2, dtype=f32)
    q, sfa = _there(8, 128, dtype=fp8), _there(1, 8, dtype=f32)
    gu, col = _there(8, 256, dtype=bf16), _there(128, dtype=f32)
    r = _there(4, dtype=f32)
    ws = _there(64, dtype=torch.uint8)
    return {
        "dg_moe_sort": lambda: moe.sort(plan, ids),
        "dg_moe_dispatch": lambda: moe.dispatch(plan, x, rows, topk_ids=ids),
        "dg_moe_dispatch_fp8": lambda: moe.dispatch_fp8(plan, x, q, sfa, topk_ids=ids),
        "dg_moe_combine": lambda: moe.combine(plan, rows, x, weights=w),
        "dg_moe_combine_bwd": lambda: moe.combine_bwd(plan, x, rows, w, rows, w),
        "dg_moe_swiglu_fp8": lambda: moe.swiglu_fp8(gu, q, sfa),
        "dg_moe_swiglu_bwd": lambda: moe.swiglu_bwd(rows, gu, gu),
        "dg_moe_block_norm": lambda: moe.block_norm(x, x, col, None, col, x, x),
        "dg_moe_block_norm_bwd": lambda: moe.block_norm_bwd(x, x, x, x, col, None, col, r, r, x, x, col, None, col, ws),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_calls_run_on_their_tensors_device(monkeypatch, name):
    """The entry point is called with the tensors' device current, on that
    device's stream: a default stream's handle is 0 on every device, and
    means the default stream of whichever is current."""
    machine = _Machine(monkeypatch)
    _calls()[name]()
    assert machine.calls == [(name, 1, 1000)]
    assert machine.current == 0
    # and where it is current already, without changing it
    machine.current = 1
    _calls()[name]()
    assert machine.calls[1:] == [(name, 1, 1000)] and machine.current == 1


@pytest.mark.parametrize("field", ["max_tokens", "top_k", "num_groups", "rows", "hidden"])
@pytest.mark.parametrize("past", [2 ** 32, -2 ** 32, 2 ** 31])
def test_plan_sizes_past_32_bits(field, past):
    """Sizes that the library's int32 fields would take modulo 2^32 are refused."""
    sizes = {"max_tokens": 4, "top_k": 2, "num_groups": 3, "rows": 8, "hidden": 128}
    sizes[field] += past
    with pytest.raises(ValueError, match="out of range"):
        moe.Plan(sizes["max_tokens"], sizes["top_k"], sizes["num_groups"], "nopad", sizes["rows"], sizes["hidden"],
                 "cpu")


@pytest.mark.parametrize("tokens,hidden", [(2 ** 32 + 4, 256), (4, 2 ** 32 + 256), (-2 ** 32 + 4, 256)])
def test_norm_workspace_sizes_past_32_bits(tokens, hidden):
    with pytest.raises(ValueError, match="out of range"):
        moe.block_norm_workspace(tokens, hidden, "cpu")
