"""The Python binding of the FP4 calls and of the expert layer calls the library with its
tensors' device current; no GPU is needed: the devices and the library are pretended."""

import pytest
import torch

from moe_grouped_gemm_amd import dg, moe


class _OnDevice1(torch.Tensor):
    """A host tensor that says it lives on the second GPU."""

    def get_device(self):
        return 1


def _there(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnDevice1)


def _calls():
    u8, i32, bf, f32, f8 = torch.uint8, torch.int32, torch.bfloat16, torch.float32, torch.float8_e4m3fn
    a, sfa, d, x = _there(128, 64, dtype=u8), _there(1, 128, dtype=i32), _there(128, 128, dtype=bf), _there(128, 128, dtype=f32)
    b1, sfb1 = _there(1, 256, 64, dtype=u8), _there(1, 1, 256, dtype=i32)
    rows, one = _there(128, dtype=i32), _there(1, dtype=i32)
    plan = moe.Plan.__new__(moe.Plan)
    plan.layout, plan.max_tokens, plan.top_k, plan.num_groups, plan.rows, plan.hidden = "nopad", 4, 2, 3, 128, 128
    plan.device, plan._index, plan._ref = torch.device("cuda", 1), 1, 0
    plan.rows_shape, plan.scale_shape, plan.codes_shape = (torch.Size(v) for v in ((128, 128), (1, 128), (128, 64)))
    t, ids, ws = _there(4, 128, dtype=bf), _there(4, 2, dtype=i32), _there(64, dtype=u8)
    e1, s1, e2, s2 = _there(1, 256, 128, dtype=f8), _there(1, 2, 1, dtype=f32), _there(1, 128, 128, dtype=f8), _there(1, 1, 1, dtype=f32)
    return {
        "dg_fp4_gemm_nt": lambda: dg.fp4_gemm_nt(a, sfa, a, sfa, d),
        "dg_m_grouped_fp4_gemm_nt_contiguous": lambda: dg.m_grouped_fp4_gemm_nt_contiguous(a, sfa, a[None], sfa[None], d, rows),
        "dg_m_grouped_fp4_gemm_nt_masked": lambda: dg.m_grouped_fp4_gemm_nt_masked(a[None], sfa[None], a[None], sfa[None], d[None], one),
        "dg_m_grouped_fp4_gemm_nt_nopad": lambda: dg.m_grouped_fp4_gemm_nt_nopad(a, sfa, a[None], sfa[None], d, one),
        "dg_quantize_fp4": lambda: dg.quantize_fp4(x, a, sfa),
        "dg_dequantize_fp4": lambda: dg.dequantize_fp4(a, sfa, d),
        "dg_moe_dispatch_fp4": lambda: moe.dispatch_fp4(plan, t, a, sfa, topk_ids=ids),
        "dg_moe_swiglu_fp4": lambda: moe.swiglu_fp4(_there(128, 256, dtype=bf), a, sfa),
        "dg_moe_experts": lambda: moe.experts(t, ids, None, e1, s1, e2, s2, t, ws),
        "dg_moe_experts in FP4": lambda: moe.experts(t, ids, None, b1, sfb1, a[None], sfa[None], t, ws),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_calls_run_on_their_tensors_device(monkeypatch, name):
    """A default stream's handle is 0 on every device and means the default stream
    of whichever is current, so the tensors' device has to be."""
    current, seen = [0], []

    class Guard:
        def __init__(self, device):
            self.index = device if isinstance(device, int) else device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    class Stream:
        def __init__(self, index):
            self.cuda_stream = 1000 * index

    class Library:
        def __getattr__(self, entry):
            def call(*args):
                seen.append((entry, current[0], args[-1]))
                return 0
            return call

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    for module in (dg, moe):
        monkeypatch.setattr(module, "_current_device", lambda: current[0])
        monkeypatch.setattr(module, "_raw_stream", lambda index: 1000 * index)
        monkeypatch.setattr(module, "lib", lambda: Library())
    _calls()[name]()
    current[0] = 1
    _calls()[name]()
    assert seen == [(name.split()[0], 1, 1000)] * 2 and current[0] == 1


def _vast(*shape, dtype):
    """A tensor on the second GPU with sizes and without memory."""
    return torch.empty(*shape, dtype=dtype, device="meta").as_subclass(_OnDevice1)


def _vast_calls():
    u8, i32, bf, f32, f8 = torch.uint8, torch.int32, torch.bfloat16, torch.float32, torch.float8_e4m3fn
    k = 2 ** 32 + 128                                # 128, taken modulo 2^32
    x, q, sf = _vast(1, k, dtype=bf), _vast(1, k // 2, dtype=u8), _vast(k // 128, 4, dtype=i32)
    b, sfb, d = _vast(128, k // 2, dtype=u8), _vast(k // 128, 128, dtype=i32), _vast(1, 128, dtype=bf)
    n = _vast(k, 64, dtype=u8), _vast(1, k, dtype=i32)
    one, a, sfa = _vast(1, dtype=i32), _vast(1, 64, dtype=u8), _vast(1, 4, dtype=i32)
    a8, sfa8, b8, sfb8 = _vast(1, k, dtype=f8), _vast(k // 128, 4, dtype=f32), _vast(128, k, dtype=f8), _vast(1, k // 128, dtype=f32)
    t, ids, w = _vast(1, 128, dtype=bf), _vast(1, 2 ** 32 + 2, dtype=i32), _vast(64, dtype=u8)
    e1, s1, e2, s2 = _vast(1, 256, 128, dtype=f8), _vast(1, 2, 1, dtype=f32), _vast(1, 128, 128, dtype=f8), _vast(1, 1, 1, dtype=f32)
    return {
        "quantize_fp4": lambda: dg.quantize_fp4(x, q, sf),
        "quantize_fp4 of groups": lambda: dg.quantize_fp4(_vast(k, 1, 128, dtype=bf), _vast(k, 1, 64, dtype=u8), _vast(k, 1, 4, dtype=i32)),
        "dequantize_fp4": lambda: dg.dequantize_fp4(q, sf, x),
        "fp4_gemm_nt, k": lambda: dg.fp4_gemm_nt(q, sf, b, sfb, d),
        "fp4_gemm_nt, n": lambda: dg.fp4_gemm_nt(a, sfa, *n, _vast(1, k, dtype=bf)),
        "fp4_gemm_nt_nopad": lambda: dg.m_grouped_fp4_gemm_nt_nopad(q, sf, b[None], sfb[None], d, one),
        "fp8_gemm_nt": lambda: dg.fp8_gemm_nt(a8, sfa8, b8, sfb8, d),
        "fp8_gemm_nt_nopad": lambda: dg.m_grouped_fp8_gemm_nt_nopad(a8, sfa8, b8[None], sfb8[None], d, one),
        "swiglu_fp4": lambda: moe.swiglu_fp4(_vast(1, 2 * k, dtype=bf), q, sf),
        "swiglu_fp8": lambda: moe.swiglu_fp8(_vast(1, 2 * k, dtype=bf), a8, sfa8),
        "experts": lambda: moe.experts(t, ids, None, e1, s1, e2, s2, t, w),
    }


@pytest.mark.parametrize("name", sorted(_vast_calls()))
def test_sizes_past_32_bits_are_refused(monkeypatch, name):
    """The library's sizes are ints, which ctypes takes modulo 2^32: such a call would work on
    a corner of its tensors and succeed."""
    for module in (dg, moe):
        monkeypatch.setattr(module, "_current_device", lambda: 1)
        monkeypatch.setattr(module, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(dg, "_stream", lambda t: 0)
    monkeypatch.setattr(dg, "_need", lambda *args: None)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda self: 0x10000)
    with pytest.raises((ValueError, dg.DGError)) as refused:
        _vast_calls()[name]()
    if refused.type is dg.DGError:
        assert refused.value.status in (2, 4)        # shape, unsupported: before the device is asked
