"""The GEMMs' Python binding calls the library with its tensors' device
current; no GPU is needed: the devices and the library are pretended."""

import inspect

import pytest
import torch

from moe_grouped_gemm_amd import dg


class _OnDevice1(torch.Tensor):
    """A host tensor that says it lives on the second GPU."""

    def get_device(self):
        return 1


def _there(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnDevice1)


def _calls():
    f8, f32, bf, i32, u8 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32, torch.uint8
    a, sfa, b, sfb, d = (_there(128, 128, dtype=f8), _there(1, 128, dtype=f32), _there(128, 128, dtype=f8),
                         _there(1, 1, dtype=f32), _there(128, 128, dtype=bf))
    ga, gsfa, gb, gsfb, gd = (t[None] for t in (a, sfa, b, sfb, d))
    fb, fsfb = _there(1, 128, 64, dtype=u8), _there(1, 4, 128, dtype=f32)
    rows, one = _there(128, dtype=i32), _there(1, dtype=i32)
    return {
        "fp8_gemm_nt": (a, sfa, b, sfb, d),
        "m_grouped_fp8_gemm_nt_contiguous": (a, sfa, gb, gsfb, d, rows),
        "m_grouped_fp8_gemm_nt_masked": (ga, gsfa, gb, gsfb, gd, one),
        "m_grouped_fp8_gemm_nt_nopad": (a, sfa, gb, gsfb, d, one),
        "m_grouped_fp8_fp4_gemm_nt_contiguous": (a, sfa, fb, fsfb, d, rows),
        "m_grouped_fp8_fp4_gemm_nt_masked": (ga, gsfa, fb, fsfb, gd, one),
        "k_grouped_fp8_gemm_nt_contiguous": (a, sfa, b, _there(1, 128, dtype=f32), _there(1, 128, 128, dtype=f32), [128]),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_gemms_run_on_their_tensors_device(monkeypatch, name):
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

    class Library:
        def __getattr__(self, entry):
            if entry == "dg_get_tma_aligned_size":
                return lambda x, size: (x + 3) // 4 * 4

            def call(*args):
                seen.append((entry, current[0], args[-1]))
                return 0
            return call

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(dg, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(dg, "_stream", lambda t: 1000 * t.get_device())
    monkeypatch.setattr(dg, "_need", lambda *args: None)
    monkeypatch.setattr(dg, "lib", lambda: Library())
    call, args = getattr(dg, name), _calls()[name]
    call(*args)
    call(**dict(zip(inspect.signature(call).parameters, args)))
    current[0] = 1
    call(*args)
    assert seen == [("dg_" + name, 1, 1000)] * 3 and current[0] == 1
