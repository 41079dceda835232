"""Python binding of the steps around the grouped GEMMs (include/moe/dg_moe.h):
tokens sorted by expert into the GEMMs' row layouts and back with weights, the
gated activation between the GEMMs, the norms before and after the block with
its gate and residual scale, and the gradients of all of these.

Argument marshalling only, like dg.py: each function checks dtypes, shapes,
devices and contiguity and passes device pointers and the current HIP stream
to the library. There is no fallback: a missing library raises.

A block in FP8, masked layout (b1 [G, 2I, H], b2 [G, H, I] and their scales):

    plan = moe.Plan(tokens, top_k, G, "masked", max_m, H, device)
    moe.dispatch_fp8(plan, n, q, sfa, topk_ids=ids)
    dg.m_grouped_fp8_gemm_nt_masked(q, sfa, b1, sfb1, gu, plan.group_rows)
    moe.swiglu_fp8(gu, a, sfa2, rows=plan.group_rows, layout="masked")
    dg.m_grouped_fp8_gemm_nt_masked(a, sfa2, b2, sfb2, yp, plan.group_rows)
    moe.combine(plan, yp, y, weights=w)
    moe.block_norm(x, y, post_weight, gate, pre_weight, h, n)

With the UE8M0 or the FP8 x FP4 GEMMs dispatch_fp8 and swiglu_fp8 need ue8m0=True.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch

from . import dg
from .dg import DGError, _check, _current_device, _need  # noqa: F401  (DGError: what a failed call raises)

_LAYOUTS = {"dense": 0, "contiguous": 1, "masked": 2, "nopad": 3}
_BF16, _F32, _I32, _FP8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


class _PlanStruct(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int), ("max_tokens", ctypes.c_int), ("top_k", ctypes.c_int),
                ("num_groups", ctypes.c_int), ("rows", ctypes.c_int), ("hidden", ctypes.c_int),
                ("row_of", ctypes.c_void_p), ("group_rows", ctypes.c_void_p), ("grouped_layout", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_longlong)]


_vp, _i, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
# (name, argtypes, restype) of every symbol include/moe/dg_moe.h declares.
SIGNATURES = [
    ("dg_moe_workspace_bytes", [_vp], _ll),
    ("dg_moe_sort", [_vp, _vp, _i, _vp], _i),
    ("dg_moe_dispatch", [_vp, _vp, _vp, _vp, _i, _vp], _i),
    ("dg_moe_dispatch_fp8", [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp], _i),
    ("dg_moe_combine", [_vp, _vp, _vp, _vp, _i, _vp], _i),
    ("dg_moe_combine_bwd", [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp], _i),
    ("dg_moe_swiglu_fp8", [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp], _i),
    ("dg_moe_swiglu_bwd", [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp], _i),
    ("dg_moe_block_norm", [ctypes.c_char_p, _vp], _i),
    ("dg_moe_block_norm_workspace_bytes", [_i, _i], _ll),
    ("dg_moe_block_norm_bwd", [ctypes.c_char_p, _vp], _i),
]

# The argument structs dg_moe_norm and dg_moe_norm_bwd, packed in one go (a
# ctypes call converts its arguments one by one, 0.1 us each).
_NORM = struct.Struct("9P2f3i4x")
_NORM_BWD = struct.Struct("15Pqf3i")

_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library with this module's entry points bound."""
    global _lib
    if _lib is None:
        handle = dg.lib()
        for name, argtypes, restype in SIGNATURES:
            fn = getattr(handle, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = handle
    return _lib


def _int32(v: int) -> int:
    """A size as the library's int takes it; -1, which every call refuses, where it
    does not fit (ctypes would take it modulo 2^32)."""
    return v if -2 ** 31 <= v < 2 ** 31 else -1


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


# The handle of a device's current stream: a decode step's calls take a few
# microseconds each, of which torch.cuda.current_stream(...).cuda_stream, which
# builds a Stream object first, took 1.9 (this: 0.1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(index: int) -> int:
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _call(name: str, index: int, *args) -> None:
    """Calls an entry point on device `index`'s current stream, with that device
    current: the handle of a default stream is 0 on every device."""
    if _current_device() == index:
        status = getattr(lib(), name)(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            status = getattr(lib(), name)(*args, _stream(index))
    if status:
        _check(status, name)


def _want(t: torch.Tensor, name: str, dtype, shape, index: int) -> None:
    """As dg._need, with the whole shape and the device by its index (the
    cheapest way to ask: get_device() is -1 on the host)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return
    except AttributeError:
        pass
    _need(t, name, dtype, len(shape), _device(index))
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _optional(index: int, dtype, shape, **tensors) -> None:
    """_want for each tensor that is given."""
    for name, t in tensors.items():
        if t is not None:
            try:
                if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
                    continue
            except AttributeError:
                pass
            _want(t, name, dtype, shape, index)


def _device(index: int) -> torch.device:
    return torch.device("cuda", index) if index >= 0 else torch.device("cpu")


def _first(t: torch.Tensor, name: str, dtype, ndim: int) -> int:
    """Checks the tensor that says where a call runs and returns its device's index."""
    index = t.get_device() if isinstance(t, torch.Tensor) else -1
    if index < 0 or t.dtype is not dtype or t.dim() != ndim or not t.is_contiguous():
        _need(t, name, dtype, ndim, _device(index))
    return index


# ---------------------------------------------------------------------------
# Tokens to rows and back
# ---------------------------------------------------------------------------

def contiguous_rows(slots: int, num_groups: int) -> int:
    """Rows that hold `slots` slots in 128-row segments however they fall."""
    align = dg.get_mk_alignment_for_contiguous_layout()
    return (slots + min(slots, num_groups) * (align - 1) + align - 1) // align * align


class Plan:
    """Where the slots of a batch go, and the buffers that say so: kept by the
    caller from call to call, filled by sort() or by a dispatch with topk_ids.

    layout "contiguous", "masked" or "nopad"; rows: rows of the permuted
    buffers (contiguous: a multiple of 128, see contiguous_rows; masked: max_m
    rows a group); hidden: values of a token, a multiple of 128.

      row_of [max_tokens, top_k] int32: each slot's row, -1 where dropped
          (masked: group * rows + row)
      group_rows [num_groups] int32: the GEMMs' group_rows / masked_m
      grouped_layout [rows] int32 (contiguous; else None)

    Calls that use one plan have to be ordered (one stream, or events).
    """

    def __init__(self, max_tokens: int, top_k: int, num_groups: int, layout: str, rows: int, hidden: int, device):
        if layout not in ("contiguous", "masked", "nopad"):
            raise ValueError(f"layout must be contiguous, masked or nopad, got {layout!r}")
        device = torch.device(device)
        self.layout = layout
        self.max_tokens, self.top_k, self.num_groups = int(max_tokens), int(top_k), int(num_groups)
        self.rows, self.hidden = int(rows), int(hidden)
        self._struct = _PlanStruct(_LAYOUTS[layout], _int32(self.max_tokens), _int32(self.top_k),
                                   _int32(self.num_groups), _int32(self.rows), _int32(self.hidden))
        self._ref = ctypes.addressof(self._struct)
        size = lib().dg_moe_workspace_bytes(self._ref)
        if size < 0:
            raise ValueError(f"plan sizes out of range: max_tokens={max_tokens}, top_k={top_k}, "
                             f"num_groups={num_groups}, layout={layout}, rows={rows}, hidden={hidden}")
        if device.type != "cuda":
            raise ValueError(f"a plan lives on a GPU, got {device}")
        self.device = device if device.index is not None else torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        # one allocation, each part 16-byte aligned; -1: no slot has a row yet, no group has rows
        slots, rows_of_layout = self.max_tokens * self.top_k, self.rows if layout == "contiguous" else 0
        at_rows = (slots + 3) // 4 * 4
        at_layout = at_rows + (self.num_groups + 3) // 4 * 4
        ints = torch.full((at_layout + rows_of_layout,), -1, dtype=_I32, device=device)
        self.row_of = ints[:slots].view(self.max_tokens, self.top_k)
        self.group_rows = ints[at_rows:at_rows + self.num_groups]
        self.grouped_layout = ints[at_layout:] if layout == "contiguous" else None
        self.workspace = torch.empty(size, dtype=torch.uint8, device=device)
        s = self._struct
        s.row_of, s.group_rows, s.grouped_layout = (self.row_of.data_ptr(), self.group_rows.data_ptr(),
                                                    _ptr(self.grouped_layout))
        s.workspace, s.workspace_bytes = self.workspace.data_ptr(), size
        # shapes of the permuted buffers
        lead = (self.num_groups,) if layout == "masked" else ()
        self.rows_shape = torch.Size((*lead, self.rows, self.hidden))
        self.scale_shape = torch.Size((*lead, self.hidden // 128, dg.get_tma_aligned_size(self.rows, 4)))

    def _tokens(self, t: torch.Tensor, name: str, dtype, width: int) -> int:
        """Checks a [tokens, width] tensor and returns tokens."""
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype is not dtype or t.get_device() != self._index \
                or not t.is_contiguous():
            _need(t, name, dtype, 2, self.device)
        n, w = t.shape
        if w != width or n > self.max_tokens:
            raise ValueError(f"{name} must have shape (at most {self.max_tokens}, {width}), got {tuple(t.shape)}")
        return n

    def _ids(self, topk_ids, n: int) -> Optional[int]:
        if topk_ids is None:
            return None
        if self._tokens(topk_ids, "topk_ids", _I32, self.top_k) != n:
            raise ValueError("topk_ids and x differ in tokens")
        # an empty batch still sorts (to groups without rows): any address will do
        return topk_ids.data_ptr() or self.row_of.data_ptr() or self.workspace.data_ptr()


def sort(plan: Plan, topk_ids: torch.Tensor) -> Plan:
    """Sorts the slots of topk_ids [tokens, top_k] int32 by group, stably, into
    the plan; ids outside [0, num_groups) drop their slot."""
    n = plan._tokens(topk_ids, "topk_ids", _I32, plan.top_k)
    _call("dg_moe_sort", plan._index, plan._ref, topk_ids.data_ptr(), n)
    return plan


def dispatch(plan: Plan, x, xp, topk_ids=None) -> torch.Tensor:
    """xp[row_of[t, j]] = x[t] for every slot. x [tokens, hidden] bfloat16,
    xp [rows, hidden] bfloat16 (masked [G, rows, hidden]); rows without a token
    are not written. topk_ids: sorts first. Gradient: combine(plan, dxp, dx)."""
    n = plan._tokens(x, "x", _BF16, plan.hidden)
    _want(xp, "xp", _BF16, plan.rows_shape, plan._index)
    _call("dg_moe_dispatch", plan._index, plan._ref, plan._ids(topk_ids, n), x.data_ptr(), xp.data_ptr(), n)
    return xp


def dispatch_fp8(plan: Plan, x, q, sfa, topk_ids=None, ue8m0: bool = False):
    """dispatch() into the GEMMs' LHS operand: q like xp in float8_e4m3fn and
    sfa [hidden/128, tma_aligned(rows)] float32 (masked: [G, ...]), one scale
    max(amax, 1e-4) / 448 per 128 values (ue8m0: rounded up to a power of two).
    GEMMs called with ue8m0=True and the FP8 x FP4 GEMMs read only a scale's
    exponent: their operands need ue8m0=True here too, or blocks come out up to a
    factor of two too small."""
    n = plan._tokens(x, "x", _BF16, plan.hidden)
    _want(q, "q", _FP8, plan.rows_shape, plan._index)
    _want(sfa, "sfa", _F32, plan.scale_shape, plan._index)
    _call("dg_moe_dispatch_fp8", plan._index, plan._ref, plan._ids(topk_ids, n), x.data_ptr(), q.data_ptr(),
          sfa.data_ptr(), n, ue8m0)
    return q, sfa


def combine(plan: Plan, yp, y, weights=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * yp[row_of[t, j]] (weights None: ones), zeros
    for a token without rows. yp like dispatch's xp, y [tokens, hidden]
    bfloat16, weights [tokens, top_k] float32."""
    n = plan._tokens(y, "y", _BF16, plan.hidden)
    _want(yp, "yp", _BF16, plan.rows_shape, plan._index)
    if weights is not None:
        _want(weights, "weights", _F32, (n, plan.top_k), plan._index)
    _call("dg_moe_combine", plan._index, plan._ref, yp.data_ptr(), _ptr(weights), y.data_ptr(), n)
    return y


def combine_bwd(plan: Plan, dy, yp, weights, dyp, dweights=None):
    """Gradient of combine(): dyp[row_of[t, j]] = weights[t, j] * dy[t] and
    dweights[t, j] = <dy[t], yp[row_of[t, j]]>. dweights None: not wanted, and
    yp is not read (may be None)."""
    n = plan._tokens(dy, "dy", _BF16, plan.hidden)
    _want(weights, "weights", _F32, (n, plan.top_k), plan._index)
    _want(dyp, "dyp", _BF16, plan.rows_shape, plan._index)
    if dweights is not None:
        _want(dweights, "dweights", _F32, (n, plan.top_k), plan._index)
    if dweights is not None or yp is not None:
        _want(yp, "yp", _BF16, plan.rows_shape, plan._index)
    _call("dg_moe_combine_bwd", plan._index, plan._ref, dy.data_ptr(), _ptr(yp), weights.data_ptr(), dyp.data_ptr(),
          _ptr(dweights), n)
    return dyp, dweights


# ---------------------------------------------------------------------------
# The gated activation
# ---------------------------------------------------------------------------

def _glu(gu, rows, layout: str):
    """(layout, m, groups, inner, device index) of a gate-and-up buffer and its row selector."""
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {', '.join(_LAYOUTS)}, got {layout!r}")
    index = _first(gu, "gu", _BF16, 3 if layout == "masked" else 2)
    m, width = gu.shape[-2:]
    if width % 256:
        raise ValueError("gu must hold 2 * inner columns, inner a multiple of 128")
    if layout == "dense":
        if rows is not None:
            raise ValueError("the dense layout takes no rows")
        return 0, m, 1, width // 2, index
    if _first(rows, "rows", _I32, 1) != index:
        raise ValueError(f"rows must be on {gu.device}")
    if layout == "contiguous":
        if rows.shape[0] != m:
            raise ValueError("rows must be grouped_layout, one int32 a row of gu")
        return 1, m, 1, width // 2, index
    if layout == "masked" and rows.shape[0] != gu.shape[0]:
        raise ValueError("rows must be masked_m, one int32 a group of gu")
    return _LAYOUTS[layout], m, _int32(rows.shape[0]), width // 2, index


def swiglu_fp8(gu, q, sfa, rows=None, layout: str = "dense", ue8m0: bool = False):
    """silu(g) * u of gu = [g | u] ([M, 2I] bfloat16, masked [G, max_m, 2I]),
    quantised into the next GEMM's LHS operand: q [M, I] float8_e4m3fn and
    sfa [I/128, tma_aligned(M)] float32 (masked: [G, ...]).

    rows says which rows hold tokens, as the GEMM of that layout takes it:
    grouped_layout [M] (contiguous; a negative id holds none), group_rows [G]
    (nopad), masked_m [G] (masked), None (dense: all). Others are not written.
    ue8m0 by the GEMM that reads q, as for dispatch_fp8."""
    kind, m, groups, inner, index = _glu(gu, rows, layout)
    lead = gu.shape[:-2]
    _want(q, "q", _FP8, (*lead, m, inner), index)
    _want(sfa, "sfa", _F32, (*lead, inner // 128, (m + 3) // 4 * 4), index)
    _call("dg_moe_swiglu_fp8", index, gu.data_ptr(), q.data_ptr(), sfa.data_ptr(), _ptr(rows), kind, m, groups, inner,
          ue8m0)
    return q, sfa


def swiglu_bwd(da, gu, dgu, rows=None, layout: str = "dense") -> torch.Tensor:
    """Gradient of silu(g) * u: da [M, I] bfloat16 (masked [G, max_m, I]) to
    dgu like gu; rows and layout as for swiglu_fp8."""
    kind, m, groups, inner, index = _glu(gu, rows, layout)
    _want(da, "da", _BF16, (*gu.shape[:-1], inner), index)
    _want(dgu, "dgu", _BF16, gu.shape, index)
    _call("dg_moe_swiglu_bwd", index, da.data_ptr(), gu.data_ptr(), dgu.data_ptr(), _ptr(rows), kind, m, groups, inner)
    return dgu


# ---------------------------------------------------------------------------
# The norms around the block
# ---------------------------------------------------------------------------

def _gate_kind(gate, n: int, hidden: int, index: int) -> int:
    if gate is None:
        return 0
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    if gate.dim() == 1:
        if gate.shape[0] == hidden:
            _want(gate, "gate", _F32, (hidden,), index)
            return 1
        raise ValueError(f"a gate of one dimension is per channel ({hidden}); give one per token as ({n}, 1), "
                         f"got {tuple(gate.shape)}")
    if gate.shape == (n, 1):
        _want(gate, "gate", _F32, (n, 1), index)
        return 2
    _want(gate, "gate", _BF16, (n, hidden), index)
    return 3


def block_norm(x, y, post_weight, gate, pre_weight, h, n, rstd_post=None, rstd_pre=None,
               residual_scale: float = 1.0, eps: float = 1e-6):
    """The step between two blocks, with norm(v; w) = v * rsqrt(mean(v^2) + eps) * w:

        h = residual_scale * x + gate * norm(y; post_weight)
        n = norm(h; pre_weight)

    x, y, h, n [tokens, hidden] bfloat16; post_weight, pre_weight [hidden]
    float32; gate [hidden] float32, [tokens, 1] float32, [tokens, hidden]
    bfloat16 or None; rstd_post, rstd_pre [tokens] float32 or None: kept for
    block_norm_bwd. y None (with post_weight, gate, h None): only n = norm(x).
    post_weight None: y is not normalised. n None (with pre_weight): only h."""
    index = _first(x, "x", _BF16, 2)
    t, hidden = shape = x.shape
    _optional(index, _BF16, shape, y=y, h=h, n=n)
    _optional(index, _F32, (hidden,), post_weight=post_weight, pre_weight=pre_weight)
    _optional(index, _F32, (t,), rstd_post=rstd_post, rstd_pre=rstd_pre)
    kind = _gate_kind(gate, t, hidden, index)
    args = _NORM.pack(x.data_ptr(), _ptr(y), _ptr(post_weight), _ptr(gate), _ptr(pre_weight), _ptr(h), _ptr(n),
                      _ptr(rstd_post), _ptr(rstd_pre), residual_scale, eps, kind, t, hidden)
    _call("dg_moe_block_norm", index, args)
    return h, n


def block_norm_workspace(tokens: int, hidden: int, device) -> torch.Tensor:
    """A workspace for block_norm_bwd, to be kept from call to call."""
    size = lib().dg_moe_block_norm_workspace_bytes(_int32(int(tokens)), _int32(int(hidden)))
    if size < 0:
        raise ValueError(f"sizes out of range: tokens={tokens}, hidden={hidden}")
    return torch.empty(size, dtype=torch.uint8, device=device)


def block_norm_bwd(dh, dn, h, y, post_weight, gate, pre_weight, rstd_post, rstd_pre, dx, dy, dpost_weight, dgate,
                   dpre_weight, workspace, residual_scale: float = 1.0):
    """Gradient of block_norm(): from dh (of h, along the residual stream; None:
    none) and dn (of n; None: unused) to dx, dy [tokens, hidden] bfloat16,
    dpost_weight, dpre_weight [hidden] float32 and dgate like the gate. h, y,
    the weights, the gate and the rstd values are those of the forward call;
    dpost_weight, dgate and dpre_weight may be None where not wanted."""
    index = _first(dx, "dx", _BF16, 2)
    t, hidden = shape = dx.shape
    _optional(index, _BF16, shape, dh=dh, dn=dn, h=h, y=y, dy=dy)
    _optional(index, _F32, (hidden,), post_weight=post_weight, pre_weight=pre_weight, dpost_weight=dpost_weight,
              dpre_weight=dpre_weight)
    _optional(index, _F32, (t,), rstd_post=rstd_post, rstd_pre=rstd_pre)
    kind = _gate_kind(gate, t, hidden, index)
    if dgate is not None and gate is not None:
        _want(dgate, "dgate", gate.dtype, gate.shape, index)
    if _first(workspace, "workspace", torch.uint8, 1) != index:
        raise ValueError(f"workspace must be on {dx.device}")
    args = _NORM_BWD.pack(_ptr(dh), _ptr(dn), _ptr(h), _ptr(y), _ptr(post_weight), _ptr(gate), _ptr(pre_weight),
                          _ptr(rstd_post), _ptr(rstd_pre), dx.data_ptr(), _ptr(dy), _ptr(dpost_weight), _ptr(dgate),
                          _ptr(dpre_weight), workspace.data_ptr(), workspace.numel(), residual_scale, kind, t, hidden)
    _call("dg_moe_block_norm_bwd", index, args)
    return dx, dy
