"""B200-native block-scaled quantisation of BF16 tensors: FP8 block-wise
(128x128, FP32 scales), MXFP8 (1x32, UE8M0) and NVFP4 (1x16, E4M3 block
scale + FP32 global scale), quantise / dequantise / fake-quantise.

Formats as listed on "Low Precision RL" ("Choose a precision" table); NVFP4
fake-quantisation with sibling-shared global amax and the straight-through
backward as described in the verl NVFP4 QAT article (sections 2.3, 2.4).

This module is argument marshalling only: every step runs in libpwq's CUDA
kernels (include/pwq.h).  PyTorch supplies device memory and the stream.
Functions take CUDA tensors ([M, N] or batched [B, M, N], last dimension
contiguous) and return newly allocated outputs unless ``out=`` buffers are
given.  Nothing synchronises.
"""
import ctypes
from typing import List, Optional, Sequence, Tuple

import torch

from ._lib import (LIB_PATH, PWQ_MAX_SIBLINGS, PwqError, PwqTensor, check, lib,  # noqa: F401
                   status_string)

__all__ = [
    "fp8_block_quant", "fp8_block_dequant", "mxfp8_quant", "mxfp8_dequant",
    "nvfp4_group_amax", "nvfp4_quant", "nvfp4_dequant", "nvfp4_fake_quant",
    "nvfp4_workspace_size", "NVFP4FakeQuantSTE", "nvfp4_fake_quant_ste", "build_info",
    "device_error", "PwqError", "LIB_PATH", "fp8_block_quant_grouped", "fp8_block_dequant_grouped",
    "mxfp8_quant_grouped", "mxfp8_dequant_grouped", "nvfp4_dequant_grouped", "nvfp4_quant_grouped",
    "nvfp4_fake_quant_grouped", "fp8_block_requant", "fp8_block_requant_mxfp8", "fp8_block_requant_nvfp4",
    "fp8_block_requant_nvfp4_grouped", "fp8_block_requant_grouped", "fp8_block_requant_mxfp8_grouped",
    "NVFP4ActivationObserver", "nvfp4_w4a4_fake_quant_ste", "OBSERVERS", "mma_scale_bytes", "scales_to_mma",
    "scales_from_mma", "mxfp8_quant_grouped_mma", "nvfp4_quant_grouped_mma", "mxfp8_matmul", "nvfp4_matmul",
    "rms_norm_mxfp8", "rms_norm_nvfp4", "rms_norm_fake_quant", "rms_norm_backward", "rms_norm_fake_quant_ste",
]

_CODE_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


# The current stream's handle without making a Stream object (2 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _desc(t: torch.Tensor, name: str, packed: bool = False) -> PwqTensor:
    """pwq_tensor for a [M, N] / [B, M, N] CUDA tensor.  For packed E2M1 codes
    (uint8, two per byte) the logical column count is twice the byte count."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    shape, st = t.shape, t.stride()
    if len(shape) == 2:
        M, N = shape
        B, bs, rs, last = 1, M * st[0], st[0], st[1]
    elif len(shape) == 3:
        B, M, N = shape
        bs, rs, last = st
    else:
        raise ValueError("%s must be 2-D [M, N] or 3-D [B, M, N], got shape %s" % (name, tuple(shape)))
    cols = 2 * N if packed else N
    if B == 0 or M == 0 or N == 0:
        # an empty tensor's strides are arbitrary; the library launches nothing for it
        return PwqTensor(t.data_ptr(), B, M, cols, M * N, N)
    if N > 1 and last != 1:
        raise ValueError("%s: last dimension must be contiguous" % name)
    if M == 1 or B == 1:      # torch leaves the stride of a dimension of size 1 arbitrary
        if M == 1:
            rs = -(-N // 16) * 16
            if B > 1 and bs < rs:
                rs = N
        if B == 1:
            bs = M * rs
    return PwqTensor(t.data_ptr(), B, M, cols, bs, rs)


def _new_desc(t: torch.Tensor, like: PwqTensor, cols: int) -> PwqTensor:
    """_desc of a tensor just allocated with like's batch and rows (a third of its time)."""
    n = t.shape[-1]
    return PwqTensor(t.data_ptr(), like.batch, like.rows, cols, like.rows * n, n)


def _lead(x: torch.Tensor):
    return tuple(x.shape[:-2]) if x.dim() == 3 else ()


def _check_dtype(t, dtypes, name):
    if t.dtype not in dtypes:
        raise TypeError("%s must have dtype in %s, got %s" % (name, dtypes, t.dtype))


# ---------------------------------------------------------------- FP8 block-wise

def fp8_block_quant(x: torch.Tensor, out: Optional[torch.Tensor] = None,
                    scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """128x128 block-wise FP8: returns (codes float8_e4m3fn [.., M, N],
    scale float32 [.., ceil(M/128), ceil(N/128)]) with s = fl(amax/448)."""
    _check_dtype(x, (torch.bfloat16,), "x")
    M, N = x.shape[-2:]
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    if scale is None:
        scale = torch.empty(_lead(x) + (-(-M // 128), -(-N // 128)), dtype=torch.float32, device=x.device)
    _check_dtype(out, _CODE_DTYPES, "out")
    dx, dq = _desc(x, "x"), _desc(out, "out")
    check(lib.fp8_block_quant(ctypes.byref(dx), ctypes.byref(dq), scale.data_ptr(), _stream(x)),
          "fp8_block_quant")
    return out, scale


def fp8_block_dequant(q: torch.Tensor, scale: torch.Tensor,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """BF16 y = bf16(fl(dec(q) * s)) for FP8 block-wise codes and scales."""
    _check_dtype(q, _CODE_DTYPES, "q")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if not scale.is_contiguous() or scale.dtype != torch.float32:
        raise ValueError("scale must be a contiguous float32 tensor")
    dq, dy = _desc(q, "q"), _desc(out, "out")
    check(lib.fp8_block_dequant(ctypes.byref(dq), scale.data_ptr(), ctypes.byref(dy), _stream(q)),
          "fp8_block_dequant")
    return out


# ---------------------------------------------------------------- MXFP8

def mxfp8_quant(x: torch.Tensor, out: Optional[torch.Tensor] = None,
                scale: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """MXFP8 1x32: returns (codes float8_e4m3fn [.., M, N], UE8M0 scale bytes
    uint8 [.., M, N/32])."""
    _check_dtype(x, (torch.bfloat16,), "x")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    if scale is None:
        scale = torch.empty(x.shape[:-1] + (x.shape[-1] // 32,), dtype=torch.uint8, device=x.device)
    dx, dq = _desc(x, "x"), _desc(out, "out")
    check(lib.mxfp8_quant(ctypes.byref(dx), ctypes.byref(dq), scale.data_ptr(), _stream(x)), "mxfp8_quant")
    return out, scale


def mxfp8_dequant(q: torch.Tensor, scale: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _check_dtype(q, _CODE_DTYPES, "q")
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if not scale.is_contiguous():
        raise ValueError("scale must be contiguous")
    dq, dy = _desc(q, "q"), _desc(out, "out")
    check(lib.mxfp8_dequant(ctypes.byref(dq), scale.data_ptr(), ctypes.byref(dy), _stream(q)),
          "mxfp8_dequant")
    return out


# ---------------------------------------------------------------- NVFP4

def _siblings(xs) -> List[torch.Tensor]:
    if isinstance(xs, torch.Tensor):
        xs = [xs]
    xs = list(xs)
    if not 1 <= len(xs) <= PWQ_MAX_SIBLINGS:
        raise ValueError("1..%d sibling tensors expected" % PWQ_MAX_SIBLINGS)
    for i, x in enumerate(xs):
        _check_dtype(x, (torch.bfloat16,), "x[%d]" % i)
    return xs


def _desc_array(ts, name, packed=False):
    arr = (PwqTensor * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = _desc(t, "%s[%d]" % (name, i), packed)
    return arr


def _batch(x: torch.Tensor) -> int:
    return x.shape[0] if x.dim() == 3 else 1


def nvfp4_workspace_size(xs) -> int:
    xs = _siblings(xs)
    return int(lib.nvfp4_workspace_size(len(xs), _desc_array(xs, "x")))


def _workspace(xs, arr) -> torch.Tensor:
    n = int(lib.nvfp4_workspace_size(len(xs), arr))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=xs[0].device)


def nvfp4_group_amax(xs, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Group amax A_b = max |x| over all siblings' batch slice b, float32 [B].
    This is the value to all-reduce (MAX) when a group is sharded."""
    xs = _siblings(xs)
    if out is None:
        out = torch.empty(_batch(xs[0]), dtype=torch.float32, device=xs[0].device)
    arr = _desc_array(xs, "x")
    check(lib.nvfp4_group_amax(arr, len(xs), out.data_ptr(), _stream(xs[0])), "nvfp4_group_amax")
    return out


def nvfp4_quant(xs, amax: Optional[torch.Tensor] = None, out=None, sb=None,
                global_scale: Optional[torch.Tensor] = None):
    """NVFP4 quantisation of a sibling group (one tensor or a list sharing
    one global amax per batch index).  Returns (packed codes list uint8
    [.., M, N/2], block scales list float8_e4m3fn [.., M, N/16], global
    scales float32 [B]).  ``amax`` (float32 [B]) replaces the on-device
    group amax reduction (cached or all-reduced value)."""
    single = isinstance(xs, torch.Tensor)
    xs = _siblings(xs)
    dev = xs[0].device
    B = _batch(xs[0])
    if out is None:
        out = [torch.empty(x.shape[:-1] + (x.shape[-1] // 2,), dtype=torch.uint8, device=dev) for x in xs]
    if sb is None:
        sb = [torch.empty(x.shape[:-1] + (x.shape[-1] // 16,), dtype=torch.float8_e4m3fn, device=dev)
              for x in xs]
    if global_scale is None:
        global_scale = torch.empty(B, dtype=torch.float32, device=dev)
    for t in sb:
        if not t.is_contiguous():
            raise ValueError("block scale tensors must be contiguous")
    ax = _desc_array(xs, "x")
    aq = _desc_array(out, "out", packed=True)
    sbp = (ctypes.c_void_p * len(xs))(*[t.data_ptr() for t in sb])
    ws = None if amax is not None else _workspace(xs, ax)
    check(lib.nvfp4_quant(ax, len(xs), aq, sbp, global_scale.data_ptr(),
                          amax.data_ptr() if amax is not None else None,
                          ws.data_ptr() if ws is not None else None,
                          ws.numel() if ws is not None else 0, _stream(xs[0])), "nvfp4_quant")
    if single:
        return out[0], sb[0], global_scale
    return out, sb, global_scale


def nvfp4_dequant(packed: torch.Tensor, sb: torch.Tensor, global_scale: torch.Tensor,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """BF16 y = bf16(fl((dec(c) * dec(sb)) * gs)) for one NVFP4 tensor."""
    _check_dtype(packed, (torch.uint8,), "packed")
    if out is None:
        out = torch.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), dtype=torch.bfloat16,
                          device=packed.device)
    if not sb.is_contiguous() or not global_scale.is_contiguous():
        raise ValueError("sb and global_scale must be contiguous")
    dq, dy = _desc(packed, "packed", packed=True), _desc(out, "out")
    check(lib.nvfp4_dequant(ctypes.byref(dq), sb.data_ptr(), global_scale.data_ptr(), ctypes.byref(dy),
                            _stream(packed)), "nvfp4_dequant")
    return out


def nvfp4_fake_quant(xs, amax: Optional[torch.Tensor] = None, out=None, inplace: bool = False,
                     amax_out: Optional[torch.Tensor] = None):
    """NVFP4 QDQ of a sibling group: BF16 outputs equal to
    nvfp4_dequant(nvfp4_quant(x)), without materialising codes.  Returns the
    output tensor (single input) or list of outputs."""
    single = isinstance(xs, torch.Tensor)
    xs = _siblings(xs)
    if out is None:
        out = xs if inplace else [torch.empty_like(x) for x in xs]
    elif isinstance(out, torch.Tensor):
        out = [out]
    ax = _desc_array(xs, "x")
    ay = _desc_array(out, "out")
    ws = None if amax is not None else _workspace(xs, ax)
    check(lib.nvfp4_fake_quant(ax, ay, len(xs), amax.data_ptr() if amax is not None else None,
                               amax_out.data_ptr() if amax_out is not None else None,
                               ws.data_ptr() if ws is not None else None,
                               ws.numel() if ws is not None else 0, _stream(xs[0])), "nvfp4_fake_quant")
    return out[0] if single else out


class NVFP4FakeQuantSTE(torch.autograd.Function):
    """Fake-quantised forward, straight-through backward: grad_x = grad_y and
    no gradient for the amax (verl NVFP4 QAT article, section 2.3)."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, amax: Optional[torch.Tensor] = None):
        return nvfp4_fake_quant(x, amax=amax)

    @staticmethod
    def backward(ctx, grad_y):
        return grad_y, None


class _SiblingSTE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, amax, *xs):
        return tuple(nvfp4_fake_quant(list(xs), amax=amax))

    @staticmethod
    def backward(ctx, *grads):
        return (None,) + tuple(grads)


def nvfp4_fake_quant_ste(xs: Sequence[torch.Tensor], amax: Optional[torch.Tensor] = None):
    """Sibling-group fake-quantisation with the straight-through backward."""
    if isinstance(xs, torch.Tensor):
        return NVFP4FakeQuantSTE.apply(xs, amax)
    return list(_SiblingSTE.apply(amax, *xs))


# ---------------------------------------------------------------- NVFP4 4over6

def nvfp4_4over6_quant(xs, e4m3_max: int = 256, amax: Optional[torch.Tensor] = None, out=None, sb=None,
                       global_scale: Optional[torch.Tensor] = None):
    """NVFP4 "4over6" quantisation of a sibling group (vime pull request
    #503, NVFP4 QDQ config: NVTE_NVFP4_4OVER6, E4M3 maximum 256 by default).
    Every block keeps the candidate -- its amax mapped to 6 or to 4 -- whose
    dequantised values have the smaller squared error; gs = fl(A / (6 E)).
    Returns what nvfp4_quant returns; nvfp4_dequant reads the result."""
    single = isinstance(xs, torch.Tensor)
    xs = _siblings(xs)
    dev = xs[0].device
    B = _batch(xs[0])
    if out is None:
        out = [torch.empty(x.shape[:-1] + (x.shape[-1] // 2,), dtype=torch.uint8, device=dev) for x in xs]
    if sb is None:
        sb = [torch.empty(x.shape[:-1] + (x.shape[-1] // 16,), dtype=torch.float8_e4m3fn, device=dev)
              for x in xs]
    if global_scale is None:
        global_scale = torch.empty(B, dtype=torch.float32, device=dev)
    for t in sb:
        if not t.is_contiguous():
            raise ValueError("block scale tensors must be contiguous")
    ax = _desc_array(xs, "x")
    aq = _desc_array(out, "out", packed=True)
    sbp = (ctypes.c_void_p * len(xs))(*[t.data_ptr() for t in sb])
    ws = None
    if amax is None:
        ws = torch.empty(max(int(lib.nvfp4_4over6_workspace_size(len(xs), ax)), 256), dtype=torch.uint8, device=dev)
    check(lib.nvfp4_4over6_quant(ax, len(xs), aq, sbp, global_scale.data_ptr(),
                                 amax.data_ptr() if amax is not None else None, int(e4m3_max),
                                 ws.data_ptr() if ws is not None else None,
                                 ws.numel() if ws is not None else 0, _stream(xs[0])), "nvfp4_4over6_quant")
    if single:
        return out[0], sb[0], global_scale
    return out, sb, global_scale


def nvfp4_4over6_fake_quant(xs, e4m3_max: int = 256, amax: Optional[torch.Tensor] = None, out=None,
                            inplace: bool = False, amax_out: Optional[torch.Tensor] = None):
    """BF16 outputs equal to nvfp4_dequant(nvfp4_4over6_quant(x)), without
    materialising codes.  Returns the output tensor or list of outputs."""
    single = isinstance(xs, torch.Tensor)
    xs = _siblings(xs)
    if out is None:
        out = xs if inplace else [torch.empty_like(x) for x in xs]
    elif isinstance(out, torch.Tensor):
        out = [out]
    ax = _desc_array(xs, "x")
    ay = _desc_array(out, "out")
    ws = None
    if amax is None:
        ws = torch.empty(max(int(lib.nvfp4_4over6_workspace_size(len(xs), ax)), 256), dtype=torch.uint8,
                         device=xs[0].device)
    check(lib.nvfp4_4over6_fake_quant(ax, ay, len(xs), amax.data_ptr() if amax is not None else None,
                                      amax_out.data_ptr() if amax_out is not None else None, int(e4m3_max),
                                      ws.data_ptr() if ws is not None else None,
                                      ws.numel() if ws is not None else 0, _stream(xs[0])),
          "nvfp4_4over6_fake_quant")
    return out[0] if single else out


# ---------------------------------------------------------------- grouped calls (one launch per list)

def _ptrs(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def fp8_block_quant_grouped(xs: Sequence[torch.Tensor], out=None, scale=None):
    """fp8_block_quant of every tensor of a list (a layer's weights) in one
    launch.  Returns (codes list, scales list)."""
    xs = list(xs)
    for i, x in enumerate(xs):
        _check_dtype(x, (torch.bfloat16,), "x[%d]" % i)
    if out is None:
        out = [torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device) for x in xs]
    if scale is None:
        scale = [torch.empty(_lead(x) + (-(-x.shape[-2] // 128), -(-x.shape[-1] // 128)), dtype=torch.float32,
                             device=x.device) for x in xs]
    if xs:
        check(lib.fp8_block_quant_grouped(len(xs), _desc_array(xs, "x"), _desc_array(out, "out"), _ptrs(scale),
                                          _stream(xs[0])), "fp8_block_quant_grouped")
    return out, scale


def fp8_block_dequant_grouped(qs: Sequence[torch.Tensor], scales: Sequence[torch.Tensor], out=None):
    qs = list(qs)
    if out is None:
        out = [torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) for q in qs]
    if qs:
        check(lib.fp8_block_dequant_grouped(len(qs), _desc_array(qs, "q"), _ptrs(scales), _desc_array(out, "out"),
                                            _stream(qs[0])), "fp8_block_dequant_grouped")
    return out


def mxfp8_quant_grouped(xs: Sequence[torch.Tensor], out=None, scale=None):
    xs = list(xs)
    if out is None:
        out = [torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device) for x in xs]
    if scale is None:
        scale = [torch.empty(x.shape[:-1] + (x.shape[-1] // 32,), dtype=torch.uint8, device=x.device) for x in xs]
    if xs:
        check(lib.mxfp8_quant_grouped(len(xs), _desc_array(xs, "x"), _desc_array(out, "out"), _ptrs(scale),
                                      _stream(xs[0])), "mxfp8_quant_grouped")
    return out, scale


def mxfp8_dequant_grouped(qs: Sequence[torch.Tensor], scales: Sequence[torch.Tensor], out=None):
    qs = list(qs)
    if out is None:
        out = [torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) for q in qs]
    if qs:
        check(lib.mxfp8_dequant_grouped(len(qs), _desc_array(qs, "q"), _ptrs(scales), _desc_array(out, "out"),
                                        _stream(qs[0])), "mxfp8_dequant_grouped")
    return out


def nvfp4_dequant_grouped(packed: Sequence[torch.Tensor], sb: Sequence[torch.Tensor],
                          global_scale: Sequence[torch.Tensor], out=None):
    packed = list(packed)
    if out is None:
        out = [torch.empty(p.shape[:-1] + (p.shape[-1] * 2,), dtype=torch.bfloat16, device=p.device)
               for p in packed]
    if packed:
        check(lib.nvfp4_dequant_grouped(len(packed), _desc_array(packed, "packed", packed=True), _ptrs(sb),
                                        _ptrs(global_scale), _desc_array(out, "out"), _stream(packed[0])),
              "nvfp4_dequant_grouped")
    return out


def _groups(groups):
    groups = [_siblings(g) for g in groups]
    flat = [x for g in groups for x in g]
    sizes = (ctypes.c_int * len(groups))(*[len(g) for g in groups])
    return groups, flat, sizes


def nvfp4_quant_grouped(groups: Sequence[Sequence[torch.Tensor]], out=None, sb=None, global_scale=None):
    """NVFP4 quantisation of several sibling groups (e.g. a layer's {q,k,v},
    {o}, {gate,up}, {down}) in one single-pass launch.  Returns (packed
    codes per group, block scales per group, global scales per group)."""
    groups, flat, sizes = _groups(groups)
    dev = flat[0].device
    if out is None:
        out = [[torch.empty(x.shape[:-1] + (x.shape[-1] // 2,), dtype=torch.uint8, device=dev) for x in g]
               for g in groups]
    if sb is None:
        sb = [[torch.empty(x.shape[:-1] + (x.shape[-1] // 16,), dtype=torch.float8_e4m3fn, device=dev) for x in g]
              for g in groups]
    if global_scale is None:
        global_scale = [torch.empty(_batch(g[0]), dtype=torch.float32, device=dev) for g in groups]
    ax = _desc_array(flat, "x")
    ws_bytes = int(lib.nvfp4_workspace_size_grouped(len(groups), sizes, ax))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    check(lib.nvfp4_quant_grouped(len(groups), sizes, ax, _desc_array([p for g in out for p in g], "out", packed=True),
                                  _ptrs([s for g in sb for s in g]), _ptrs(global_scale), ws.data_ptr(), ws.numel(),
                                  _stream(flat[0])), "nvfp4_quant_grouped")
    return out, sb, global_scale


def nvfp4_fake_quant_grouped(groups: Sequence[Sequence[torch.Tensor]], out=None, inplace: bool = False,
                             amax_out=None):
    """NVFP4 fake-quantisation of several sibling groups in one single-pass
    launch.  Returns the BF16 outputs per group."""
    groups, flat, sizes = _groups(groups)
    dev = flat[0].device
    if out is None:
        out = groups if inplace else [[torch.empty_like(x) for x in g] for g in groups]
    ax = _desc_array(flat, "x")
    ws_bytes = int(lib.nvfp4_workspace_size_grouped(len(groups), sizes, ax))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    ao = None
    if amax_out is not None:
        ao = (ctypes.c_void_p * len(groups))(*[a.data_ptr() if a is not None else None for a in amax_out])
    check(lib.nvfp4_fake_quant_grouped(len(groups), sizes, ax, _desc_array([y for g in out for y in g], "out"), ao,
                                       ws.data_ptr(), ws.numel(), _stream(flat[0])), "nvfp4_fake_quant_grouped")
    return out


def nvfp4_4over6_quant_grouped(groups: Sequence[Sequence[torch.Tensor]], e4m3_max: int = 256, out=None, sb=None,
                               global_scale=None):
    """NVFP4 "4over6" quantisation of several sibling groups (two launches per
    16 members).  Returns what nvfp4_quant_grouped returns."""
    groups, flat, sizes = _groups(groups)
    dev = flat[0].device
    if out is None:
        out = [[torch.empty(x.shape[:-1] + (x.shape[-1] // 2,), dtype=torch.uint8, device=dev) for x in g]
               for g in groups]
    if sb is None:
        sb = [[torch.empty(x.shape[:-1] + (x.shape[-1] // 16,), dtype=torch.float8_e4m3fn, device=dev) for x in g]
              for g in groups]
    if global_scale is None:
        global_scale = [torch.empty(_batch(g[0]), dtype=torch.float32, device=dev) for g in groups]
    ax = _desc_array(flat, "x")
    ws_bytes = int(lib.nvfp4_4over6_workspace_size_grouped(len(groups), sizes, ax))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    check(lib.nvfp4_4over6_quant_grouped(len(groups), sizes, ax,
                                         _desc_array([p for g in out for p in g], "out", packed=True),
                                         _ptrs([s for g in sb for s in g]), _ptrs(global_scale), int(e4m3_max),
                                         ws.data_ptr(), ws.numel(), _stream(flat[0])), "nvfp4_4over6_quant_grouped")
    return out, sb, global_scale


def nvfp4_4over6_fake_quant_grouped(groups: Sequence[Sequence[torch.Tensor]], e4m3_max: int = 256, out=None,
                                    inplace: bool = False, amax_out=None):
    """NVFP4 "4over6" fake-quantisation of several sibling groups.  Returns
    the BF16 outputs per group."""
    groups, flat, sizes = _groups(groups)
    dev = flat[0].device
    if out is None:
        out = groups if inplace else [[torch.empty_like(x) for x in g] for g in groups]
    ax = _desc_array(flat, "x")
    ws_bytes = int(lib.nvfp4_4over6_workspace_size_grouped(len(groups), sizes, ax))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    ao = None
    if amax_out is not None:
        ao = (ctypes.c_void_p * len(groups))(*[a.data_ptr() if a is not None else None for a in amax_out])
    check(lib.nvfp4_4over6_fake_quant_grouped(len(groups), sizes, ax, _desc_array([y for g in out for y in g], "out"),
                                              ao, int(e4m3_max), ws.data_ptr(), ws.numel(), _stream(flat[0])),
          "nvfp4_4over6_fake_quant_grouped")
    return out


# ---------------------------------------------------------------- block scales in the tensor-core layout

def mma_scale_bytes(batch: int, rows: int, scale_cols: int) -> int:
    """Bytes of an [B][M][S] scale array in the tensor-core tile layout
    (include/pwq.h: 128 x 4 tiles of 512 bytes, zero padding)."""
    return int(lib.pwq_mma_scale_bytes(batch, rows, scale_cols))


def _scale_shape(dense_or_shape):
    shape = tuple(dense_or_shape.shape) if isinstance(dense_or_shape, torch.Tensor) else tuple(dense_or_shape)
    return (1,) + shape if len(shape) == 2 else shape


def scales_to_mma(dense: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense scale bytes [.., M, S] (uint8 or float8_e4m3fn) -> the tile
    layout, a flat uint8 tensor of mma_scale_bytes(B, M, S) bytes."""
    if not dense.is_contiguous():
        raise ValueError("dense scales must be contiguous")
    B, M, S = _scale_shape(dense)
    if out is None:
        out = torch.empty(mma_scale_bytes(B, M, S), dtype=torch.uint8, device=dense.device)
    check(lib.pwq_scales_to_mma(dense.data_ptr(), B, M, S, out.data_ptr(), _stream(dense)), "pwq_scales_to_mma")
    return out


def scales_from_mma(mma: torch.Tensor, shape, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The tile layout back to dense uint8 scale bytes of `shape` ([M, S] or [B, M, S])."""
    B, M, S = _scale_shape(shape)
    if out is None:
        out = torch.empty(tuple(shape), dtype=torch.uint8, device=mma.device)
    check(lib.pwq_scales_from_mma(mma.data_ptr(), B, M, S, out.data_ptr(), _stream(mma)), "pwq_scales_from_mma")
    return out


def mxfp8_quant_grouped_mma(xs: Sequence[torch.Tensor], out=None, scale=None):
    """mxfp8_quant_grouped with every tensor's UE8M0 scales written in the
    tensor-core tile layout.  Returns (codes list, flat uint8 scale arrays)."""
    xs = list(xs)
    if out is None:
        out = [torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device) for x in xs]
    if scale is None:
        scale = [torch.empty(mma_scale_bytes(*_scale_shape(x.shape[:-1] + (x.shape[-1] // 32,))), dtype=torch.uint8,
                             device=x.device) for x in xs]
    if xs:
        check(lib.mxfp8_quant_grouped_mma(len(xs), _desc_array(xs, "x"), _desc_array(out, "out"), _ptrs(scale),
                                          _stream(xs[0])), "mxfp8_quant_grouped_mma")
    return out, scale


def nvfp4_quant_grouped_mma(groups: Sequence[Sequence[torch.Tensor]], out=None, sb=None, global_scale=None):
    """nvfp4_quant_grouped with the E4M3 block scales written in the
    tensor-core tile layout (flat uint8 arrays, one per member)."""
    groups, flat, sizes = _groups(groups)
    dev = flat[0].device
    if out is None:
        out = [[torch.empty(x.shape[:-1] + (x.shape[-1] // 2,), dtype=torch.uint8, device=dev) for x in g]
               for g in groups]
    if sb is None:
        sb = [[torch.empty(mma_scale_bytes(*_scale_shape(x.shape[:-1] + (x.shape[-1] // 16,))), dtype=torch.uint8,
                           device=dev) for x in g] for g in groups]
    if global_scale is None:
        global_scale = [torch.empty(_batch(g[0]), dtype=torch.float32, device=dev) for g in groups]
    ax = _desc_array(flat, "x")
    ws_bytes = int(lib.nvfp4_workspace_size_grouped(len(groups), sizes, ax))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    check(lib.nvfp4_quant_grouped_mma(len(groups), sizes, ax,
                                      _desc_array([p for g in out for p in g], "out", packed=True),
                                      _ptrs([s for g in sb for s in g]), _ptrs(global_scale), ws.data_ptr(),
                                      ws.numel(), _stream(flat[0])), "nvfp4_quant_grouped_mma")
    return out, sb, global_scale


# ---------------------------------------------------------------- block-scaled products

def _on(t: torch.Tensor, f, *args):
    """f(*args) with t's device current."""
    index = t.device.index
    if torch.cuda.current_device() == index:
        return f(*args)
    with torch.cuda.device(index):
        return f(*args)


def _launch(t: torch.Tensor, name: str, *args):
    """Calls the library on t's device and its current stream (the library launches on the current device)."""
    status = _on(t, getattr(lib, name), *args, _raw_stream(t.device.index))
    if status:
        check(status, name)


def _same_device(first, *others):
    dev = first.device
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError("tensors on different devices: %s and %s" % (dev, t.device))


def _tile_bytes(B: int, rows: int, cols: int) -> int:
    """mma_scale_bytes without the call."""
    return B * -(-rows // 128) * -(-cols // 4) * 512


def _one_byte(t: torch.Tensor, n: int, name: str, layout: str) -> int:
    """Address of a contiguous one-byte tensor of n values."""
    if t.element_size() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous one-byte tensor of the %d bytes of the %s layout"
                         % (name, n, layout))
    return t.data_ptr()


def _floats(t: torch.Tensor, n: int, name: str) -> int:
    """Address of a contiguous float32 tensor of n values."""
    if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous float32 tensor of %d values" % (name, n))
    return t.data_ptr()


def _product_out(a, w, da, dw, out):
    """The output and its descriptor."""
    if a.dim() != w.dim():
        raise ValueError("a and w must both be 2-D or both 3-D, got %s and %s" % (tuple(a.shape), tuple(w.shape)))
    if out is None:
        # separate sizes: torch parses them 2 us faster than a shape
        out = torch.empty(*a.shape[:-1], w.shape[-2], dtype=torch.bfloat16, device=a.device)
        return out, _new_desc(out, da, dw.rows)
    _check_dtype(out, (torch.bfloat16,), "out")
    return out, _desc(out, "out")


def mxfp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """BF16 y = a w^T of MXFP8 operands: codes a [.., M, K] and w [.., N, K]
    (2-D or batched alike), UE8M0 scales in the tensor-core tile layout
    (mxfp8_quant_grouped_mma, scales_to_mma, rms_norm_mxfp8).  Block scales
    and products are exact, the sum is FP32, y is rounded once.  Code rows
    are 16-byte aligned; ``out`` may have any row stride.  No gradient: codes
    are not differentiable."""
    _check_dtype(a, _CODE_DTYPES, "a")
    _check_dtype(w, _CODE_DTYPES, "w")
    da, dw = _desc(a, "a"), _desc(w, "w")
    out, dy = _product_out(a, w, da, dw, out)
    _same_device(a, a_scale, w, w_scale, out)
    S = da.cols // 32
    _launch(a, "mxfp8_matmul", ctypes.byref(da), _one_byte(a_scale, _tile_bytes(da.batch, da.rows, S), "a_scale", "tile"),
            ctypes.byref(dw), _one_byte(w_scale, _tile_bytes(da.batch, dw.rows, S), "w_scale", "tile"),
            ctypes.byref(dy))
    return out


def nvfp4_matmul(a: torch.Tensor, a_sb: torch.Tensor, a_global_scale: torch.Tensor, w: torch.Tensor,
                 w_sb: torch.Tensor, w_global_scale: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """BF16 y = a w^T of NVFP4 operands (W4A4): packed codes a [.., M, K/2]
    and w [.., N, K/2], E4M3 block scales in the tensor-core tile layout
    (nvfp4_quant_grouped_mma, scales_to_mma, rms_norm_nvfp4), FP32 global
    scales [B].  K % 32 == 16 needs padded code rows: rms_norm_nvfp4 makes
    them, nvfp4_quant_grouped_mma writes them when given through its ``out``.
    As mxfp8_matmul otherwise."""
    _check_dtype(a, (torch.uint8,), "a")
    _check_dtype(w, (torch.uint8,), "w")
    da, dw = _desc(a, "a", True), _desc(w, "w", True)
    out, dy = _product_out(a, w, da, dw, out)
    _same_device(a, a_sb, a_global_scale, w, w_sb, w_global_scale, out)
    B, S = da.batch, da.cols // 16
    _launch(a, "nvfp4_matmul", ctypes.byref(da), _one_byte(a_sb, _tile_bytes(B, da.rows, S), "a_sb", "tile"),
            _floats(a_global_scale, B, "a_global_scale"), ctypes.byref(dw),
            _one_byte(w_sb, _tile_bytes(B, dw.rows, S), "w_sb", "tile"),
            _floats(w_global_scale, B, "w_global_scale"), ctypes.byref(dy))
    return out


# ---------------------------------------------------------------- residual RMS norm with a block-scaled output

def _norm_inputs(x, weight, residual, h):
    """Checks and descriptors shared by the norms: (x, residual and h descriptor references, x's descriptor, h)."""
    _check_dtype(x, (torch.bfloat16,), "x")
    _check_dtype(weight, (torch.bfloat16,), "weight")
    dx = _desc(x, "x")
    if weight.dim() != 1 or weight.shape[0] != dx.cols or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous 1-D tensor of %d values" % dx.cols)
    if residual is None:
        if h is not None:
            raise ValueError("h is an output of the residual form only")
        return ctypes.byref(dx), None, None, dx, x
    _check_dtype(residual, (torch.bfloat16,), "residual")
    if h is None:
        h = torch.empty(*x.shape, dtype=torch.bfloat16, device=x.device)
        dh = _new_desc(h, dx, dx.cols)
    else:
        _check_dtype(h, (torch.bfloat16,), "h")
        dh = _desc(h, "h")
    return ctypes.byref(dx), ctypes.byref(_desc(residual, "residual")), ctypes.byref(dh), dx, h


def rms_norm_mxfp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, mma: bool = True, out: Optional[torch.Tensor] = None,
                   scale: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None):
    """h = x + residual; y = h * rsqrt(mean(h^2) + eps) * weight; MXFP8 of y,
    in one launch (include/pwq.h).  x [.., M, D] BF16, weight [D] BF16.
    Returns (codes float8_e4m3fn [.., M, D], UE8M0 scales, h): scales in the
    tensor-core tile layout (mma=True, for mxfp8_matmul) or dense
    [.., M, D/32]; h is x itself without a residual, and ``h=residual``
    updates the residual in place."""
    px, pr, ph, dx, h = _norm_inputs(x, weight, residual, h)
    B, M, S = dx.batch, dx.rows, dx.cols // 32
    n = _tile_bytes(B, M, S) if mma else B * M * S
    if out is None:
        out = torch.empty(*x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        do = _new_desc(out, dx, dx.cols)
    else:
        _check_dtype(out, _CODE_DTYPES, "out")
        do = _desc(out, "out")
    if scale is None:
        scale = (torch.empty(n, dtype=torch.uint8, device=x.device) if mma else
                 torch.empty(*x.shape[:-1], S, dtype=torch.uint8, device=x.device))
    _same_device(x, weight, residual, out, scale, h)
    _launch(x, "rms_norm_mxfp8", px, pr, weight.data_ptr(), eps, ph, ctypes.byref(do),
            _one_byte(scale, n, "scale", "tile" if mma else "dense"), int(mma), None)
    return out, scale, h


def rms_norm_nvfp4(x: torch.Tensor, weight: torch.Tensor, amax: torch.Tensor,
                   residual: Optional[torch.Tensor] = None, eps: float = 1e-6, mma: bool = True,
                   out: Optional[torch.Tensor] = None, sb: Optional[torch.Tensor] = None,
                   global_scale: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None):
    """rms_norm_mxfp8 with NVFP4 output for a given activation amax (float32
    [B], an NVFP4ActivationObserver's).  Returns (packed codes uint8
    [.., M, D/2], block scales, global scales float32 [B], h); with mma=True
    the code rows are 16-byte aligned, as nvfp4_matmul reads them (D % 32 == 16
    gives rows padded by 8 bytes)."""
    px, pr, ph, dx, h = _norm_inputs(x, weight, residual, h)
    B, M, S = dx.batch, dx.rows, dx.cols // 16
    n = _tile_bytes(B, M, S) if mma else B * M * S
    dev = x.device
    if out is None:
        cols = dx.cols // 2
        # the product reads code rows that are 16-byte aligned: an odd number of 16-element blocks pads its rows
        wide = -(-cols // 16) * 16 if mma else cols
        out = torch.empty(*x.shape[:-1], wide, dtype=torch.uint8, device=dev)
        do = _new_desc(out, dx, dx.cols)
        if wide != cols:
            out = out[..., :cols]
    else:
        _check_dtype(out, (torch.uint8,), "out")
        do = _desc(out, "out", True)
    if sb is None:
        sb = (torch.empty(n, dtype=torch.uint8, device=dev) if mma else
              torch.empty(*x.shape[:-1], S, dtype=torch.float8_e4m3fn, device=dev))
    if global_scale is None:
        global_scale = torch.empty(B, dtype=torch.float32, device=dev)
    _same_device(x, weight, residual, amax, out, sb, global_scale, h)
    _launch(x, "rms_norm_nvfp4", px, pr, weight.data_ptr(), eps, _floats(amax, B, "amax"), ph,
            ctypes.byref(do), _one_byte(sb, n, "sb", "tile" if mma else "dense"), int(mma),
            _floats(global_scale, B, "global_scale"), None)
    return out, sb, global_scale, h


def rms_norm_fake_quant(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                        format: str = "mxfp8", amax: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        out: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None):
    """The norm with its output fake-quantised (BF16 values of the codes of
    rms_norm_mxfp8 / rms_norm_nvfp4), for quantisation-aware training.
    Returns (y, h, rstd float32 [.., M])."""
    if format not in ("mxfp8", "nvfp4"):
        raise ValueError("format must be 'mxfp8' or 'nvfp4', got %r" % (format,))
    if (format == "nvfp4") != (amax is not None):
        raise ValueError("amax is given exactly with format='nvfp4'")
    px, pr, ph, dx, h = _norm_inputs(x, weight, residual, h)
    if out is None:
        out = torch.empty(*x.shape, dtype=torch.bfloat16, device=x.device)
        do = _new_desc(out, dx, dx.cols)
    else:
        _check_dtype(out, (torch.bfloat16,), "out")
        do = _desc(out, "out")
    rstd = torch.empty(*x.shape[:-1], dtype=torch.float32, device=x.device)
    _same_device(x, weight, residual, amax, out, h)
    head = (px, pr, weight.data_ptr(), eps)
    tail = (ph, ctypes.byref(do), rstd.data_ptr())
    if format == "mxfp8":
        _launch(x, "rms_norm_mxfp8_fake_quant", *head, *tail)
    else:
        _launch(x, "rms_norm_nvfp4_fake_quant", *head, _floats(amax, dx.batch, "amax"), *tail)
    return out, h, rstd


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      dh: Optional[torch.Tensor] = None, dweight_dtype=torch.float32, need_dweight: bool = True,
                      out: Optional[torch.Tensor] = None):
    """Gradient of the residual RMS norm, straight through its quantiser:
    (dx, dweight) from dy (of the output), dh (of h, optional) and the
    forward's h and rstd.  dx is the gradient of x and of the residual;
    dweight [D] is float32 or bfloat16, or None when not needed."""
    if dweight_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dweight_dtype must be float32 or bfloat16")
    _check_dtype(dy, (torch.bfloat16,), "dy")
    if dh is not None:
        _check_dtype(dh, (torch.bfloat16,), "dh")
    px, _, _, dhh, _ = _norm_inputs(h, weight, None, None)
    if rstd.shape != h.shape[:-1]:
        raise ValueError("rstd must have shape %s" % (tuple(h.shape[:-1]),))
    if out is not None:
        _check_dtype(out, (torch.bfloat16,), "out")
    _floats(rstd, dhh.batch * dhh.rows, "rstd")
    _same_device(h, dy, weight, rstd, dh, out)
    return _norm_backward(dy, h, weight, rstd, dh, dweight_dtype if need_dweight else None, out)


def _norm_backward(dy, h, weight, rstd, dh, dweight_dtype, out=None):
    """rms_norm_backward of checked arguments (dweight_dtype None: no dweight)."""
    dev = h.device
    dhh = _desc(h, "h")
    ph = ctypes.byref(dhh)
    if out is None:
        out = torch.empty(*h.shape, dtype=torch.bfloat16, device=dev)
        do = _new_desc(out, dhh, dhh.cols)
    else:
        do = _desc(out, "out")
    dw = None
    pw = pws = None
    n = 0
    if dweight_dtype is not None:
        n = max(_on(h, lib.rms_norm_backward_workspace_size, ph), 256)      # depends on the device's SM count
        dw = torch.empty(h.shape[-1], dtype=dweight_dtype, device=dev)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        pw, pws = dw.data_ptr(), ws.data_ptr()
    _launch(h, "rms_norm_backward", ctypes.byref(_desc(dy, "dy")),
            ctypes.byref(_desc(dh, "dh")) if dh is not None else None, ph, weight.data_ptr(), rstd.data_ptr(),
            ctypes.byref(do), pw, int(dweight_dtype == torch.bfloat16), pws, n)
    return out, dw


class _RMSNormSTE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, format, amax, eps):
        y, h, rstd = rms_norm_fake_quant(x, weight, residual, format, amax, eps)
        ctx.save_for_backward(h, weight, rstd)
        ctx.set_materialize_grads(False)
        return (y, h) if residual is not None else y

    @staticmethod
    def backward(ctx, dy, dh=None):
        if torch.is_grad_enabled():     # create_graph: the gradient below records no graph
            raise RuntimeError("rms_norm_fake_quant_ste has no second derivative")
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        dx, dw = dh, None
        if dy is not None:
            h, weight, rstd = ctx.saved_tensors
            dx, dw = _norm_backward(_last_contiguous(dy), h, weight, rstd,
                                    _last_contiguous(dh) if dh is not None else None,
                                    torch.bfloat16 if need_w else None)
        return dx if need_x else None, dw, dx if need_r else None, None, None, None


def _last_contiguous(g):
    """A gradient in the layout the library reads: an expanded or transposed one is copied."""
    if g.is_contiguous() and g.data_ptr() % 16 == 0:
        return g
    st = g.stride()
    ok = g.data_ptr() % 16 == 0 and st[-1] == 1 and all(s % 8 == 0 and s > 0 for s in st[:-1]) and (
        st[-2] >= g.shape[-1]) and (g.dim() < 3 or st[0] >= g.shape[1] * st[1])
    return g if ok else g.clone(memory_format=torch.contiguous_format)


def rms_norm_fake_quant_ste(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                            format: str = "mxfp8", amax: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """rms_norm_fake_quant with its backward pass (the quantiser straight
    through, verl NVFP4 QAT article 2.3).  Returns (y, h); h is x itself
    without a residual.  No second derivative.  As with any operation of
    torch, a backward pass is captured into a graph only while no eager graph of
    the same leaves is alive (torch raises otherwise)."""
    if residual is None:
        return _RMSNormSTE.apply(x, weight, None, format, amax, eps), x
    return _RMSNormSTE.apply(x, weight, residual, format, amax, eps)


# ---------------------------------------------------------------- diagnostics

# ---------------------------------------------------------------- FP8 block-wise -> rollout formats

def _fp8_input(q, scale, name="q"):
    _check_dtype(q, _CODE_DTYPES, name)
    if not scale.is_contiguous() or scale.dtype != torch.float32:
        raise ValueError("scale must be a contiguous float32 tensor")


def fp8_block_requant(q: torch.Tensor, scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                      scale_out: Optional[torch.Tensor] = None, inplace: bool = False):
    """FP8 block-wise codes + tile scales -> the FP8 block-wise codes and
    scales of their dequantised BF16 values, in one pass (no BF16 tensor):
    fp8_block_quant(fp8_block_dequant(q, scale)).  inplace=True overwrites
    q and scale."""
    _fp8_input(q, scale)
    if out is None:
        out = q if inplace else torch.empty(q.shape, dtype=torch.float8_e4m3fn, device=q.device)
    if scale_out is None:
        scale_out = scale if inplace else torch.empty_like(scale)
    _check_dtype(out, _CODE_DTYPES, "out")
    dq, do = _desc(q, "q"), _desc(out, "out")
    check(lib.fp8_block_requant(ctypes.byref(dq), scale.data_ptr(), ctypes.byref(do), scale_out.data_ptr(),
                                _stream(q)), "fp8_block_requant")
    return out, scale_out


def fp8_block_requant_mxfp8(q: torch.Tensor, scale: torch.Tensor, out: Optional[torch.Tensor] = None,
                            scale_out: Optional[torch.Tensor] = None, inplace: bool = False):
    """FP8 block-wise -> MXFP8 in one pass: mxfp8_quant(fp8_block_dequant(q,
    scale)).  Returns (codes, UE8M0 bytes [.., M, N/32]); inplace=True
    writes the codes over q."""
    _fp8_input(q, scale)
    if out is None:
        out = q if inplace else torch.empty(q.shape, dtype=torch.float8_e4m3fn, device=q.device)
    if scale_out is None:
        scale_out = torch.empty(q.shape[:-1] + (q.shape[-1] // 32,), dtype=torch.uint8, device=q.device)
    _check_dtype(out, _CODE_DTYPES, "out")
    dq, do = _desc(q, "q"), _desc(out, "out")
    check(lib.fp8_block_requant_mxfp8(ctypes.byref(dq), scale.data_ptr(), ctypes.byref(do),
                                      scale_out.data_ptr(), _stream(q)), "fp8_block_requant_mxfp8")
    return out, scale_out


def fp8_block_requant_nvfp4(qs, scales, amax: Optional[torch.Tensor] = None, out=None, sb=None,
                            global_scale: Optional[torch.Tensor] = None):
    """A sibling group of FP8 block-wise members -> NVFP4 in one pass (amax
    over the dequantised members, then encode): nvfp4_quant of the
    dequantised group.  Returns (packed codes list, block scales list,
    global scales [B]) like nvfp4_quant; ``amax`` replaces the reduction."""
    single = isinstance(qs, torch.Tensor)
    qs = [qs] if single else list(qs)
    scales = [scales] if isinstance(scales, torch.Tensor) else list(scales)
    if not 1 <= len(qs) <= PWQ_MAX_SIBLINGS or len(scales) != len(qs):
        raise ValueError("1..%d members, one scale tensor each" % PWQ_MAX_SIBLINGS)
    for i, (q, s_) in enumerate(zip(qs, scales)):
        _fp8_input(q, s_, "q[%d]" % i)
    dev = qs[0].device
    B = _batch(qs[0])
    if out is None:
        out = [torch.empty(q.shape[:-1] + (q.shape[-1] // 2,), dtype=torch.uint8, device=dev) for q in qs]
    if sb is None:
        sb = [torch.empty(q.shape[:-1] + (q.shape[-1] // 16,), dtype=torch.float8_e4m3fn, device=dev) for q in qs]
    if global_scale is None:
        global_scale = torch.empty(B, dtype=torch.float32, device=dev)
    aq = _desc_array(qs, "q")
    ao = _desc_array(out, "out", packed=True)
    sp = (ctypes.c_void_p * len(qs))(*[t.data_ptr() for t in scales])
    sbp = (ctypes.c_void_p * len(qs))(*[t.data_ptr() for t in sb])
    ws = None
    if amax is None:
        n = int(lib.fp8_block_requant_nvfp4_workspace_size(len(qs), aq))
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    check(lib.fp8_block_requant_nvfp4(aq, sp, len(qs), ao, sbp, global_scale.data_ptr(),
                                      amax.data_ptr() if amax is not None else None,
                                      ws.data_ptr() if ws is not None else None,
                                      ws.numel() if ws is not None else 0, _stream(qs[0])),
          "fp8_block_requant_nvfp4")
    if single:
        return out[0], sb[0], global_scale
    return out, sb, global_scale


def fp8_block_requant_grouped(qs: Sequence[torch.Tensor], scales: Sequence[torch.Tensor], out=None,
                              scale_out=None, inplace: bool = False):
    """fp8_block_requant over a list of tensors in one launch per 16."""
    qs, scales = list(qs), list(scales)
    for i, (q, s_) in enumerate(zip(qs, scales)):
        _fp8_input(q, s_, "q[%d]" % i)
    if out is None:
        out = qs if inplace else [torch.empty(q.shape, dtype=torch.float8_e4m3fn, device=q.device) for q in qs]
    if scale_out is None:
        scale_out = scales if inplace else [torch.empty_like(s_) for s_ in scales]
    check(lib.fp8_block_requant_grouped(len(qs), _desc_array(qs, "q"), _ptrs(scales), _desc_array(out, "out"),
                                        _ptrs(scale_out), _stream(qs[0])), "fp8_block_requant_grouped")
    return out, scale_out


def fp8_block_requant_mxfp8_grouped(qs: Sequence[torch.Tensor], scales: Sequence[torch.Tensor], out=None,
                                    scale_out=None, inplace: bool = False):
    """fp8_block_requant_mxfp8 over a list of tensors in one launch per 16."""
    qs, scales = list(qs), list(scales)
    for i, (q, s_) in enumerate(zip(qs, scales)):
        _fp8_input(q, s_, "q[%d]" % i)
    if out is None:
        out = qs if inplace else [torch.empty(q.shape, dtype=torch.float8_e4m3fn, device=q.device) for q in qs]
    if scale_out is None:
        scale_out = [torch.empty(q.shape[:-1] + (q.shape[-1] // 32,), dtype=torch.uint8, device=q.device)
                     for q in qs]
    check(lib.fp8_block_requant_mxfp8_grouped(len(qs), _desc_array(qs, "q"), _ptrs(scales),
                                              _desc_array(out, "out"), _ptrs(scale_out), _stream(qs[0])),
          "fp8_block_requant_mxfp8_grouped")
    return out, scale_out


def fp8_block_requant_nvfp4_grouped(groups, scales, out=None, sb=None, global_scale=None):
    """Several sibling groups of FP8 block-wise members (codes; `scales`
    mirrors `groups` with their tile scales) -> NVFP4 in one single-pass
    launch.  Returns (packed codes per group, block scales per group, global
    scales per group)."""
    groups = [list(g) for g in groups]
    scales = [list(g) for g in scales]
    if [len(g) for g in groups] != [len(g) for g in scales]:
        raise ValueError("scales must mirror groups")
    for gi, g in enumerate(groups):
        if not 1 <= len(g) <= PWQ_MAX_SIBLINGS:
            raise ValueError("1..%d members per group" % PWQ_MAX_SIBLINGS)
        for i, (q, s_) in enumerate(zip(g, scales[gi])):
            _fp8_input(q, s_, "groups[%d][%d]" % (gi, i))
    flat = [q for g in groups for q in g]
    sizes = (ctypes.c_int * len(groups))(*[len(g) for g in groups])
    dev = flat[0].device
    if out is None:
        out = [[torch.empty(q.shape[:-1] + (q.shape[-1] // 2,), dtype=torch.uint8, device=dev) for q in g]
               for g in groups]
    if sb is None:
        sb = [[torch.empty(q.shape[:-1] + (q.shape[-1] // 16,), dtype=torch.float8_e4m3fn, device=dev) for q in g]
              for g in groups]
    if global_scale is None:
        global_scale = [torch.empty(_batch(g[0]), dtype=torch.float32, device=dev) for g in groups]
    aq = _desc_array(flat, "q")
    ws_bytes = int(lib.fp8_block_requant_nvfp4_workspace_size_grouped(len(groups), sizes, aq))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    check(lib.fp8_block_requant_nvfp4_grouped(len(groups), sizes, aq, _ptrs([t for g in scales for t in g]),
                                              _desc_array([p_ for g in out for p_ in g], "out", packed=True),
                                              _ptrs([t for g in sb for t in g]), _ptrs(global_scale),
                                              ws.data_ptr(), ws.numel(), _stream(flat[0])),
          "fp8_block_requant_nvfp4_grouped")
    return out, sb, global_scale


# ---------------------------------------------------------------- W4A4 activation observers

OBSERVERS = {"memoryless_minmax": 0, "static_minmax": 1, "minmax": 2}


class NVFP4ActivationObserver:
    """An activation observer of W4A4 NVFP4 fake-quantisation (verl NVFP4 QAT
    article 2.2 / 3.1): keeps the running extremes (lo, hi) of the activations
    it sees on the device and gives the activation's amax and
    input_global_scale = fl(amax / 2688).  kind: "static_minmax" (default),
    "memoryless_minmax" or "minmax" (moving average with constant
    `averaging_constant`); the exact rules are those of nvfp4_activation_observe
    in include/pwq.h.  No host synchronisation."""

    def __init__(self, kind: str = "static_minmax", averaging_constant: float = 0.01, device="cuda"):
        if kind not in OBSERVERS:
            raise ValueError("observer kind must be one of %s" % sorted(OBSERVERS))
        self.kind = kind
        self.averaging_constant = float(averaging_constant)
        self.state = torch.tensor([float("inf"), float("-inf")], dtype=torch.float32, device=device)
        self.amax = torch.zeros(1, dtype=torch.float32, device=device)
        self.input_global_scale = torch.zeros(1, dtype=torch.float32, device=device)
        self._ws = torch.empty(int(lib.nvfp4_observe_workspace_size()), dtype=torch.uint8, device=device)

    def reset(self):
        self.state.copy_(torch.tensor([float("inf"), float("-inf")], dtype=torch.float32))

    def observe(self, x: torch.Tensor) -> torch.Tensor:
        """One observer step over x (BF16, last dim % 16 == 0); returns the
        amax tensor (float32 [1], on the device)."""
        _check_dtype(x, (torch.bfloat16,), "x")
        dx = _desc(x, "x")
        check(lib.nvfp4_activation_observe(ctypes.byref(dx), OBSERVERS[self.kind], self.averaging_constant,
                                           self.state.data_ptr(), self.amax.data_ptr(),
                                           self.input_global_scale.data_ptr(), self._ws.data_ptr(),
                                           self._ws.numel(), _stream(x)), "nvfp4_activation_observe")
        return self.amax

    def fake_quant(self, x: torch.Tensor, out=None) -> torch.Tensor:
        """Observe x, then NVFP4 fake-quantise it with the observed amax (one
        global scale for the whole tensor: a 3-D x gets the amax once per
        batch index, as nvfp4_fake_quant expects amax[B])."""
        amax = self.observe(x)
        if x.dim() == 3 and x.shape[0] != 1:
            amax = amax.expand(x.shape[0]).contiguous()
        return nvfp4_fake_quant(x, amax=amax, out=out)


class _W4A4STE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, observer):
        return observer.fake_quant(x)

    @staticmethod
    def backward(ctx, grad_out):
        return grad_out, None


def nvfp4_w4a4_fake_quant_ste(x: torch.Tensor, observer: NVFP4ActivationObserver) -> torch.Tensor:
    """W4A4 activation fake-quantisation with the straight-through backward
    (the gradient passes unchanged, verl NVFP4 QAT article 2.3)."""
    return _W4A4STE.apply(x, observer)


def build_info() -> str:
    return lib.pwq_build_info().decode()


def device_error() -> int:
    """Reads and clears the device-side error word (synchronous)."""
    code = ctypes.c_uint32(0)
    check(lib.pwq_device_error(ctypes.byref(code)), "pwq_device_error")
    return int(code.value)
