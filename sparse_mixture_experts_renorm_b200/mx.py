"""MXFP4 (microscaled 4-bit) matrices and the layer with its experts in them:
``mx_quantize`` / ``mx_dequantize``, ``mx_matmul``, ``mx_experts`` and
``moe_forward_mx`` (``moe_mx_*`` in include/moe.h, which has the formulas)."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _binding as B
from ._call import check, cuda, device_status, dtype_code, need, on, ptr, record

_BYTE = torch.uint8
_args10, _args13, _args21 = record(10), record(13), record(21)


@dataclass(slots=True)
class MXTensor:
    """An MXFP4 matrix or stack of matrices: ``data`` [rows, cols / 2] or
    [groups, rows, cols / 2] uint8 (two E2M1 codes a byte, the even column in
    the low half) and ``scales``, the E8M0 bytes in the library's tiles
    (include/moe.h has the layout; ``mx_scale_bytes`` of them)."""
    data: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return torch.Size((*self.data.shape[:-1], 2 * self.data.shape[-1]))

    @property
    def device(self):
        return self.data.device


def mx_scale_bytes(groups: int, rows: int, cols: int, ragged: bool = False) -> int:
    """Bytes of scales of ``groups`` groups of ``rows`` rows each, or (ragged)
    of ``rows`` rows in ``groups`` groups of any lengths."""
    lib = B.load_library()
    n = lib.moe_mx_scale_bytes(groups, rows, cols, int(ragged))
    if n == 0:
        raise B.MoEError(B.MOE_ERR_INVALID_ARG, B.last_error_detail(lib))
    return int(n)


def _need_scales(groups, rows, cols, ragged=False):
    """``mx_scale_bytes`` of a valid matrix, without a call into the library
    (which checks the sizes again): include/moe.h has the layout."""
    tiles = rows // 256 + min(rows, groups) if ragged else groups * ((rows + 255) // 256)
    return max(tiles, 1) * 2048 * ((cols + 255) // 256)


def _offsets(offsets, dev):
    """(pointer, groups) of ragged groups; offsets [groups + 1] int32."""
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be a one-dimensional int32 tensor of groups + 1 row numbers")
    need("offsets", offsets, torch.int32, None, dev)
    return offsets.data_ptr(), offsets.numel() - 1


def _check_mx(name, q, dev):
    if not isinstance(q, MXTensor):
        raise TypeError(f"{name} must be an MXTensor")
    if not isinstance(q.data, torch.Tensor) or not isinstance(q.scales, torch.Tensor):
        raise TypeError(f"{name}.data and {name}.scales must be tensors")
    if q.data.dim() not in (2, 3):
        raise ValueError(f"{name}.data must be [rows, cols / 2] or [groups, rows, cols / 2]")
    for t in (q.data, q.scales):
        if t.dtype is not _BYTE or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name}.data and {name}.scales must be contiguous uint8 tensors on {dev}")


def mx_quantize(x, offsets=None, *, stream=None) -> MXTensor:
    """``x`` ([rows, cols] or [groups, rows, cols], bf16 or fp32, contiguous,
    cols % 32 == 0) in MXFP4. With ``offsets`` ([groups + 1] int32 on the
    device, ``x`` [rows, cols]) group g is rows offsets[g] .. offsets[g + 1] - 1;
    rows of no group get no codes."""
    dev = cuda("x", x)
    if x.dim() not in (2, 3) or (offsets is not None and x.dim() != 2):
        raise ValueError("x must be [rows, cols], or [groups, rows, cols] without offsets")
    dt = dtype_code(x.dtype)
    need("x", x, x.dtype, None, dev)
    lib = B.load_library()
    rows, cols = x.shape[-2], x.shape[-1]
    off, groups = _offsets(offsets, dev) if offsets is not None else (0, x.shape[0] if x.dim() == 3 else 1)
    with on(dev, stream) as s:
        if cols <= 0 or cols % 32 or groups <= 0:
            mx_scale_bytes(groups, rows, cols, offsets is not None)  # raises, with the reason
        n = _need_scales(groups, rows, cols, offsets is not None)
        data = x.new_empty((*x.shape[:-1], cols // 2), dtype=_BYTE)
        scales = torch.empty_strided((n,), (1,), dtype=_BYTE, device=dev)
        check(lib.moe_bind_mx_quantize(_args10(x.data_ptr(), off, groups, rows, cols, dt, data.data_ptr(),
                                               scales.data_ptr(), n, s)), lib)
    return MXTensor(data, scales)


def mx_dequantize(q: MXTensor, dtype=torch.bfloat16, offsets=None, *, out=None, stream=None) -> torch.Tensor:
    """The values of ``q`` in ``dtype`` (bf16 or fp32: exact in both, infinite
    from 2^128 on, which only scales that ``mx_quantize`` does not write reach). With
    ``offsets`` as given to ``mx_quantize``; rows of no group are left as they
    are in ``out`` (unset in a new one)."""
    if not isinstance(q, MXTensor):
        raise TypeError("q must be an MXTensor")
    dev = cuda("q.data", q.data)
    _check_mx("q", q, dev)
    dt = dtype_code(dtype)
    shape = q.data.shape
    if offsets is not None and len(shape) != 2:
        raise ValueError("a matrix with offsets is [rows, cols]")
    lib = B.load_library()
    rows, cols = shape[-2], 2 * shape[-1]
    shape = (*shape[:-1], cols)
    off, groups = _offsets(offsets, dev) if offsets is not None else (0, shape[0] if len(shape) == 3 else 1)
    with on(dev, stream) as s:
        if out is None:
            out = q.data.new_empty(shape, dtype=dtype)
        else:
            need("out", out, dtype, shape, dev)
        check(lib.moe_bind_mx_dequantize(_args10(q.data.data_ptr(), q.scales.data_ptr(), q.scales.numel(), off, groups,
                                                 rows, cols, dt, out.data_ptr(), s)), lib)
    return out


def mx_matmul(a: MXTensor, b: MXTensor, offsets=None, *, out_dtype=torch.bfloat16, out=None, status=None,
              stream=None) -> torch.Tensor:
    """out[r] = a[r] @ b[g].T for the rows r of every group g: ``a`` [M, K] with
    ``offsets`` [groups + 1] (and quantised with them), or [M, K] / [groups, M,
    K] without; ``b`` [N, K] or [groups, N, K], N % 8 == 0. The result is [M, N]
    or [groups, M, N] in ``out_dtype`` (bf16 or fp32); rows of no group are left
    as they are. ``status``: [1] int32, MOE_DEV_* bits are OR-ed in (default:
    ``device_status``, one word for all such calls on the device)."""
    if not isinstance(a, MXTensor):
        raise TypeError("a must be an MXTensor")
    dev = cuda("a.data", a.data)
    _check_mx("a", a, dev)
    _check_mx("b", b, dev)
    dt = dtype_code(out_dtype)
    sa, sb = a.data.shape, b.data.shape
    groups = sb[0] if len(sb) == 3 else 1
    N, K = sb[-2], 2 * sb[-1]
    M = sa[-2]
    off = 0
    if offsets is not None:
        off, n = _offsets(offsets, dev)
        if len(sa) != 2 or n != groups:
            raise ValueError(f"with offsets a is [M, K] and there are as many groups as in b ({groups})")
    elif (sa[0] if len(sa) == 3 else 1) != groups:
        raise ValueError("without offsets a and b have the same number of groups")
    if 2 * sa[-1] != K:
        raise ValueError(f"a has {2 * sa[-1]} columns and b {K}")
    lib = B.load_library()
    for name, q, g, rows, ragged in (("a", a, groups, M, offsets is not None), ("b", b, groups, N, False)):
        if q.scales.numel() < _need_scales(g, rows, K, ragged):
            raise ValueError(f"{name}.scales holds {q.scales.numel()} bytes, "
                             f"{_need_scales(g, rows, K, ragged)} are needed")
    if status is not None:
        need("status", status, torch.int32, (1,), dev)
    shape = (*sa[:-1], N)
    with on(dev, stream) as s:
        if status is None:
            status = device_status(dev)
        if out is None:
            out = a.data.new_empty(shape, dtype=out_dtype)
        else:
            need("out", out, out_dtype, shape, dev)
        check(lib.moe_bind_mx_matmul(_args13(a.data.data_ptr(), a.scales.data_ptr(), b.data.data_ptr(),
                                             b.scales.data_ptr(), off, groups, M, N, K, dt, out.data_ptr(),
                                             status.data_ptr(), s)), lib)
    return out


@dataclass(slots=True)
class MXOutputs:
    out: torch.Tensor  # [T, d] bf16
    counts: torch.Tensor  # [E] int32
    status: torch.Tensor  # [1] int32, MOE_DEV_* bits of this call
    workspace: torch.Tensor  # uint8
    topk_idx: torch.Tensor | None = None  # [T, k] int32 (moe_forward_mx)
    topk_gate: torch.Tensor | None = None  # [T, k] fp32 (moe_forward_mx)
    aux: torch.Tensor | None = None  # [1] fp32 (moe_forward_mx)


def mx_workspace_size(T: int, d: int, E: int, k: int, I: int) -> int:
    """Bytes of scratch of ``mx_experts`` and ``moe_forward_mx``."""
    lib = B.load_library()
    n = lib.moe_mx_workspace_size(T, d, E, k, I)
    if n == 0:
        raise B.MoEError(B.MOE_ERR_INVALID_ARG, B.last_error_detail(lib))
    return int(n)


def _weights(w_gate, w_up, w_down, dev, d):
    for name, q in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _check_mx(name, q, dev)
        if q.data.dim() != 3:
            raise ValueError(f"{name} must be [E, rows, cols]")
    E, I, _ = w_gate.data.shape
    n_up, n_down = _need_scales(E, I, d), _need_scales(E, d, I)
    for name, q, shape, n in (("w_gate", w_gate, (E, I, d), n_up), ("w_up", w_up, (E, I, d), n_up),
                              ("w_down", w_down, (E, d, I), n_down)):
        got = q.data.shape
        if got[0] != shape[0] or got[1] != shape[1] or 2 * got[2] != shape[2]:
            raise ValueError(f"{name} must have the shape {shape} (got {tuple(q.shape)})")
        if q.scales.numel() < n:
            raise ValueError(f"{name}.scales holds {q.scales.numel()} bytes, {n} are needed")
    return (w_gate.data.data_ptr(), w_gate.scales.data_ptr(), w_up.data.data_ptr(), w_up.scales.data_ptr(),
            w_down.data.data_ptr(), w_down.scales.data_ptr()), E, I


def _buffers(x, T, d, E, k, I, out, counts, workspace, status):
    dev = x.device
    if out is None:
        out = x.new_empty((T, d), dtype=torch.bfloat16)
    else:
        need("out", out, torch.bfloat16, (T, d), dev)
    if counts is None:
        counts = x.new_empty((E,), dtype=torch.int32)
    else:
        need("counts", counts, torch.int32, (E,), dev)
    if workspace is None:
        workspace = x.new_empty((mx_workspace_size(T, d, E, k, I),), dtype=_BYTE)
    else:  # its size is checked by the call
        need("workspace", workspace, _BYTE, None, dev)
    if status is not None:
        need("status", status, torch.int32, (1,), dev)
    return out, counts, workspace


def _status_of(status, workspace):
    """The call's own status word is the workspace's first four bytes."""
    return workspace[:4].view(torch.int32) if status is None else status


def _rows(x):
    dev = cuda("x", x)
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    dt = dtype_code(x.dtype)
    need("x", x, x.dtype, None, dev)
    return dev, dt


def mx_experts(x, topk_idx, topk_gate, w_gate: MXTensor, w_up: MXTensor, w_down: MXTensor, *, out=None, counts=None,
               workspace=None, status=None, stream=None) -> MXOutputs:
    """The layer's experts in MXFP4 for given choices: ``x`` [T, d] (bf16 or
    fp32), ``topk_idx`` [T, k] int32, ``topk_gate`` [T, k] fp32, weights
    [E, I, d], [E, I, d] and [E, d, I]. out[t] = sum_j gate[t, j] y of expert
    idx[t, j], bf16. ``workspace``: uint8, ``mx_workspace_size`` bytes, one for
    each call that may run at the same time. Without ``status`` the call's word
    is the workspace's first four bytes (cleared by the call). x and the hidden
    rows are rounded to MXFP4 too: on normal data ``out`` is 0.30 of its norm
    off, of which the weights alone would make 0.20 (include/moe.h)."""
    dev, dt = _rows(x)
    T, d = x.shape
    w, E, I = _weights(w_gate, w_up, w_down, dev, d)
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be a [T, k] tensor")
    k = topk_idx.shape[1]
    need("topk_idx", topk_idx, torch.int32, (T, k), dev)
    need("topk_gate", topk_gate, torch.float32, (T, k), dev)
    lib = B.load_library()
    with on(dev, stream) as s:
        out, counts, workspace = _buffers(x, T, d, E, k, I, out, counts, workspace, status)
        check(lib.moe_bind_mx_experts(_args21(
            x.data_ptr(), topk_idx.data_ptr(), topk_gate.data_ptr(), *w, T, d, E, k, I, dt, out.data_ptr(),
            counts.data_ptr(), workspace.data_ptr(), workspace.numel(), 0 if status is None else status.data_ptr(),
            s)), lib)
        status = _status_of(status, workspace)
    return MXOutputs(out, counts, status, workspace)


def moe_forward_mx(x, w_router, b_router, w_gate: MXTensor, w_up: MXTensor, w_down: MXTensor, k: int, renorm: bool, *,
                   out=None, topk_idx=None, topk_gate=None, counts=None, aux=None, workspace=None, status=None,
                   stream=None) -> MXOutputs:
    """``moe_forward`` with the experts in MXFP4: the router runs on ``x`` and
    ``w_router`` [E, d] as they are (one dtype, bf16 or fp32; ``b_router`` [E]
    fp32 or None), then ``mx_experts`` on its choices."""
    dev, dt = _rows(x)
    T, d = x.shape
    w, E, I = _weights(w_gate, w_up, w_down, dev, d)
    need("w_router", w_router, x.dtype, (E, d), dev)
    if b_router is not None:
        need("b_router", b_router, torch.float32, (E,), dev)
    lib = B.load_library()
    with on(dev, stream) as s:
        out, counts, workspace = _buffers(x, T, d, E, k, I, out, counts, workspace, status)
        if topk_idx is None:
            topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        if topk_gate is None:
            topk_gate = torch.empty((T, k), dtype=torch.float32, device=dev)
        if aux is None:
            aux = torch.empty((1,), dtype=torch.float32, device=dev)
        need("topk_idx", topk_idx, torch.int32, (T, k), dev)
        need("topk_gate", topk_gate, torch.float32, (T, k), dev)
        need("aux", aux, torch.float32, (1,), dev)
        weights = B.moe_mx_weights(ctypes.sizeof(B.moe_mx_weights), *w)
        check(lib.moe_mx_forward(ptr(x), ptr(w_router), ptr(b_router), ctypes.byref(weights), T, d, E, k, I,
                                 int(bool(renorm)), dt, ptr(out), ptr(topk_idx), ptr(topk_gate), ptr(counts),
                                 ptr(aux), ptr(workspace), workspace.numel(), ptr(status), s), lib)
        status = _status_of(status, workspace)
    return MXOutputs(out, counts, status, workspace, topk_idx, topk_gate, aux)
