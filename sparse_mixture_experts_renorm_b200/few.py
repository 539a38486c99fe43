"""The layer for a few tokens in two kernels: ``moe_forward_few`` (include/moe.h
has the definition)."""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _binding as B
from ._call import check, cuda, dtype_code, need, on, record

_args = record(22)


@dataclass(slots=True)
class FewOutputs:
    out: torch.Tensor  # [T, d] in x's dtype
    topk_idx: torch.Tensor  # [T, k] int32
    topk_gate: torch.Tensor  # [T, k] fp32
    workspace: torch.Tensor  # uint8
    counts: torch.Tensor | None = None  # [E] int32, when given
    aux: torch.Tensor | None = None  # [1] fp32, when given
    given_status: torch.Tensor | None = None

    @property
    def status(self) -> torch.Tensor:
        """[1] int32, MOE_DEV_* bits: the word that was given, into which this call OR-ed its own, or this call's
        alone, the workspace's first four bytes (until the next call with this workspace)."""
        return self.workspace[:4].view(torch.int32) if self.given_status is None else self.given_status


def few_workspace_size(T: int, d: int, E: int, k: int, I: int, dtype: torch.dtype) -> int:
    """Bytes of scratch of ``moe_forward_few``."""
    lib = B.load_library()
    n = lib.moe_few_workspace_size(T, d, E, k, I, dtype_code(dtype))
    if n == 0:
        raise B.MoEError(B.MOE_ERR_INVALID_ARG, B.last_error_detail(lib))
    return int(n)


def moe_forward_few(x, w_router, b_router, w_gate, w_up, w_down, k: int, renorm: bool, *, out=None, topk_idx=None,
                    topk_gate=None, counts=None, aux=None, workspace=None, status=None, stream=None) -> FewOutputs:
    """``moe_forward`` for ``x`` of at most 16 tokens ([T, d], bf16 or fp32), in
    two kernels, with the output in x's dtype. ``counts`` ([E] int32) and
    ``aux`` ([1] fp32) are filled when given. ``workspace``: uint8,
    ``few_workspace_size`` bytes, one for each call that may run at the same
    time (default: a new one). ``status``: [1] int32, into which the call's bits
    are OR-ed; without it the call's word is the workspace's first four bytes
    (cleared by the call)."""
    dev = cuda("x", x)
    dt = x.dtype
    code = dtype_code(dt)
    if x.dim() != 2 or not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 3:
        raise ValueError("x must be [T, d] and w_gate [E, I, d]")
    T, d = x.shape
    E, I, _ = w_gate.shape
    need("x", x, dt, (T, d), dev)
    need("w_router", w_router, dt, (E, d), dev)
    need("w_gate", w_gate, dt, (E, I, d), dev)
    need("w_up", w_up, dt, (E, I, d), dev)
    need("w_down", w_down, dt, (E, d, I), dev)
    if b_router is not None:
        need("b_router", b_router, torch.float32, (E,), dev)
    if counts is not None:
        need("counts", counts, torch.int32, (E,), dev)
    if aux is not None:
        need("aux", aux, torch.float32, (1,), dev)
    if status is not None:
        need("status", status, torch.int32, (1,), dev)
    lib = B.load_library()
    with on(dev, stream) as s:
        if workspace is None:
            workspace = torch.empty((few_workspace_size(T, d, E, k, I, dt),), dtype=torch.uint8, device=dev)
        else:
            need("workspace", workspace, torch.uint8, None, dev)
        if out is None:
            out = torch.empty_like(x)
        else:
            need("out", out, dt, (T, d), dev)
        if topk_idx is None:
            topk_idx = torch.empty_strided((T, k), (k, 1), dtype=torch.int32, device=dev)
        else:
            need("topk_idx", topk_idx, torch.int32, (T, k), dev)
        if topk_gate is None:
            topk_gate = torch.empty_strided((T, k), (k, 1), dtype=torch.float32, device=dev)
        else:
            need("topk_gate", topk_gate, torch.float32, (T, k), dev)
        check(lib.moe_bind_forward_few(_args(
            x.data_ptr(), w_router.data_ptr(), 0 if b_router is None else b_router.data_ptr(), w_gate.data_ptr(),
            w_up.data_ptr(), w_down.data_ptr(), T, d, E, k, I, 1 if renorm else 0, code, out.data_ptr(),
            topk_idx.data_ptr(), topk_gate.data_ptr(), 0 if counts is None else counts.data_ptr(),
            0 if aux is None else aux.data_ptr(), workspace.data_ptr(), workspace.numel(),
            workspace.data_ptr() if status is None else status.data_ptr(), s)), lib)
    return FewOutputs(out, topk_idx, topk_gate, workspace, counts, aux, status)
