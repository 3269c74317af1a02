"""Low-rank adapters of many requests beside a shared projection (lora_apply in
include/groupmm.h): the projection is any product of this package, on its quantized weight;
the adapters stay in 16 bits, one set of them for all requests of a batch."""

from __future__ import annotations

import functools

import torch

from . import binding, groups, mx4
from .binding import _need


@functools.lru_cache(maxsize=1024)
def workspace_bytes(M: int, K: int, S: int, R: int) -> int:
    return int(groups.lib().lora_workspace_bytes(M, K, S, R))


def _need_adapters(t: torch.Tensor, dims: str, X: torch.Tensor, name: str) -> None:
    _need(t, X.dtype, name)
    if t.dim() != 3 or t.device != X.device:
        raise ValueError(f"{name} must be [{dims}] on {X.device}, got {tuple(t.shape)} on {t.device}")


def apply(Y: torch.Tensor, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor,
          scales: torch.Tensor | None = None, ranks: torch.Tensor | None = None,
          workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """out [M, N] = Y + scales[a] (X A_a^T) B_a^T with a = ids[m] for each row m, in X's type (fp16
    or bf16); rows whose id is no adapter (say -1) keep Y.

    Y [M, N] is the shared projection of X [M, K] (K and N multiples of 16, rows contiguous, any
    row stride of a multiple of 8). A [S, R, K] and B [S, N, R] hold S adapters of R ranks (a multiple of 8, at most 128);
    ids int32 [M] in any order; scales fp32 [S]; ranks int32 [S]: an adapter's own rank, what A
    and B hold beyond it is not looked at. out=Y adds in place.

    For inference: there is no backward, so a call that autograd would have to record (one of its
    tensors requires a gradient, outside torch.no_grad() and inference_mode()) is refused.
    """
    M, K, ldx, dt = mx4._need_rows(X, "X")
    my, N, ldy, dty = mx4._need_rows(Y, "Y")
    if my != M or dty != dt or Y.get_device() != X.get_device():
        raise ValueError(f"Y must be {X.dtype} with {M} rows on {X.device}, got {Y.dtype} {tuple(Y.shape)} on {Y.device}")
    _need_adapters(A, "S, R, K", X, "A")
    _need_adapters(B, "S, N, R", X, "B")
    S, R = A.shape[:2]
    if A.shape[2] != K or B.shape != (S, N, R):
        raise ValueError(f"A must be [S, R, {K}] and B [S, {N}, R], got {tuple(A.shape)} and {tuple(B.shape)}")
    groups.need_vector(ids, torch.int32, (M,), X, "ids")
    if scales is not None:
        groups.need_vector(scales, torch.float32, (S,), X, "scales")
    if ranks is not None:
        groups.need_vector(ranks, torch.int32, (S,), X, "ranks")
    if out is None:
        out, ldo = X.new_empty((M, N)), N
    else:
        mo, no, ldo, dto = mx4._need_rows(out, "out")
        if (mo, no, dto) != (M, N, dt) or out.get_device() != X.get_device():
            raise ValueError(f"out must be {X.dtype} [{M}, {N}] on {X.device}, got {out.dtype} {tuple(out.shape)} on "
                             f"{out.device}")
    if ((Y.requires_grad or X.requires_grad or A.requires_grad or B.requires_grad or out.requires_grad
         or (scales is not None and scales.requires_grad)) and torch.is_grad_enabled()):
        raise ValueError("lora.apply has no backward: call it under torch.no_grad(), or with detached tensors")
    nbytes = workspace_bytes(M, K, S, R)
    if nbytes == 0:
        raise ValueError(f"bad shape for lora.apply: M={M} K={K} S={S} R={R}")
    workspace = mx4._scratch(workspace, nbytes, X)
    groups.launch("lora_apply", X, Y.data_ptr(), ldy, X.data_ptr(), M, K, ldx, dt, A.data_ptr(), B.data_ptr(), S, R, N,
                  ids.data_ptr(), 0 if scales is None else scales.data_ptr(),
                  0 if ranks is None else ranks.data_ptr(), out.data_ptr(), ldo, workspace.data_ptr(), workspace.numel())
    return out
