"""A mixture-of-experts layer for a few tokens (moe_layer in include/mx4mm.h): routing, gate
and up products, SiLU, down product and the weighted sum over experts in two launches, with
expert weights in int8 (``binding.prepare_weight`` / ``tile_weight``) or MX4
(``mx4.prepare_weight`` / ``tile_weight``)."""

from __future__ import annotations

import functools

import torch

from . import binding, mx4
from .binding import _need_shape


@functools.lru_cache(maxsize=1024)
def workspace_bytes(T: int, I: int, top_k: int) -> int:
    return int(mx4.lib().moe_layer_workspace_bytes(T, I, top_k))


def _rows(pair, name: str) -> tuple[int, int]:
    """(weight format, output features) of a prepared weight pair."""
    codes, _ = pair
    shape = codes.shape if isinstance(codes, torch.Tensor) else ()
    if len(shape) != 4 or codes.dtype not in (torch.int8, torch.uint8):
        raise ValueError(f"{name} must be a prepared int8 or MX4 weight")
    return int(codes.dtype is torch.uint8), 16 * shape[0]


def _need_pair(pair, fmt: int, rows: int, K: int, like: torch.Tensor, name: str) -> None:
    codes, consts = pair
    if fmt:
        mx4._need_mx4(codes, consts, rows, K, like, name)
        return
    if (consts.dtype is torch.float32 and codes.is_contiguous() and consts.is_contiguous() and consts.numel() == rows
            and consts.dim() == 1 and codes.numel() == binding._prepared_bytes(K, rows) != 0
            and codes.get_device() == consts.get_device() == like.get_device()):
        return
    if binding._need_weight(codes, consts, K, like.device) != rows:
        raise ValueError(f"{name} has {pair[1].numel()} column constants for {rows} output features")


def moe_layer(X: torch.Tensor, logits: torch.Tensor, gate_up: tuple, down: tuple, top_k: int,
              renormalize: bool = True, workspace: torch.Tensor | None = None,
              out: torch.Tensor | None = None):
    """(Y [T, D] in X's type, ids int32 [T, top_k], weights fp32 [T, top_k]) for fp16 or bf16 X
    [T <= 16, D] and router logits [T, E] (fp16, bf16 or fp32; -inf: the expert is off).

    gate_up: one prepared weight of E * 2 I output features over D (per expert the I gate
    rows, then the I up rows); down: one of E * D output features over I; both in the same
    format. Lists are in descending order of the logits, ties to the lower index; past the
    last expert that is on, id is -1 and weight 0. renormalize: weights sum to 1 over the
    chosen experts, otherwise they are the softmax over all of them.

    More than 16 tokens: 16 at a time, or, for a prompt, each expert's tokens through ``mx4.matmul``
    or ``binding.mixed_matmul`` on its part of the prepared weights (of gate_up the row groups
    e * 2 I / 16 up to (e + 1) * 2 I / 16 of codes and scales; int8 constants by row).
    """
    T, D, ld, dt = mx4._need_rows(X, "X")
    if not isinstance(logits, torch.Tensor) or logits.dtype not in mx4.DTYPES or logits.dim() != 2:
        raise ValueError("logits must be a 2-D fp16, bf16 or fp32 tensor")
    rows, E = logits.shape
    if rows != T or not logits.is_contiguous() or logits.get_device() != X.get_device():
        _need_shape(logits, logits.dtype, (T, E), X.device, "logits")
    fmt, rows = _rows(gate_up, "gate_up")
    if _rows(down, "down")[0] != fmt:
        raise ValueError("gate_up and down must be in the same format")
    if E < 1 or rows % (32 * E):
        raise ValueError(f"gate_up has {rows} output features: not E = {E} times 2 I with I a multiple of 16")
    I = rows // (2 * E)
    _need_pair(gate_up, fmt, rows, D, X, "gate_up")
    _need_pair(down, fmt, E * D, I, X, "down")
    if out is None:
        out = X.new_empty((T, D))
    else:
        _need_shape(out, X.dtype, (T, D), X.device, "out")
    nbytes = workspace_bytes(T, I, top_k)
    if nbytes == 0:
        raise ValueError(f"bad shape for moe_layer: T={T} I={I} top_k={top_k}")
    workspace = mx4._scratch(workspace, nbytes, X)
    ids = X.new_empty((T, top_k), dtype=torch.int32)
    weights = X.new_empty((T, top_k), dtype=torch.float32)
    mx4._launch("moe_layer", X, X.data_ptr(), T, D, ld, dt, logits.data_ptr(), E, mx4.DTYPES[logits.dtype],
                top_k, int(renormalize), fmt, gate_up[0].data_ptr(), gate_up[1].data_ptr(), down[0].data_ptr(),
                down[1].data_ptr(), I, out.data_ptr(), ids.data_ptr(), weights.data_ptr(), workspace.data_ptr(),
                workspace.numel())
    return out, ids, weights
