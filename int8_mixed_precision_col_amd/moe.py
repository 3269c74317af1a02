"""A mixture-of-experts layer, with expert weights in int8 (``binding.prepare_weight`` /
``tile_weight``) or MX4 (``mx4.prepare_weight`` / ``tile_weight``).

For a few tokens ``moe_layer`` (include/mx4mm.h): routing, gate and up products, SiLU, down
product and the weighted sum over experts in two launches. For few or many tokens
``moe_prompt`` and its parts (include/groupmm.h): ``route``, ``grouped_matmul`` and ``combine``.
"""

from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from . import binding, groups, mx4
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

    More than 16 tokens: ``moe_prompt``, which quantizes the activations, or 16 at a time.
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


class Routing(NamedTuple):
    """What ``route`` gives: each token's experts and their weights, and the order of the rows of
    a product grouped by expert."""
    ids: torch.Tensor       # int32 [T, top_k], -1 past the last expert that is on
    weights: torch.Tensor   # fp32 [T, top_k]
    offsets: torch.Tensor   # int32 [E + 1]: expert e has rows offsets[e] up to offsets[e + 1]
    rows: torch.Tensor      # int32 [T * top_k]: the token of each row, -1 behind the last
    slots: torch.Tensor     # int32 [T, top_k]: the row of each token and place, -1 for none


@functools.lru_cache(maxsize=1024)
def _route_workspace_bytes(T: int, E: int) -> int:
    return int(groups.lib().moe_route_workspace_bytes(T, E))


def _outliers(K: int, max_outliers: int | None) -> int:
    """How many outlier columns a call makes room for."""
    most = min(K, 8192)
    return most if max_outliers is None else min(max_outliers, most)


@functools.lru_cache(maxsize=1024)
def grouped_workspace_bytes(M: int, K: int, P: int, E: int, N: int, weight_format: int,
                            max_outliers: int | None = None) -> int:
    """What ``grouped_matmul`` needs for X [M, K], P rows of the product and E experts of N features
    (0 on bad shapes); weight_format 0: int8, 1: MX4; max_outliers as given to the call."""
    return int(groups.lib().moe_grouped_workspace_bytes(M, K, P, E, N, weight_format, _outliers(K, max_outliers)))


def _need_logits(logits: torch.Tensor, top_k: int) -> tuple[int, int]:
    """(T, E) of what ``route`` takes."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in mx4.DTYPES or logits.dim() != 2:
        raise ValueError("logits must be a 2-D fp16, bf16 or fp32 tensor")
    T, E = logits.shape
    if not logits.is_contiguous() or not binding._on_device(logits):
        _need_shape(logits, logits.dtype, (T, E), logits.device, "logits")
    if not (1 <= top_k <= min(E, 16) and 1 <= T <= 1 << 24 and E <= 512):
        raise ValueError(f"bad shape for route: T={T} E={E} top_k={top_k}")
    return T, E


def _need_experts(weight: tuple, M: int, K: int, P: int, E: int, gated: bool, max_outliers: int | None,
                  X: torch.Tensor, name: str) -> tuple[int, int, int]:
    """(weight format, features per expert, bytes of workspace) of a product of [M, K] in X's type."""
    fmt, features = _rows(weight, name)
    step = 32 if gated else 16
    if features % (step * E):
        raise ValueError(f"{name} has {features} output features: not E = {E} times a multiple of {step}")
    N = features // E
    if not fmt and X.dtype is not torch.float16:
        raise ValueError("int8 weights take contiguous fp16 X")
    _need_pair(weight, fmt, features, K, X, name)
    nbytes = grouped_workspace_bytes(M, K, P, E, N, fmt, max_outliers)
    if nbytes == 0:
        raise ValueError(f"bad shape for a grouped product: M={M} K={K} P={P} E={E} N={N} max_outliers={max_outliers}")
    return fmt, N, nbytes


def _grouped(X: torch.Tensor, M: int, K: int, ld: int, dt: int, weight: tuple, experts: tuple, offsets: torch.Tensor,
             E: int, rows: torch.Tensor | None, P: int, gated: bool, threshold: float, max_outliers: int | None,
             workspace: torch.Tensor | None, out: torch.Tensor) -> torch.Tensor:
    """The launch of ``grouped_matmul``, its arguments checked; experts as from ``_need_experts``."""
    fmt, N, nbytes = experts
    workspace = mx4._scratch(workspace, nbytes, X)
    groups.launch("moe_grouped_matmul", X, X.data_ptr(), M, K, ld, dt, fmt, weight[0].data_ptr(),
                  weight[1].data_ptr(), E, N, offsets.data_ptr(), 0 if rows is None else rows.data_ptr(), P, int(gated),
                  float(threshold), _outliers(K, max_outliers), out.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out


def route(logits: torch.Tensor, top_k: int, renormalize: bool = True) -> Routing:
    """Routing of T tokens from their router logits [T, E] (fp16, bf16 or fp32; -inf: the expert is
    off; E <= 512, top_k <= 16): lists as in ``moe_layer``, and the pairs of token and expert in
    order of expert and then token. The same inputs give the same order."""
    T, E = _need_logits(logits, top_k)
    nbytes = _route_workspace_bytes(T, E)
    i32 = torch.int32
    r = Routing(logits.new_empty((T, top_k), dtype=i32), logits.new_empty((T, top_k), dtype=torch.float32),
                logits.new_empty((E + 1,), dtype=i32), logits.new_empty((T * top_k,), dtype=i32),
                logits.new_empty((T, top_k), dtype=i32))
    ws = mx4._scratch(None, nbytes, logits)
    groups.launch("moe_route", logits, logits.data_ptr(), T, E, mx4.DTYPES[logits.dtype], top_k, int(renormalize),
                  r.ids.data_ptr(), r.weights.data_ptr(), r.offsets.data_ptr(), r.rows.data_ptr(), r.slots.data_ptr(),
                  0 if ws is None else ws.data_ptr(), nbytes)
    return r


def grouped_matmul(X: torch.Tensor, weight: tuple, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                   gated: bool = False, threshold: float = 6.0, max_outliers: int | None = None,
                   workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Products grouped by expert with ragged sizes: row p of Y, offsets[e] <= p < offsets[e + 1],
    is the product of row rows[p] of X [M, K] (row p without rows) with expert e's part of `weight`,
    one prepared weight of E * N output features. Y is [P, N] in X's type, or, gated (N: gate
    features, then as many up features), silu(gate) * up [P, N / 2].

    MX4 weights: fp16 or bf16 X, rounded to MX4 as in ``mx4.matmul``. int8 weights: fp16 X,
    decomposed as in ``binding.mixed_matmul`` (outlier columns are those of the whole of X; more than
    max_outliers of them, without one any number up to 8192, give NaN). The workspace has room for
    max_outliers columns of X in fp16: give a smaller number where all of X is too much.
    offsets int32 [E + 1] ascending from 0 and rows int32 [P] are on the GPU and stay there
    (``route`` makes both). Rows of Y behind offsets[E] are zeros, and a row
    whose index is outside X counts as zeros.
    """
    M, K, ld, dt = mx4._need_rows(X, "X")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be an int32 tensor [E + 1]")
    E = offsets.shape[0] - 1
    groups.need_vector(offsets, torch.int32, (E + 1,), X, "offsets")
    P = M
    if rows is not None:
        if not isinstance(rows, torch.Tensor) or rows.dim() != 1:
            raise ValueError("rows must be an int32 tensor [P]")
        P = rows.shape[0]
        groups.need_vector(rows, torch.int32, (P,), X, "rows")
    experts = _need_experts(weight, M, K, P, E, gated, max_outliers, X, "weight")
    if not experts[0] and ld != K:
        raise ValueError("int8 weights take contiguous fp16 X")
    width = experts[1] // 2 if gated else experts[1]
    if out is None:
        out = X.new_empty((P, width))
    else:
        _need_shape(out, X.dtype, (P, width), X.device, "out")
    return _grouped(X, M, K, ld, dt, weight, experts, offsets, E, rows, P, gated, threshold, max_outliers, workspace, out)


def combine(P: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [T, D] in P's type: Y[t] = sum over j of weights[t, j] P[slots[t, j]], slots int32 and weights
    fp32 [T, top_k] as from ``route``; a slot that is no row of P adds nothing."""
    _need_shape(P, P.dtype, tuple(P.shape), P.device, "P")
    if P.dim() != 2 or P.dtype not in mx4._HALF or P.shape[1] % 16:
        raise ValueError(f"P must be fp16 or bf16 [rows, D], D a multiple of 16, got {P.dtype} {tuple(P.shape)}")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
        raise ValueError("slots must be an int32 tensor [T, top_k]")
    T, k = slots.shape
    groups.need_vector(slots, torch.int32, (T, k), P, "slots")
    groups.need_vector(weights, torch.float32, (T, k), P, "weights")
    n, D = P.shape
    if out is None:
        out = P.new_empty((T, D))
    else:
        _need_shape(out, P.dtype, (T, D), P.device, "out")
    groups.launch("moe_combine", P, P.data_ptr(), n, D, mx4.DTYPES[P.dtype], slots.data_ptr(), weights.data_ptr(), T, k,
                  out.data_ptr())
    return out


def moe_prompt(X: torch.Tensor, logits: torch.Tensor, gate_up: tuple, down: tuple, top_k: int,
               renormalize: bool = True, threshold: float = 6.0, max_outliers: int | None = None,
               out: torch.Tensor | None = None):
    """(Y [T, D], ids, weights) as ``moe_layer``, for few or many tokens: ``route``, the gated
    product of gate_up, the product of down and ``combine``. The activations are quantized like the
    weights (MX4, or int8 with fp16 outlier columns, threshold and max_outliers as in
    ``grouped_matmul``), and the hidden values and each expert's outputs are rounded to X's type
    between the launches, where ``moe_layer`` keeps both in 16 bits or more.

    T * top_k is at most 2^24; with MX4 weights X and the hidden values [T * top_k, I], their rows
    padded to 128 elements, have less than 2^33. Shapes that do not fit are refused before the first
    launch.
    """
    M, D, ld, dt = mx4._need_rows(X, "X")
    T, E = _need_logits(logits, top_k)
    if T != M or logits.get_device() != X.get_device():
        raise ValueError(f"logits must be [{M}, E] on {X.device}, got {tuple(logits.shape)} on {logits.device}")
    P = T * top_k
    first = _need_experts(gate_up, T, D, P, E, True, max_outliers, X, "gate_up")
    if not first[0] and ld != D:
        raise ValueError("int8 weights take contiguous fp16 X")
    I = first[1] // 2
    second = _need_experts(down, P, I, P, E, False, max_outliers, X, "down")
    if out is not None:
        _need_shape(out, X.dtype, (T, second[1]), X.device, "out")
    r = route(logits, top_k, renormalize)
    h = _grouped(X, T, D, ld, dt, gate_up, first, r.offsets, E, r.rows, P, True, threshold, max_outliers, None,
                 X.new_empty((P, I)))
    p = _grouped(h, P, I, I, dt, down, second, r.offsets, E, None, P, False, threshold, max_outliers, None,
                 X.new_empty((P, second[1])))
    return combine(p, r.slots, r.weights, out), r.ids, r.weights
