"""Microscaled 4-bit (MX4) operands and products (declared in include/mx4mm.h).

Blocks of 32 elements share a power of two (one byte); an element is a 4-bit floating point
code. ``quantize`` / ``prepare_weight`` / ``tile_weight`` give the tiled pair
``(codes, scales)`` that the products take, for activations and weights alike; a weight
takes 17/32 bytes per element. Argument marshalling only, as in ``binding``: every step runs
in the library's HIP kernels, on the current stream of the tensors' device.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import binding
from .binding import Int8mmError, _i64, _int, _need, _need_shape, _p

_sz = ctypes.c_size_t

# name -> (restype, argtypes); exactly the symbols include/mx4mm.h declares
SIGNATURES = {
    "mx4_codes_bytes": (_sz, [_i64, _i64]),
    "mx4_scales_bytes": (_sz, [_i64, _i64]),
    "mx4_quantize": (_int, [_p, _i64, _i64, _i64, _int, _p, _p, _p]),
    "mx4_prepare_weight": (_int, [_p, _i64, _i64, _int, _int, _p, _p, _p]),
    "mx4_tile_weight": (_int, [_p, _p, _i64, _i64, _p, _p, _p]),
    "mx4_dequantize": (_int, [_p, _p, _i64, _i64, _int, _p, _i64, _p]),
    "mx4_matmul_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mx4_matmul": (_int, [_p, _i64, _i64, _i64, _int, _p, _p, _i64, _p, _p, _sz, _p]),
    "mx4_matmul_q_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "mx4_matmul_q": (_int, [_p, _p, _i64, _i64, _p, _p, _i64, _int, _p, _p, _sz, _p]),
    "mx4_weight_only_matmul": (_int, [_p, _i64, _i64, _i64, _int, _p, _p, _i64, _p, _p]),
    "moe_layer_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "moe_layer": (_int, [_p, _i64, _i64, _i64, _int, _p, _i64, _int, _i64, _int, _int, _p, _p, _p,
                         _p, _i64, _p, _p, _p, _p, _sz, _p]),
}

DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

_lib = None


def lib() -> ctypes.CDLL:
    """libint8mm.so with these entry points' signatures set."""
    global _lib
    if _lib is None:
        L = binding.lib()
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _stream(index: int) -> int:
    """Handle of the current stream of device `index` (no Stream object: these calls are a few
    microseconds long)."""
    return torch._C._cuda_getCurrentRawStream(index)


@functools.cache
def _function(name: str):
    return getattr(lib(), name)


def _launch(name: str, t: torch.Tensor, *args) -> None:
    """One library call on t's device, current or not, and on its current stream."""
    index = t.get_device()
    if index == torch._C._cuda_getDevice():
        rc = _function(name)(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            rc = _function(name)(*args, _stream(index))
    if rc:
        raise Int8mmError(rc, name)


@functools.lru_cache(maxsize=1024)
def _sizes(rows: int, K: int) -> tuple[int, int]:
    """Bytes of the tiled codes and scales (asked of the library once per shape)."""
    L = lib()
    return int(L.mx4_codes_bytes(rows, K)), int(L.mx4_scales_bytes(rows, K))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(M: int, K: int, N: int) -> tuple[int, int]:
    """What mx4_matmul and mx4_matmul_q need."""
    L = lib()
    return int(L.mx4_matmul_workspace_bytes(M, K, N)), int(L.mx4_matmul_q_workspace_bytes(M, K, N))


_HALF = {torch.float16: 0, torch.bfloat16: 1}


def _need_rows(X: torch.Tensor, name: str, types=_HALF) -> tuple:
    """(M, K, row stride, dtype code) of a matrix whose rows are contiguous."""
    if not isinstance(X, torch.Tensor) or not binding._on_device(X):
        raise ValueError(f"{name} must be a HIP device tensor")
    dt = types.get(X.dtype)
    if dt is None:
        raise ValueError(f"{name} must be one of {tuple(types)}, got {X.dtype}")
    shape = X.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D [M, K], got shape {tuple(shape)}")
    M, K = shape
    ld, unit = X.stride()
    if M == 1:
        ld = K
    if (K > 1 and unit != 1) or ld < K or ld % 8:
        raise ValueError(f"{name}'s rows must be contiguous, with a row stride that is a multiple of 8 "
                         f"and at least {K}: its strides are {X.stride()}")
    return M, K, ld, dt


def _need_mx4(codes: torch.Tensor, scales: torch.Tensor, rows: int, K: int, like: torch.Tensor, name: str) -> None:
    """A tiled pair of `rows` rows of K elements on `like`'s device: the kernels trust its
    sizes and that it is in device memory (`like` may be the pair itself)."""
    want = _sizes(rows, K)
    if (binding._on_device(codes) and codes.dtype is torch.uint8 and scales.dtype is torch.uint8 and codes.is_contiguous()
            and scales.is_contiguous() and want[0] and codes.numel() == want[0] and scales.numel() == want[1]
            and codes.get_device() == scales.get_device() == like.get_device()):
        return
    _need(codes, torch.uint8, f"{name} codes")
    _need(scales, torch.uint8, f"{name} scales")
    if codes.device != like.device or scales.device != like.device:
        raise ValueError(f"{name} codes and scales must be on {like.device}")
    raise ValueError(f"{name}: {codes.numel()} bytes of codes and {scales.numel()} of scales; {rows} rows of "
                     f"{K} elements have {want[0]} and {want[1]}")


def _scratch(workspace: torch.Tensor | None, nbytes: int, like: torch.Tensor) -> torch.Tensor | None:
    """The caller's workspace, checked, or a new one of nbytes (None for 0)."""
    if workspace is None:
        return like.new_empty((nbytes,), dtype=torch.uint8) if nbytes else None
    _need(workspace, torch.uint8, "workspace")
    if workspace.device != like.device:
        raise ValueError(f"workspace must be on {like.device}")
    return workspace


def _empty(rows: int, K: int, like: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    if _sizes(rows, K)[0] == 0:
        raise ValueError(f"bad shape: {rows} rows of {K} elements")
    groups, ks = (rows + 15) // 16, (K + 127) // 128
    return (like.new_empty((groups, ks, 16, 64), dtype=torch.uint8),
            like.new_empty((groups, (ks + 3) // 4, 64, 4), dtype=torch.uint8))


def quantize(X: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows of fp16 or bf16 X [M, K] -> tiled (codes, scales); M is padded to 16 rows."""
    M, K, ld, dt = _need_rows(X, "X")
    codes, scales = _empty(M, K, X)
    _launch("mx4_quantize", X, X.data_ptr(), M, K, ld, dt, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def prepare_weight(W: torch.Tensor, layout: int = 0) -> tuple[torch.Tensor, torch.Tensor]:
    """fp16 or bf16 W ([K, N] for layout 0, [N, K] for layout 1) -> tiled (codes, scales), one
    row per output feature."""
    R, C, ld, dt = _need_rows(W, "W")
    if ld != C:
        raise ValueError("W must be contiguous")
    K, N = (R, C) if layout == 0 else (C, R)
    if N % 16:
        raise ValueError("N must be a multiple of 16")
    codes, scales = _empty(N, K, W)
    _launch("mx4_prepare_weight", W, W.data_ptr(), K, N, layout, dt, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def tile_weight(packed: torch.Tensor, block_scales: torch.Tensor, K: int | None = None):
    """A row-major MX4 weight, packed codes uint8 [N, 16 ceil(K / 32)] (even elements in the
    low four bits) and scale bytes uint8 [N, ceil(K / 32)], -> tiled (codes, scales). K is
    twice packed's width unless given. Layout only."""
    _need(packed, torch.uint8, "packed")
    _need(block_scales, torch.uint8, "block_scales")
    if packed.dim() != 2 or block_scales.dim() != 2 or packed.shape[1] % 16:
        raise ValueError("packed must be [N, 16 ceil(K / 32)] and block_scales [N, ceil(K / 32)], got "
                         f"{tuple(packed.shape)} and {tuple(block_scales.shape)}")
    N, blocks = packed.shape[0], packed.shape[1] // 16
    K = 32 * blocks if K is None else K
    if (K + 31) // 32 != blocks or tuple(block_scales.shape) != (N, blocks) or N % 16:
        raise ValueError(f"packed {tuple(packed.shape)} and block_scales {tuple(block_scales.shape)} are not those of "
                         f"N rows (a multiple of 16) of K = {K} elements")
    if block_scales.device != packed.device:
        raise ValueError(f"block_scales must be on {packed.device}")
    codes, scales = _empty(N, K, packed)
    _launch("mx4_tile_weight", packed, packed.data_ptr(), block_scales.data_ptr(), K, N, codes.data_ptr(),
            scales.data_ptr())
    return codes, scales


def untile(codes: torch.Tensor, scales: torch.Tensor, M: int, K: int):
    """Packed codes [M, 16 ceil(K / 32)] and scale bytes [M, ceil(K / 32)] held in a tiled pair
    (a copy; layout only)."""
    if codes.dim() != 4 or not 0 <= M <= 16 * codes.shape[0] or not 0 <= K <= 128 * codes.shape[1]:
        raise ValueError(f"codes of shape {tuple(codes.shape)} do not hold {M} rows of {K} elements")
    g, ks, nb = codes.shape[0], codes.shape[1], (K + 31) // 32
    packed = codes.permute(0, 2, 1, 3).reshape(g * 16, ks * 64)[:M, :16 * nb].contiguous()
    # scales [group, quad, (block of the unit, row), unit]
    s = scales.view(g, -1, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(g * 16, -1)
    return packed, s[:M, :nb].contiguous()


def dequantize(codes: torch.Tensor, scales: torch.Tensor, M: int, K: int,
               dtype: torch.dtype = torch.float16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values [M, K] of a tiled pair, in fp16, bf16 or fp32."""
    _need_mx4(codes, scales, M, K, codes, "operand")
    if out is None:
        if dtype not in DTYPES:
            raise ValueError(f"dtype must be one of {tuple(DTYPES)}, got {dtype}")
        out = codes.new_empty((M, K), dtype=dtype)
        ld, dt = K, DTYPES[dtype]
    else:
        m, k, ld, dt = _need_rows(out, "out", DTYPES)
        if (m, k) != (M, K) or out.device != codes.device or out.dtype != dtype:
            raise ValueError(f"out must be {dtype} [{M}, {K}] on {codes.device}, got {out.dtype} {tuple(out.shape)} "
                             f"on {out.device}")
    _launch("mx4_dequantize", codes, codes.data_ptr(), scales.data_ptr(), M, K, dt, out.data_ptr(), ld)
    return out


def _need_weight(w_codes: torch.Tensor, w_scales: torch.Tensor, K: int, like: torch.Tensor) -> int:
    """A tiled weight for K input features; returns N."""
    shape = w_codes.shape if isinstance(w_codes, torch.Tensor) else ()
    if len(shape) != 4:
        raise ValueError("the weight's codes must be the tiled tensor (N / 16, ceil(K / 128), 16, 64)")
    N = 16 * shape[0]
    _need_mx4(w_codes, w_scales, N, K, like, "weight")
    return N


def make_workspace(M: int, K: int, N: int, device="cuda") -> torch.Tensor:
    """A workspace for ``matmul`` (empty where the shape needs none: few rows), enough for
    ``matmul_q`` too."""
    if _sizes(M, K)[0] == 0 or _sizes(N, K)[0] == 0 or N % 16:
        raise ValueError(f"bad shape for mx4_matmul: M={M} K={K} N={N}")
    return torch.empty((_workspace_bytes(M, K, N)[0],), dtype=torch.uint8, device=device)


def matmul(X: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
           workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [M, N] = MX4(X) W^T in X's type, for an MX4 weight: X is quantized in the call."""
    M, K, ld, dt = _need_rows(X, "X")
    N = _need_weight(w_codes, w_scales, K, X)
    if out is None:
        out = X.new_empty((M, N))
    else:
        _need_shape(out, X.dtype, (M, N), X.device, "out")
    workspace = _scratch(workspace, _workspace_bytes(M, K, N)[0], X)
    ws, wb = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _launch("mx4_matmul", X, X.data_ptr(), M, K, ld, dt, w_codes.data_ptr(), w_scales.data_ptr(), N,
            out.data_ptr(), ws, wb)
    return out


def matmul_q(x_codes: torch.Tensor, x_scales: torch.Tensor, M: int, K: int, w_codes: torch.Tensor,
             w_scales: torch.Tensor, dtype: torch.dtype = torch.float16,
             workspace: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [M, N] in fp16 or bf16 from X [M, K] already quantized (once for several weights)."""
    if dtype not in _HALF:
        raise ValueError(f"dtype must be fp16 or bf16, got {dtype}")
    _need_mx4(x_codes, x_scales, M, K, x_codes, "X")
    N = _need_weight(w_codes, w_scales, K, x_codes)
    if out is None:
        out = x_codes.new_empty((M, N), dtype=dtype)
    else:
        _need_shape(out, dtype, (M, N), x_codes.device, "out")
    workspace = _scratch(workspace, _workspace_bytes(M, K, N)[1], x_codes)
    ws, wb = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _launch("mx4_matmul_q", x_codes, x_codes.data_ptr(), x_scales.data_ptr(), M, K, w_codes.data_ptr(),
            w_scales.data_ptr(), N, DTYPES[dtype], out.data_ptr(), ws, wb)
    return out


def weight_only_matmul(X: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [M, N] = X W^T for at most 16 rows of 16-bit X, as it is, and an MX4 weight."""
    M, K, ld, dt = _need_rows(X, "X")
    N = _need_weight(w_codes, w_scales, K, X)
    if out is None:
        out = X.new_empty((M, N))
    else:
        _need_shape(out, X.dtype, (M, N), X.device, "out")
    _launch("mx4_weight_only_matmul", X, X.data_ptr(), M, K, ld, dt, w_codes.data_ptr(), w_scales.data_ptr(), N,
            out.data_ptr())
    return out
