"""Entry points of include/groupmm.h, whose rows have weights of their own: what ``moe`` and
``lora`` share."""

from __future__ import annotations

import ctypes

import torch

from . import mx4
from .binding import _f32, _i64, _int, _need_shape, _p

_sz = ctypes.c_size_t

# name -> (restype, argtypes); exactly the symbols include/groupmm.h declares
SIGNATURES = {
    "moe_route_workspace_bytes": (_sz, [_i64, _i64]),
    "moe_route": (_int, [_p, _i64, _i64, _int, _i64, _int, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "moe_grouped_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64, _i64, _int, _i64]),
    "moe_grouped_matmul": (_int, [_p, _i64, _i64, _i64, _int, _int, _p, _p, _i64, _i64, _p, _p, _i64, _int, _f32, _i64,
                                  _p, _p, _sz, _p]),
    "moe_combine": (_int, [_p, _i64, _i64, _int, _p, _p, _i64, _i64, _p, _p]),
    "lora_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "lora_apply": (_int, [_p, _i64, _p, _i64, _i64, _i64, _int, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _i64, _p, _sz,
                          _p]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """libint8mm.so with these entry points' signatures set."""
    global _lib
    if _lib is None:
        L = mx4.lib()
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def launch(name: str, t: torch.Tensor, *args) -> None:
    """One library call on t's device, current or not, and on its current stream."""
    lib()
    mx4._launch(name, t, *args)


def need_vector(t: torch.Tensor, dtype: torch.dtype, shape: tuple, like: torch.Tensor, name: str) -> None:
    """A contiguous tensor of exactly this type and shape on `like`'s device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == like.get_device() and t.is_cuda):
        return
    _need_shape(t, dtype, shape, like.device, name)
