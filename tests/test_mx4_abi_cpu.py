"""Host-side checks of the MX4 and mixture-of-experts entry points: header, binding and
exports agree, bad arguments are refused before any HIP call (fake pointers, no GPU)."""

import os
import re

import pytest

from int8_mixed_precision_col_amd import binding, mx4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mx4mm.h")
P, U = 0x10000, 0x10008
E_NULL, E_SHAPE, E_ALIGN, E_WS = 1, 2, 3, 5
BIG = 1 << 40

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH),
                                reason="libint8mm.so not built (run __graft_entry__.build())")


@pytest.fixture(scope="module")
def L():
    return mx4.lib()


def test_header_binding_and_exports_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b((?:mx4|moe)_\w+)\s*\(", text)))
    assert declared == sorted(mx4.SIGNATURES)
    for name in declared:
        assert hasattr(L, name), name


def test_sizes(L):
    for rows, K in [(1, 16), (16, 128), (17, 144), (333, 1040), (4096, 12288)]:
        g, ks = -(-rows // 16), -(-K // 128)
        assert L.mx4_codes_bytes(rows, K) == g * ks * 1024
        assert L.mx4_scales_bytes(rows, K) == g * -(-ks // 4) * 256
        need = L.mx4_matmul_workspace_bytes(rows, K, 64)
        one_launch = rows <= 16 or (rows <= 64 and rows * -(-ks // 4) <= 96)
        assert need == 0 if one_launch else need >= g * ks * 1024 + g * -(-ks // 4) * 256
    for rows, K in [(0, 64), (64, 0), (64, 24), (1 << 25, 64), (64, (1 << 20) + 16), (1 << 24, 1 << 20), (-5, 64)]:
        assert L.mx4_codes_bytes(rows, K) == 0 and L.mx4_scales_bytes(rows, K) == 0
    assert L.mx4_matmul_workspace_bytes(64, 64, 24) == 0
    assert L.mx4_matmul_q_workspace_bytes(64, 64, 24) == 0 and L.mx4_matmul_q_workspace_bytes(300, 1040, 528) == 0
    # a long K over few tiles: fp32 sums of the splits
    need = L.mx4_matmul_q_workspace_bytes(128, 12288, 512)
    assert need > 0 and need % (4 * 128 * 512) == 0
    assert L.mx4_matmul_workspace_bytes(128, 12288, 512) >= need + 8 * 96 * 1024 + 8 * 24 * 256
    assert L.moe_layer_workspace_bytes(16, 1280, 8) >= 16 * 8 * 1280 * 4
    for bad in [(0, 64, 2), (17, 64, 2), (4, 60, 2), (4, 64, 0), (4, 64, 17)]:
        assert L.moe_layer_workspace_bytes(*bad) == 0


def call(L, name, args, kw):
    a = dict(args)
    assert not set(kw) - set(a)
    a.update(kw)
    return getattr(L, name)(*a.values(), None)


QUANT = dict(X=P, M=8, K=64, ldx=64, dt=0, codes=P, scales=P)
PREP = dict(W=P, K=64, N=32, layout=0, dt=0, codes=P, scales=P)
TILE = dict(packed=P, bs=P, K=64, N=32, codes=P, scales=P)
DEQ = dict(codes=P, scales=P, M=8, K=64, dt=2, out=P, ldo=64)
MM = dict(X=P, M=100, K=64, ldx=64, dt=1, wc=P, ws=P, N=32, Y=P, work=P, wb=BIG)
MMQ = dict(xc=P, xs=P, M=100, K=8192, wc=P, ws=P, N=128, dt=0, Y=P, work=P, wb=BIG)
WO = dict(X=P, M=8, K=64, ldx=64, dt=0, wc=P, ws=P, N=32, Y=P)
MOE = dict(X=P, T=4, D=64, ldx=64, dt=0, logits=P, E=8, ldt=2, k=2, renorm=1, fmt=0, w13=P, s13=P, w2=P, s2=P,
           I=32, Y=P, ids=P, weights=P, work=P, wb=BIG)
ALL = {"mx4_quantize": QUANT, "mx4_prepare_weight": PREP, "mx4_tile_weight": TILE, "mx4_dequantize": DEQ,
       "mx4_matmul": MM, "mx4_matmul_q": MMQ, "mx4_weight_only_matmul": WO, "moe_layer": MOE}
OPTIONAL = {"ids", "weights"}


@pytest.mark.parametrize("name", ALL)
def test_every_pointer_is_checked(L, name):
    for key, v in ALL[name].items():
        if v != P:
            continue
        if key not in OPTIONAL:
            assert call(L, name, ALL[name], {key: None}) == E_NULL, key
        assert call(L, name, ALL[name], {key: U}) == E_ALIGN, key


@pytest.mark.parametrize("name,kw,code", [
    *[(n, dict(K=k, **({"ldx": 1 << 22} if "ldx" in ALL[n] else {})), E_SHAPE)
      for n in ALL if "K" in ALL[n] for k in (0, -16, 24, (1 << 20) + 16)],
    *[(n, dict(M=m), E_SHAPE) for n in ALL if "M" in ALL[n] for m in (0, -1, 1 << 25)],
    *[(n, dict(N=m), E_SHAPE) for n in ALL if "N" in ALL[n] for m in (0, 8, 40, (1 << 24) + 16)],
    *[(n, {key: ld}, E_SHAPE) for n, key in (("mx4_quantize", "ldx"), ("mx4_dequantize", "ldo"), ("mx4_matmul", "ldx"),
                                             ("mx4_weight_only_matmul", "ldx"), ("moe_layer", "ldx"))
      for ld in (63, 56, 68, -64)],
    *[(n, dict(dt=d), E_SHAPE) for n in ("mx4_quantize", "mx4_prepare_weight", "mx4_matmul", "mx4_matmul_q",
                                         "mx4_weight_only_matmul", "moe_layer") for d in (-1, 2, 3)],
    ("mx4_dequantize", dict(dt=3), E_SHAPE), ("mx4_dequantize", dict(dt=-1), E_SHAPE),
    ("mx4_quantize", dict(M=1 << 24, K=1 << 20, ldx=1 << 20), E_SHAPE),
    ("mx4_prepare_weight", dict(layout=2), E_SHAPE),
    ("mx4_matmul", dict(M=64, ldx=1 << 24), E_SHAPE),   # one launch: X behind a buffer resource
    ("mx4_matmul_q", dict(wb=64), E_WS), ("mx4_matmul", dict(M=16, ldx=1 << 26), E_SHAPE), ("mx4_matmul", dict(wb=0), E_WS), ("mx4_matmul", dict(M=4096, wb=4096), E_WS),
    ("mx4_weight_only_matmul", dict(M=17), E_SHAPE), ("mx4_weight_only_matmul", dict(M=16, ldx=1 << 26), E_SHAPE),
    ("moe_layer", dict(T=0), E_SHAPE), ("moe_layer", dict(T=17), E_SHAPE), ("moe_layer", dict(D=56), E_SHAPE),
    ("moe_layer", dict(I=24), E_SHAPE), ("moe_layer", dict(E=0), E_SHAPE), ("moe_layer", dict(E=513), E_SHAPE),
    ("moe_layer", dict(k=0), E_SHAPE), ("moe_layer", dict(k=9), E_SHAPE), ("moe_layer", dict(E=64, k=17), E_SHAPE),
    ("moe_layer", dict(ldt=3), E_SHAPE), ("moe_layer", dict(fmt=2), E_SHAPE), ("moe_layer", dict(wb=64), E_WS),
    ("moe_layer", dict(T=16, ldx=1 << 26), E_SHAPE), ("moe_layer", dict(D=133152, ldx=133152), E_SHAPE),
])
def test_refusals(L, name, kw, code):
    assert call(L, name, ALL[name], kw) == code
