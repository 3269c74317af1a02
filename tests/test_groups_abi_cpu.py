"""Host-side checks of include/groupmm.h's entry points: header, binding and exports agree, bad
arguments are refused before any HIP call (fake pointers, no GPU)."""

import os
import re

import pytest

from int8_mixed_precision_col_amd import binding, groups

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "groupmm.h")
P, U, V = 0x10000, 0x10008, 0x10002
E_NULL, E_SHAPE, E_ALIGN, E_THRESHOLD, E_WS = 1, 2, 3, 4, 5
BIG = 1 << 50

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH),
                                reason="libint8mm.so not built (run __graft_entry__.build())")


@pytest.fixture(scope="module")
def L():
    return groups.lib()


def test_header_binding_and_exports_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b((?:moe|lora)_\w+)\s*\(", text)))
    assert declared == sorted(groups.SIGNATURES)
    for name in declared:
        assert hasattr(L, name), name


def test_sizes(L):
    assert L.moe_route_workspace_bytes(64, 512) == 0
    assert L.moe_route_workspace_bytes(65, 512) >= 2 * 512 * 2
    assert L.moe_route_workspace_bytes(1 << 24, 512) >= 256 * 512 * 2
    for bad in [(0, 8), (8, 0), (8, 513), ((1 << 24) + 1, 8), (-1, 8)]:
        assert L.moe_route_workspace_bytes(*bad) == 0
    # codes and scales of X and a row of zeros
    assert L.moe_grouped_workspace_bytes(100, 1040, 300, 10, 528, 1, 0) >= 101 * 9 * 64 + 101 * 3 * 16 
    assert L.moe_grouped_workspace_bytes(100, 1040, 300, 10, 528, 0, 256) >= L.int8_quant_state_bytes(100, 1040, 256)
    good = dict(M=8, K=64, P=16, E=4, N=32, fmt=1, mo=16)
    assert L.moe_grouped_workspace_bytes(*good.values()) > 0
    for kw in (dict(M=0), dict(K=24), dict(K=0), dict(P=0), dict(E=0), dict(E=1025), dict(N=8), dict(N=24), dict(fmt=2),
               dict(fmt=-1), dict(fmt=0, mo=65), dict(fmt=0, mo=-1), dict(fmt=0, K=133152), dict(E=1024, N=1 << 20),
               dict(M=1 << 24, K=4096), dict(P=1 << 24, N=1 << 20), dict(M=1 << 21, K=4096)):
        assert L.moe_grouped_workspace_bytes(*{**good, **kw}.values()) == 0, kw
    assert L.lora_workspace_bytes(1000, 64, 5, 24) >= 1000 * 32 * 4
    for bad in [(0, 64, 1, 8), (8, 24, 1, 8), (8, 64, 0, 8), (8, 64, 1025, 8), (8, 64, 1, 0), (8, 64, 1, 12), (8, 64, 1, 136)]:
        assert L.lora_workspace_bytes(*bad) == 0


def call(L, name, args, kw):
    a = dict(args)
    assert not set(kw) - set(a)
    a.update(kw)
    return getattr(L, name)(*a.values(), None)


ROUTE = dict(logits=P, T=100, E=8, dt=2, k=2, renorm=1, ids=P, weights=P, offsets=P, rows=P, slots=P, work=P, wb=BIG)
GROUPED = dict(X=P, M=8, K=64, ldx=64, dt=0, fmt=1, w=P, s=P, E=4, N=32, offsets=P, rows=P, P=16, gated=1, t=6.0, mo=16,
               Y=P, work=P, wb=BIG)
COMBINE = dict(P=P, rows=16, D=64, dt=0, slots=P, weights=P, T=8, k=2, Y=P)
LORA = dict(Y=P, ldy=32, X=P, M=8, K=64, ldx=64, dt=1, A=P, B=P, S=3, R=16, N=32, ids=P, scales=P, ranks=P, out=P + 4096,
            ldo=40, work=P, wb=BIG)
ALL = {"moe_route": ROUTE, "moe_grouped_matmul": GROUPED, "moe_combine": COMBINE, "lora_apply": LORA}
OPTIONAL = {"scales", "ranks"}                              # rows too, but not with these P and M
VECTORS = {"ids", "weights", "offsets", "rows", "slots", "scales", "ranks"}


@pytest.mark.parametrize("name", ALL)
def test_every_pointer_is_checked(L, name):
    for key, v in ALL[name].items():
        if v not in (P, P + 4096) or isinstance(v, float):
            continue
        if key not in OPTIONAL:
            want = E_SHAPE if (name, key) == ("moe_grouped_matmul", "rows") else E_NULL
            assert call(L, name, ALL[name], {key: None}) == want, key
        assert call(L, name, ALL[name], {key: V if key in VECTORS else U}) == E_ALIGN, key


@pytest.mark.parametrize("name,kw,code", [
    *[("moe_route", kw, E_SHAPE) for kw in (dict(T=0), dict(T=-1), dict(T=(1 << 24) + 1), dict(E=0), dict(E=513), dict(dt=3),
                                            dict(dt=-1), dict(k=0), dict(k=9), dict(E=64, k=17))],
    ("moe_route", dict(wb=64), E_WS),
    *[("moe_grouped_matmul", kw, E_SHAPE) for kw in (
        dict(M=0), dict(K=24), dict(K=1 << 21, ldx=1 << 21), dict(ldx=56), dict(ldx=68), dict(dt=2), dict(dt=-1), dict(fmt=2),
        dict(E=0), dict(E=1025), dict(N=24), dict(N=48), dict(P=0), dict(P=1 << 25), dict(rows=None), dict(M=1 << 24, K=4096, ldx=4096),
        dict(fmt=0, dt=1), dict(fmt=0, ldx=72), dict(fmt=0, mo=65))],
    ("moe_grouped_matmul", dict(fmt=0, t=-1.0), E_THRESHOLD), ("moe_grouped_matmul", dict(fmt=0, t=float("nan")), E_THRESHOLD),
    ("moe_grouped_matmul", dict(wb=64), E_WS), ("moe_grouped_matmul", dict(fmt=0, wb=64), E_WS),
    *[("moe_combine", kw, E_SHAPE) for kw in (dict(rows=0), dict(D=8), dict(D=24), dict(dt=2), dict(T=0), dict(k=0), dict(k=17),
                                              dict(rows=(1 << 28) + 1))],
    *[("lora_apply", kw, E_SHAPE) for kw in (
        dict(M=0), dict(K=24), dict(N=24), dict(N=0), dict(S=0), dict(S=1025), dict(R=0), dict(R=12), dict(R=136), dict(ldy=24),
        dict(ldy=36), dict(ldx=56), dict(ldx=66), dict(ldo=24), dict(ldo=44), dict(out=P), dict(dt=2), dict(dt=-1))],
    ("lora_apply", dict(wb=64), E_WS),
])
def test_refusals(L, name, kw, code):
    assert call(L, name, ALL[name], kw) == code
