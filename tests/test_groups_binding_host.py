"""Host-side checks of moe's and lora's bindings: tensors whose type, shape, strides or sizes do
not fit are refused with ValueError before the library is asked to launch anything. Runs on
the CPU with the device predicate and the launches replaced by stand-ins; the size helpers are
the library's own."""

import os

import pytest
import torch

from int8_mixed_precision_col_amd import binding, groups, lora, moe, mx4
from tests.test_mx4_binding_host import f16, int8_pair, pair

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH),
                                reason="libint8mm.so not built (run __graft_entry__.build())")


@pytest.fixture
def calls(monkeypatch):
    seen = []
    groups.lib()
    monkeypatch.setattr(binding, "_on_device", lambda t: True)
    monkeypatch.setattr(mx4, "_launch", lambda name, t, *args: seen.append((name, args)))
    yield seen


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def grouped_args(**kw):
    return {**dict(X=f16(5, 64), weight=pair(3 * 32, 64), offsets=i32(4), rows=i32(11)), **kw}


def lora_args(**kw):
    return {**dict(Y=f16(5, 48), X=f16(5, 64), A=f16(3, 16, 64), B=f16(3, 48, 16), ids=i32(5), scales=torch.zeros(3),
                   ranks=i32(3)), **kw}


def test_good_calls_reach_the_library(calls):
    r = moe.route(torch.zeros(70, 9), 3)
    assert [tuple(t.shape) for t in r] == [(70, 3), (70, 3), (10,), (210,), (70, 3)]
    assert moe.grouped_matmul(**grouped_args()).shape == (11, 32)
    assert moe.grouped_matmul(**grouped_args(gated=True)).shape == (11, 16)
    assert moe.grouped_matmul(**grouped_args(rows=None, X=f16(5, 64).bfloat16())).dtype == torch.bfloat16
    assert calls[-1][1][11] == 0 and calls[-1][1][12] == 5            # no rows: P = M
    moe.grouped_matmul(**grouped_args(X=f16(5, 144)[:, 16:80]))
    assert calls[-1][1][1:4] == (5, 64, 144)
    moe.grouped_matmul(**grouped_args(weight=int8_pair(3 * 32, 64)))
    assert calls[-1][1][5] == 0 and calls[-1][1][15] == 64            # every column may be an outlier
    assert moe.combine(f16(11, 64), i32(5, 2), torch.zeros(5, 2)).shape == (5, 64)
    assert lora.apply(**lora_args()).shape == (5, 48)
    assert lora.apply(**lora_args(scales=None, ranks=None)).shape == (5, 48)
    assert calls[-1][1][13:15] == (0, 0)
    t = lora_args()
    assert lora.apply(**t, out=t["Y"]) is t["Y"]
    y, ids, w = moe.moe_prompt(f16(20, 64), torch.zeros(20, 4), pair(4 * 64, 64), pair(4 * 64, 32), 2)
    assert y.shape == (20, 64) and ids.shape == w.shape == (20, 2)
    assert [c[0] for c in calls[-4:]] == ["moe_route", "moe_grouped_matmul", "moe_grouped_matmul", "moe_combine"]


@pytest.mark.parametrize("K", [64, 144, 2048, 16384])
@pytest.mark.parametrize("most", [None, 0, 40, 256, 1 << 20])
@pytest.mark.parametrize("weights", ["int8", "mx4"])
def test_the_size_helper_sizes_the_call(calls, weights, most, K):
    """The helper's size is what the library asks for with the outlier columns that the call tells it."""
    w = int8_pair(96, K) if weights == "int8" else pair(96, K)
    args = {} if most is None else {"max_outliers": most}
    fmt = int(weights == "mx4")
    need = moe.grouped_workspace_bytes(5, K, 11, 3, 32, fmt, **args)
    t = grouped_args(X=f16(5, K), weight=w, **args)
    assert moe.grouped_matmul(**t, workspace=torch.zeros(need, dtype=torch.uint8)).shape == (11, 32)
    told = calls[-1][1]
    assert told[18] == need == groups.lib().moe_grouped_workspace_bytes(5, K, 11, 3, 32, fmt, told[15])


@pytest.mark.parametrize("logits,k", [
    (torch.zeros(4, 8, dtype=torch.float64), 2), (torch.zeros(8), 1), (torch.zeros(8, 4).T, 2), (torch.zeros(4, 8), 0),
    (torch.zeros(4, 8), 9), (torch.zeros(4, 20), 17), (torch.zeros(0, 8), 2), (torch.zeros(4, 0), 1), (torch.zeros(2, 513), 2)])
def test_route_refused(calls, logits, k):
    with pytest.raises(ValueError):
        moe.route(logits, k)
    assert calls == []


@pytest.mark.parametrize("kw", [
    dict(X=f16(5, 64).float()), dict(X=f16(64)), dict(X=f16(64, 5).T), dict(X=f16(5, 68)[:, :64]), dict(X=f16(0, 64)),
    dict(offsets=i32(4).long()), dict(offsets=i32(1)), dict(offsets=i32(8)[::2]), dict(offsets=i32(2, 2)), dict(offsets=i32(6)),
    dict(rows=i32(11).long()), dict(rows=i32(0)), dict(rows=i32(22)[::2]), dict(rows=i32(11, 1)),
    dict(weight=pair(3 * 32, 192)), dict(weight=pair(3 * 32 + 16, 64)), dict(weight=(pair(96, 64)[0], pair(64, 64)[1])),
    dict(weight=pair(3 * 48, 64), gated=True), dict(weight=int8_pair(96, 64), X=f16(5, 64).bfloat16()),
    dict(weight=int8_pair(96, 64), X=f16(5, 128)[:, :64]), dict(weight=(int8_pair(96, 64)[0], torch.zeros(80))),
    dict(out=f16(11, 16)), dict(out=f16(10, 32)), dict(out=f16(11, 32).bfloat16()), dict(out=f16(11, 64)[:, :32]),
    dict(gated=True, out=f16(11, 32)), dict(workspace=torch.zeros(1 << 20)),
])
def test_grouped_refused(calls, kw):
    with pytest.raises(ValueError):
        moe.grouped_matmul(**grouped_args(**kw))
    assert calls == []


@pytest.mark.parametrize("args", [
    (f16(11, 64).float(), i32(5, 2), torch.zeros(5, 2)), (f16(11, 24), i32(5, 2), torch.zeros(5, 2)),
    (f16(64, 11).T, i32(5, 2), torch.zeros(5, 2)), (f16(11, 64), i32(5, 2).long(), torch.zeros(5, 2)),
    (f16(11, 64), i32(5, 2), torch.zeros(5, 3)), (f16(11, 64), i32(5, 2), torch.zeros(5, 2).half()),
    (f16(11, 64), i32(10), torch.zeros(10)), (f16(11, 64), i32(2, 5).T, torch.zeros(5, 2)),
    (f16(11, 64), i32(5, 2), torch.zeros(5, 2), f16(5, 48)), (f16(11, 64), i32(5, 2), torch.zeros(5, 2), f16(4, 64)),
])
def test_combine_refused(calls, args):
    with pytest.raises(ValueError):
        moe.combine(*args)
    assert calls == []


@pytest.mark.parametrize("kw", [
    dict(X=f16(5, 64).float()), dict(X=f16(4, 64)), dict(Y=f16(5, 48).bfloat16()), dict(Y=f16(4, 48)), dict(Y=f16(5, 52)[:, :48]),
    dict(A=f16(3, 16, 80)), dict(A=f16(3, 16, 64).bfloat16()), dict(A=f16(3, 64, 16).transpose(1, 2)), dict(A=f16(48, 64)),
    dict(A=f16(3, 12, 64), B=f16(3, 48, 12)), dict(A=f16(3, 136, 64), B=f16(3, 48, 136)), dict(A=f16(3, 8, 64)),
    dict(B=f16(3, 32, 16)), dict(B=f16(2, 48, 16)), dict(A=f16(0, 16, 64), B=f16(0, 48, 16), scales=None, ranks=None),
    dict(ids=i32(5).long()), dict(ids=i32(6)), dict(ids=i32(10)[::2]), dict(scales=torch.zeros(2)), dict(scales=f16(3)),
    dict(ranks=i32(3).long()), dict(ranks=i32(4)), dict(out=f16(5, 32)), dict(out=f16(5, 48).bfloat16()),
    dict(out=f16(6, 48)), dict(workspace=torch.zeros(1 << 20)),
])
def test_lora_refused(calls, kw):
    with pytest.raises(ValueError):
        lora.apply(**lora_args(**kw))
    assert calls == []


@pytest.mark.parametrize("logits", [torch.zeros(19, 4), torch.zeros(21, 4), torch.zeros(0, 4), torch.zeros(20), None])
def test_prompt_of_other_tokens_than_the_logits_refused(calls, logits):
    with pytest.raises(ValueError):
        moe.moe_prompt(f16(20, 64), logits, pair(4 * 64, 64), pair(4 * 64, 32), 2)
    assert calls == []


@pytest.mark.parametrize("name", ["Y", "X", "A", "B", "scales", "out"])
def test_lora_that_autograd_would_have_to_record_refused(calls, name):
    t = lora_args(out=f16(5, 48))
    t[name] = t[name].clone().requires_grad_()
    with pytest.raises(ValueError, match="no backward"):
        lora.apply(**t)
    assert calls == []
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            assert lora.apply(**t).shape == (5, 48)
    t[name] = t[name].detach()
    assert lora.apply(**t).shape == (5, 48) and len(calls) == 3


@pytest.mark.parametrize("T,D,E,gate_up,down,k,kw", [
    (20, 64, 4, pair(4 * 64, 64), pair(4 * 64, 160), 2, {}), (20, 64, 4, pair(4 * 64, 64), pair(4 * 64 + 16, 32), 2, {}),
    (20, 64, 4, pair(4 * 48, 64), pair(4 * 64, 32), 2, {}), (20, 64, 4, pair(4 * 64, 192), pair(4 * 64, 32), 2, {}),
    (20, 64, 4, pair(4 * 64, 64), (pair(4 * 64, 32)[0], pair(16, 32)[1]), 2, {}), (20, 64, 4, pair(4 * 64, 64), (None, None), 2, {}),
    (20, 64, 4, pair(4 * 64, 64), pair(4 * 64, 32), 5, {}), (20, 64, 4, pair(4 * 64, 64), pair(4 * 64, 32), 0, {}),
    (20, 64, 4, pair(4 * 64, 64), pair(4 * 64, 32), 2, dict(out=f16(19, 64))),
    (20, 64, 4, pair(4 * 64, 64), pair(4 * 64, 32), 2, dict(out=f16(20, 64).bfloat16())),
    (20, 64, 4, int8_pair(4 * 64, 64), int8_pair(4 * 64, 32), 2, dict(max_outliers=-1)),
    (600000, 16, 1, pair(2 * 14336, 16), pair(16, 14336), 1, {}),     # the hidden values are 2^33 elements
    ((1 << 21) + 1, 16, 8, pair(8 * 32, 16), pair(8 * 16, 16), 8, {}),    # more than 2^24 rows
])
def test_prompt_is_refused_before_its_first_launch(calls, T, D, E, gate_up, down, k, kw):
    with pytest.raises(ValueError):
        moe.moe_prompt(f16(T, D), torch.zeros(T, E), gate_up, down, k, **kw)
    assert calls == []


def test_prompt_over_int8_refuses_bf16_and_strided_rows_before_its_first_launch(calls):
    w = int8_pair(4 * 64, 64), int8_pair(4 * 64, 32)
    for x in (f16(20, 64).bfloat16(), f16(20, 128)[:, :64]):
        with pytest.raises(ValueError):
            moe.moe_prompt(x, torch.zeros(20, 4), *w, 2)
        assert calls == []


def test_cpu_tensors_are_refused_by_every_call(monkeypatch):
    launched = []
    monkeypatch.setattr(mx4, "_launch", lambda name, t, *args: launched.append(name))
    for f in (lambda: moe.route(torch.zeros(4, 8), 2), lambda: moe.grouped_matmul(**grouped_args()),
              lambda: moe.combine(f16(11, 64), i32(5, 2), torch.zeros(5, 2)), lambda: lora.apply(**lora_args()),
              lambda: moe.moe_prompt(f16(20, 64), torch.zeros(20, 4), pair(4 * 64, 64), pair(4 * 64, 32), 2)):
        with pytest.raises(ValueError):
            f()
        assert launched == []
