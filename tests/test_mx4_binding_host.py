"""Host-side checks of the MX4 and mixture-of-experts bindings: tensors whose type, shape,
strides or sizes do not fit are refused with ValueError before the library is asked to
launch anything. Runs on the CPU with the device predicate, the stream lookup and the
launches replaced by stand-ins; the size helpers are the library's own."""

import os

import pytest
import torch

from int8_mixed_precision_col_amd import binding, moe, mx4

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH),
                                reason="libint8mm.so not built (run __graft_entry__.build())")


class FakeLib:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLib(mx4.lib())
    monkeypatch.setattr(mx4, "lib", lambda: lib)
    monkeypatch.setattr(binding, "_on_device", lambda t: True)
    monkeypatch.setattr(mx4, "_launch", lambda name, t, *args: getattr(lib, name)(*args))
    yield lib


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def pair(rows, K):
    g, ks = -(-rows // 16), -(-K // 128)
    return (torch.zeros((g, ks, 16, 64), dtype=torch.uint8), torch.zeros((g, -(-ks // 4), 64, 4), dtype=torch.uint8))


def int8_pair(N, K):
    return torch.zeros((N // 16, -(-K // 64), 16, 64), dtype=torch.int8), torch.zeros(N)


def test_good_calls_reach_the_library(fake):
    X, W = f16(5, 272), pair(48, 272)
    assert mx4.matmul(X, *W).shape == (5, 48)
    assert mx4.weight_only_matmul(X.bfloat16(), *W).dtype == torch.bfloat16
    q = mx4.quantize(X)
    assert mx4.matmul_q(*q, 5, 272, *W, dtype=torch.bfloat16).shape == (5, 48)
    assert mx4.dequantize(*q, 5, 272, torch.float32).shape == (5, 272)
    wide = f16(5, 400)[:, 64:336]
    mx4.matmul(wide, *W)
    assert fake.calls[-1][1][1:4] == (5, 272, 400)      # M, K, the row stride
    mx4.matmul(f16(1, 400)[:, :272], *W)
    assert fake.calls[-1][1][1:4] == (1, 272, 272)      # one row has no stride
    assert [c[0] for c in fake.calls] == ["mx4_matmul", "mx4_weight_only_matmul", "mx4_quantize", "mx4_matmul_q",
                                          "mx4_dequantize", "mx4_matmul", "mx4_matmul"]
    y, ids, w = moe.moe_layer(f16(3, 64), torch.zeros(3, 4), pair(4 * 2 * 32, 64), pair(4 * 64, 32), 2)
    assert y.shape == (3, 64) and ids.shape == w.shape == (3, 2) and ids.dtype == torch.int32
    moe.moe_layer(f16(3, 64), torch.zeros(3, 4).half(), int8_pair(4 * 2 * 32, 64), int8_pair(4 * 64, 32), 2)
    assert fake.calls[-1][1][10] == 0 and fake.calls[-2][1][10] == 1


@pytest.mark.parametrize("make", [
    lambda: f16(5, 272).float(), lambda: f16(272), lambda: f16(1, 5, 272), lambda: f16(272, 5).T,
    lambda: f16(5, 276)[:, :272], lambda: f16(5, 544)[:, ::2], lambda: f16(1, 272).expand(5, 272),
    lambda: f16(5, 1088)[:, :272].to(torch.int16),
])
def test_activations_refused(fake, make):
    X, W = make(), pair(48, 272)
    for f in (lambda: mx4.quantize(X), lambda: mx4.matmul(X, *W), lambda: mx4.weight_only_matmul(X, *W),
              lambda: moe.moe_layer(X, torch.zeros(5, 4), pair(4 * 2 * 32, 272), pair(4 * 272, 32), 2)):
        with pytest.raises(ValueError):
            f()
    assert fake.calls == []


@pytest.mark.parametrize("W", [
    pair(48, 144), (pair(48, 272)[0], pair(32, 272)[1]), (pair(48, 272)[0].view(torch.int8), pair(48, 272)[1]),
    (pair(48, 272)[0].reshape(-1), pair(48, 272)[1]), (pair(48, 272)[0][:, :, :, ::2], pair(48, 272)[1]),
])
def test_weights_refused(fake, W):
    X = f16(5, 272)
    for f in (lambda: mx4.matmul(X, *W), lambda: mx4.weight_only_matmul(X, *W),
              lambda: mx4.matmul_q(*pair(5, 272), 5, 272, *W)):
        with pytest.raises(ValueError):
            f()
    assert fake.calls == []


def test_outputs_and_workspaces_refused(fake):
    X, W = f16(5, 272), pair(48, 272)
    for out in (f16(5, 32), f16(6, 48), f16(5, 48).bfloat16(), f16(48, 5).T, f16(5, 96)[:, :48]):
        for f in (lambda: mx4.matmul(X, *W, out=out), lambda: mx4.weight_only_matmul(X, *W, out=out),
                  lambda: mx4.matmul_q(*pair(5, 272), 5, 272, *W, out=out)):
            with pytest.raises(ValueError):
                f()
    with pytest.raises(ValueError):
        mx4.matmul(X, *W, workspace=torch.zeros(1 << 20))
    for out in (f16(5, 256), f16(4, 272), f16(272, 5).T, f16(5, 272).float()):
        with pytest.raises(ValueError):
            mx4.dequantize(*pair(5, 272), 5, 272, torch.float16, out=out)
    for kw in (dict(M=17, K=272), dict(M=5, K=400), dict(M=5, K=272, dtype=torch.int8)):
        with pytest.raises(ValueError):
            mx4.dequantize(*pair(5, 272), **kw)
    with pytest.raises(ValueError):
        mx4.matmul_q(*pair(5, 272), 5, 272, *W, dtype=torch.float32)
    assert fake.calls == []


def test_weight_conversion_refused(fake):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for args in ((u8(32, 24), u8(32, 2)), (u8(32, 32), u8(32, 1)), (u8(24, 32), u8(24, 2)), (u8(32, 32), u8(32, 2), 16),
                 (u8(32, 32), u8(32, 2), 80), (u8(32, 32).view(torch.int8), u8(32, 2)), (u8(32, 32, 1), u8(32, 2))):
        with pytest.raises(ValueError):
            mx4.tile_weight(*args)
    for W, layout in ((f16(64, 24), 0), (f16(24, 64), 1), (f16(64, 96)[:, :64], 0), (f16(64, 64).float(), 0)):
        with pytest.raises(ValueError):
            mx4.prepare_weight(W, layout)
    assert fake.calls == []
    mx4.tile_weight(u8(32, 32), u8(32, 2), 48)
    assert fake.calls[-1][1][2:4] == (48, 32)


def test_untile_refused():
    codes, scales = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 64, 4, dtype=torch.uint8)
    assert mx4.untile(codes, scales, 32, 128)[0].shape == (32, 64)
    for args in ((codes, scales, 33, 128), (codes, scales, 32, 144), (codes, scales, -1, 128), (codes[0], scales, 16, 128)):
        with pytest.raises(ValueError):
            mx4.untile(*args)


def test_moe_refused(fake):
    X, lg, gu, dn = f16(3, 64), torch.zeros(3, 4), pair(4 * 2 * 32, 64), pair(4 * 64, 32)
    bad = [
        dict(logits=torch.zeros(2, 4)), dict(logits=torch.zeros(3, 5)), dict(logits=torch.zeros(4, 3).T),
        dict(logits=torch.zeros(3, 4, dtype=torch.float64)), dict(logits=torch.zeros(3, 0)),
        dict(gate_up=pair(4 * 2 * 32, 192)), dict(gate_up=pair(4 * 2 * 160, 64)), dict(down=pair(4 * 48, 32)),
        dict(down=int8_pair(4 * 64, 32)), dict(gate_up=int8_pair(4 * 2 * 32, 64)), dict(down=pair(4 * 64, 144)),
        dict(out=f16(3, 48)), dict(out=f16(3, 64).bfloat16()), dict(workspace=torch.zeros(64)), dict(top_k=0),
        dict(top_k=17),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            moe.moe_layer(**{**dict(X=X, logits=lg, gate_up=gu, down=dn, top_k=2), **kw})
    a8, b8 = int8_pair(4 * 2 * 32, 64), int8_pair(4 * 64, 32)
    with pytest.raises(ValueError):
        moe.moe_layer(X, lg, a8, (b8[0], torch.zeros(4 * 48)), 2)
    assert fake.calls == []


def test_launch_makes_the_tensors_device_current(monkeypatch):
    """A tensor on another device than the current one: the call runs under its device, on its
    stream; a status other than 0 is raised."""
    seen = []

    class Tensor:
        def get_device(self):
            return 1

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            seen.append(("enter", self.index))

        def __exit__(self, *exc):
            seen.append(("exit", self.index))

    status = 0
    monkeypatch.setattr(mx4.torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(mx4.torch.cuda, "device", Device)
    monkeypatch.setattr(mx4, "_stream", lambda index: 100 + index)
    monkeypatch.setattr(mx4, "_function", lambda name: lambda *args: (seen.append((name, args)), status)[1])
    mx4._launch("mx4_quantize", Tensor(), 7, 8)
    assert seen == [("enter", 1), ("mx4_quantize", (7, 8, 101)), ("exit", 1)]
    status = 2
    with pytest.raises(binding.Int8mmError):
        mx4._launch("mx4_quantize", Tensor(), 7, 8)
    assert seen[-1] == ("exit", 1)


def test_cpu_tensors_are_refused_by_every_call(monkeypatch):
    """With the device predicate as it is: tensors in host memory, alone or all of them, never
    reach a launch."""
    launched = []
    monkeypatch.setattr(mx4, "_launch", lambda name, t, *args: launched.append(name))
    X, W, q = f16(5, 272), pair(48, 272), pair(5, 272)
    packed, bytes_ = torch.zeros((48, 144), dtype=torch.uint8), torch.zeros((48, 9), dtype=torch.uint8)
    calls = {
        "quantize": lambda: mx4.quantize(X), "prepare_weight": lambda: mx4.prepare_weight(f16(272, 48)),
        "tile_weight": lambda: mx4.tile_weight(packed, bytes_, 272),
        "dequantize": lambda: mx4.dequantize(*q, 5, 272), "dequantize, out": lambda: mx4.dequantize(*q, 5, 272, out=X),
        "matmul": lambda: mx4.matmul(X, *W), "matmul_q": lambda: mx4.matmul_q(*q, 5, 272, *W),
        "weight_only_matmul": lambda: mx4.weight_only_matmul(X, *W),
        "moe_layer": lambda: moe.moe_layer(f16(3, 64), torch.zeros(3, 4), pair(4 * 2 * 32, 64), pair(4 * 64, 32), 2),
    }
    for name, f in calls.items():
        with pytest.raises(ValueError):
            f()
        assert launched == [], name
