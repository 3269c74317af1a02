"""GPU tests of the operators whose rows have weights of their own (routing, products grouped by
expert, the weighted sum back to tokens, low-rank adapters) against the float64 oracle. Bounds
are derived in ``oracle/groups_oracle.py``; the output's own rounding is half a step of its type."""

import numpy as np
import pytest
import torch

import oracle
from int8_mixed_precision_col_amd import binding, lora, moe, mx4
from oracle import groups_oracle as ref
from oracle import mx4_oracle
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

F16, B16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F16: 2.0 ** -25, B16: 2.0 ** -134}  # half the smallest subnormal


def f64(t):
    return t.detach().double().cpu().numpy()


def close(y, want, bound):
    y, eps, tiny = f64(y), torch.finfo(y.dtype).eps / 2, TINY[y.dtype]
    bound = bound + (np.abs(want) + bound) * eps + tiny
    assert y.shape == want.shape and np.isfinite(y).all()
    worst = (np.abs(y - want) / bound).max()
    assert worst <= 1, worst


def nearest(x, dtype):
    """Values of the type nearest to float64 x (below its largest)."""
    last = np.maximum(np.frexp(x)[1] - (11 if dtype == F16 else 8), -24 if dtype == F16 else -133)
    return np.ldexp(np.round(np.ldexp(x, -last)), last)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ---- routing ----

def check_route(logits, k, renorm):
    r = moe.route(logits, k, renormalize=renorm)
    ids, weights = mx4_oracle.moe_route(f64(logits), k, renorm)
    offsets, rows, slots = ref.group_order(ids, logits.shape[1])
    for got, want in ((r.ids, ids), (r.offsets, offsets), (r.rows, rows), (r.slots, slots)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)
    assert np.abs(f64(r.weights) - weights).max() <= 1e-6
    again = moe.route(logits, k, renormalize=renorm)
    assert all(torch.equal(a, b) for a, b in zip(r, again))
    return r


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 65, 4), (17, 10, 3), (63, 128, 2), (64, 129, 16), (65, 64, 8),
                                   (200, 257, 5), (1000, 512, 16), (64 * 257 + 3, 7, 2), (5000, 3, 3)])
def test_route(T, E, k):
    announce(f"route T={T} E={E} k={k}")
    x = torch.randn((T, E), generator=gen(T + E))
    x[torch.rand((T, E), generator=gen(E)) < 0.2] = -float("inf")
    if T > 1:
        x[T // 2] = -float("inf")      # a token without experts
        x[T - 1] = 1.0                 # all tied
    for dtype in (F32, F16, B16):
        check_route(x.to(dtype).cuda(), k, T % 2 == 0)


def test_route_every_token_off_and_all_to_one_expert():
    announce("route, nothing on and one expert")
    for T in (5, 300):
        r = check_route(torch.full((T, 9), -float("inf"), device="cuda"), 4, True)
        assert int(r.offsets.abs().max()) == 0 and bool((r.rows == -1).all()) and bool((r.weights == 0).all())
        x = torch.full((T, 9), -float("inf"), device="cuda")
        x[:, 4] = 1.0
        check_route(x, 3, False)


def test_route_of_nan_and_infinity():
    announce("route of NaN and +inf")
    x = torch.randn((70, 12), generator=gen(1))
    x[3, 5], x[4, 7], x[66, 0] = float("nan"), float("inf"), float("nan")
    r = moe.route(x.cuda(), 3)
    ids, _ = mx4_oracle.moe_route(x.double().numpy(), 3, True)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    for t in (3, 4, 66):
        assert bool(torch.isnan(r.weights[t]).any())


# ---- products grouped by expert ----

def weights_of(E, N, K, fmt, dtype, seed):
    """(prepared pair, values or codes and constants) of E experts' weights."""
    w = (torch.randn((E * N, K), generator=gen(seed)) * 0.05).to(dtype)
    if fmt == "mx4":
        return mx4.prepare_weight(w.cuda(), 1), mx4_oracle.mx4_round(f64(w)).reshape(E, N, K)
    q, a = oracle.prepare_weight(w.numpy().T.copy())
    return binding.prepare_weight(w.cuda(), 1), (q.reshape(E, N, K), a.reshape(E, N))


def activations(M, K, dtype, seed, outliers=2):
    x = torch.randn((M, K), generator=gen(seed))
    for j in torch.randint(0, K, (outliers,), generator=gen(seed + 1)).tolist():
        x[:, j] = 20 * torch.sign(x[:, j]) + x[:, j]
    return x.to(dtype).cuda()


def want_grouped(x, values, fmt, offsets, rows, P, gated, threshold=6.0):
    if fmt == "mx4":
        return ref.grouped_mx4(f64(x), values, offsets, rows, P, gated)
    return ref.grouped_int8(x.cpu().numpy(), *values, threshold, offsets, rows, P, gated)


def offsets_of(sizes):
    return np.concatenate(([0], np.cumsum(sizes)))


def check_grouped(x, weight, values, fmt, sizes, rows, P, gated, **kw):
    offsets = offsets_of(sizes)
    width = weight[0].shape[0] * 16 // len(sizes) // (2 if gated else 1)
    guard = torch.full((P * width + 64,), 3.0, dtype=x.dtype, device="cuda")
    y = moe.grouped_matmul(x, weight, i32(offsets), None if rows is None else i32(rows), gated,
                           out=guard[:P * width].view(P, width), **kw)
    close(y, *want_grouped(x, values, fmt, offsets, rows, P, gated))
    assert bool((guard[P * width:] == 3.0).all())
    assert int(torch.count_nonzero(y[offsets[-1]:])) == 0
    return y


GROUPED = [  # sizes, tokens, K, N
    ([1], 1, 16, 32), ([0, 1, 0], 5, 48, 32), ([3, 0, 16, 17, 1], 9, 1040, 96), ([64, 65, 63], 40, 528, 160),
    ([130, 7, 0, 129], 100, 144, 288), ([0, 0, 700, 3], 333, 272, 544), ([257, 255], 512, 656, 800),
    ([1000, 0, 13, 300], 600, 2064, 288), ([0, 0], 4, 64, 64),
]


@pytest.mark.parametrize("fmt,dtype", [("mx4", F16), ("mx4", B16), ("int8", F16)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sizes,T,K,N", GROUPED)
def test_grouped(sizes, T, K, N, gated, fmt, dtype):
    announce(f"grouped {sizes} T={T} K={K} N={N} gated={gated} {fmt} {dtype}")
    x = activations(T, K, dtype, T + K)
    weight, values = weights_of(len(sizes), N, K, fmt, dtype, K + N)
    n = sum(sizes)
    P = n + 37  # rows behind the last expert's
    rows = np.full(P, -1)
    rows[:n] = torch.randint(0, T, (n,), generator=gen(n)).numpy()
    y = check_grouped(x, weight, values, fmt, sizes, rows, P, gated)
    assert torch.equal(y, moe.grouped_matmul(x, weight, i32(offsets_of(sizes)), i32(rows), gated))  # the same bits
    # rows in order already, some of them behind the last expert's
    if n <= T:
        check_grouped(x, weight, values, fmt, sizes, None, T, gated)


@pytest.mark.parametrize("fmt", ["mx4", "int8"])
@pytest.mark.parametrize("E,n", [(64, 40), (3, 1500), (2, 64)])
def test_grouped_each_tile_shape(E, n, fmt):
    """Many experts of a few rows; many rows of few experts; both with empty experts."""
    announce(f"grouped E={E} rows={n} {fmt}")
    g = gen(E + n)
    sizes = torch.randint(0, 2 * n // E + 2, (E,), generator=g).numpy()
    x, (weight, values) = activations(50, 272, F16, n), weights_of(E, 160, 272, fmt, F16, E)
    P = int(sizes.sum())
    rows = torch.randint(0, 50, (P,), generator=g).numpy()
    check_grouped(x, weight, values, fmt, sizes, rows, P, False)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", ["mx4", "int8"])
@pytest.mark.parametrize("edge,N", [(64, 288), (128, 288), (64, 5152), (128, 5152), (256, 5152)])
def test_grouped_groups_at_the_edges_of_tiles(edge, N, fmt, gated):
    """Groups of a tile's rows, one less and one more, and twice that, beside empty ones; features past a
    whole tile, and enough of them that the means take each tile shape."""
    announce(f"grouped at {edge} rows N={N} {fmt} gated={gated}")
    sizes = [edge, 0, edge - 1, edge + 1, 2 * edge, 2 * edge - 1, 0, 2 * edge + 1]
    x, (weight, values) = activations(60, 272, F16, edge), weights_of(8, N, 272, fmt, F16, edge)
    P = sum(sizes)
    check_grouped(x, weight, values, fmt, sizes, np.arange(P) % 60, P, gated)
    off = np.full(P, -1)               # no row at all
    assert int(torch.count_nonzero(moe.grouped_matmul(x, weight, i32(offsets_of(sizes)), i32(off), gated))) == 0


@pytest.mark.parametrize("fmt,dtype", [("mx4", F16), ("mx4", B16), ("int8", F16)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("sizes,T,K,N", [([0, 700, 0, 3, 128, 801, 1], 333, 272, 8224), ([300, 0, 5, 92], 50, 1040, 16416),
                                         ([400, 129, 600], 77, 144, 10272)])
def test_grouped_large_tiles(sizes, T, K, N, gated, fmt, dtype):
    """Enough rows and features for tiles of 256 and 128 rows: partial ones, empty groups, rows behind
    the last group."""
    announce(f"grouped {sizes} T={T} K={K} N={N} gated={gated} {fmt} {dtype}")
    x, (weight, values) = activations(T, K, dtype, T + K), weights_of(len(sizes), N, K, fmt, dtype, K + N)
    n = sum(sizes)
    rows = np.full(n + 300, -1)
    rows[:n] = torch.randint(0, T, (n,), generator=gen(n)).numpy()
    y = check_grouped(x, weight, values, fmt, sizes, rows, n + 300, gated)
    assert torch.equal(y, moe.grouped_matmul(x, weight, i32(offsets_of(sizes)), i32(rows), gated))


def test_grouped_one_experts_weight_beyond_2_31_bytes():
    N, K = 139264, 32768
    announce(f"grouped mx4 with experts of {N} x {K}")
    w, x = (torch.randn((32, K), generator=gen(80)) * 0.05).half(), activations(5, K, F16, 81)
    tail = mx4.prepare_weight(w.cuda(), 1)
    codes = torch.zeros((N // 16, K // 128, 16, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((N // 16, K // 512, 64, 4), dtype=torch.uint8, device="cuda")
    codes[-2:], scales[-2:] = tail
    y = moe.grouped_matmul(x, (codes, scales), i32([0, 5]))
    want = ref.grouped_mx4(f64(x), mx4_oracle.mx4_round(f64(w))[None], [0, 5], None, 5, False)
    close(y[:, -32:], *want)
    assert int(torch.count_nonzero(y[:, :-32])) == 0


@pytest.mark.parametrize("fmt", ["mx4", "int8"])
def test_grouped_rows_out_of_range_are_zeros_and_offsets_stay_inside(fmt):
    announce(f"grouped, rows and offsets out of range, {fmt}")
    x, (weight, values) = activations(20, 144, F16, 3), weights_of(3, 64, 144, fmt, F16, 4)
    rows = np.array([0, -1, 20, 1 << 30, -(1 << 31), 19, 7, 3])
    y = check_grouped(x, weight, values, fmt, [3, 2, 3], rows, 8, False)
    assert int(torch.count_nonzero(y[1:5])) == 0
    for bad in ([0, 9, -5, 8], [8, 0, 8, 0], [-(1 << 31), 1 << 30, 1 << 30, (1 << 31) - 1], [5, 5, 2, 2]):
        guard = torch.full((8 * 64 + 64,), 3.0, dtype=F16, device="cuda")
        moe.grouped_matmul(x, weight, i32(bad), i32(rows), out=guard[:512].view(8, 64))
        torch.cuda.synchronize()
        assert bool((guard[512:] == 3.0).all())


@pytest.mark.parametrize("fmt", ["mx4", "int8"])
@pytest.mark.parametrize("E,P,N", [(3, 1500, 10272), (8, 1600, 5152), (300, 2000, 64)])
def test_grouped_offsets_that_mean_nothing_stay_inside_at_each_tile_shape(E, P, N, fmt):
    """Tiles of 256 and, int8, of 128 rows; groups over several chunks of 64: descending, overlapping and far offsets
    write nothing around Y or the workspace, and the next call is right."""
    announce(f"grouped, bad offsets, E={E} P={P} N={N} {fmt}")
    x, (weight, values) = activations(50, 272, F16, E), weights_of(E, N, 272, fmt, F16, P)
    rows, g = i32(np.arange(P) % 50), gen(E)
    need = moe.grouped_workspace_bytes(50, 272, P, E, N, int(fmt == "mx4"))
    guard, work = torch.full((P * N + 512,), 3.0, dtype=F16, device="cuda"), torch.full((need + 512,), 0xa5, dtype=torch.uint8, device="cuda")
    y, ws = guard[256:256 + P * N].view(P, N), work[256:256 + need]
    far = [-(1 << 31), (1 << 31) - 1, 1 << 30, -1]
    for bad in (np.linspace(P, 0, E + 1).astype(int), np.arange(E + 1) % 2 * P, np.arange(1, E + 2) % 2 * P,
                torch.randint(-P, 2 * P, (E + 1,), generator=g).numpy(), np.resize(far, E + 1), np.full(E + 1, P)):
        moe.grouped_matmul(x, weight, i32(bad), rows, out=y, workspace=ws)
        torch.cuda.synchronize()
        for t in (guard, work):
            assert bool((t[:256] == t[0]).all()) and bool((t[-256:] == t[0]).all())
        assert float(guard[0]) == 3.0 and int(work[0]) == 0xa5
    offsets = np.sort(np.concatenate(([0], torch.randint(0, P, (E,), generator=g).numpy())))
    moe.grouped_matmul(x, weight, i32(offsets), rows, out=y, workspace=ws)
    close(y, *want_grouped(x, values, fmt, offsets, np.arange(P) % 50, P, False))


@pytest.mark.parametrize("fmt", ["mx4", "int8"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,n", [(129, 700), (500, 300), (1024, 2300)])
def test_grouped_over_hundreds_of_experts(E, n, gated, fmt):
    announce(f"grouped over {E} experts, {n} rows, gated={gated} {fmt}")
    x, (weight, values) = activations(70, 144, F16, n), weights_of(E, 32, 144, fmt, F16, E)
    sizes = np.bincount(torch.randint(0, E, (n,), generator=gen(E)).numpy(), minlength=E)
    sizes[: E // 3] = 0
    P = int(sizes.sum())
    check_grouped(x, weight, values, fmt, sizes, np.arange(P) * 7 % 70, P, gated)


def test_grouped_nonfinite_rows_and_weights():
    announce("grouped mx4, non-finite blocks")
    x = activations(30, 272, F16, 5)
    x[4, 100] = float("inf")
    w = (torch.randn((3 * 48, 272), generator=gen(6)) * 0.05).half().cuda()
    w[48 + 5, 200] = float("nan")
    rows = np.arange(30)[::-1].copy()
    y = moe.grouped_matmul(x, mx4.prepare_weight(w, 1), i32([0, 10, 20, 30]), i32(rows))
    bad = torch.zeros((30, 48), dtype=torch.bool)
    bad[25], bad[10:20, 5] = True, True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert bool(torch.isfinite(y[~bad.cuda()]).all())


def test_grouped_int8_without_and_with_many_outliers():
    announce("grouped int8, outlier columns")
    (weight, values), rows = weights_of(3, 96, 528, "int8", F16, 8), np.arange(90) % 40
    for outliers in (0, 1, 16, 40):
        check_grouped(activations(40, 528, F16, 9, outliers), weight, values, "int8", [30, 0, 60], rows, 90, True)
    x = activations(40, 528, F16, 9, 40)
    y = moe.grouped_matmul(x, weight, i32([0, 30, 30, 80]), i32(rows), max_outliers=8)
    assert bool(torch.isnan(y[:80]).all()) and int(torch.count_nonzero(y[80:])) == 0


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M", [5, 300])
def test_gated_epilogue_at_every_size_of_the_gate(M, dtype):
    """silu(gate) up of gates and ups that are exact: eight powers of two, each in a block of its own. The result
    is within 1.23 |gate| + 7 units of 2^-24 and one rounding, or 0 where exp is above 2^126. exp is 2^p with p =
    -gate log2(e): p's rounding is up to 1 unit of p and the fp32 constant is off by 0.224 units, and an error of p
    is |gate| times as many units of exp; then the exponential instruction 2, 1 + exp 1, the reciprocal
    instruction 2, two products 2. Between -20 and -60 the ups are as large as it takes for every bit to count."""
    I, g = 16384, gen(M)
    announce(f"gated epilogue, {M} rows of {I} features {dtype}")
    mantissa = lambda: torch.randint(128, 256, (I,), generator=g).double()  # noqa: E731
    kind = torch.arange(I) % 4                          # large and negative twice, ordinary, far out
    size = torch.where(kind < 2, 20 + 40 * torch.rand(I, generator=g).double(),
                       torch.where(kind == 2, 8 * torch.rand(I, generator=g).double() + 0.01, 60 + 400 * torch.rand(I, generator=g).double()))
    gate = mantissa() * torch.exp2(torch.floor(torch.log2(size)) - 7)
    gate = torch.where((kind < 2) | (torch.rand(I, generator=g) < 0.5), -gate, gate)
    silu = gate / (1 + torch.exp(-gate))
    lift = torch.where(kind < 2, -torch.floor(torch.log2(silu.abs())), 0.0) + torch.randint(-6, 7, (I,), generator=g)
    up = mantissa() * torch.exp2(lift - 7)
    w = torch.zeros((2 * I, 8, 32), dtype=torch.float64)
    for half, v in ((0, gate), (I, up)):
        whole = (v.abs() / torch.exp2(torch.floor(torch.log2(v.abs())) - 7)).long()
        for b in range(8):
            w[half:half + I, b, 0] = (whole >> b & 1) * torch.exp2(torch.floor(torch.log2(v.abs())) - 7 + b) * torch.sign(v)
    x = torch.zeros((M, 8, 32), dtype=dtype)
    x[:, :, 0] = 1
    weight = mx4.prepare_weight(w.view(2 * I, 256).to(B16).cuda(), 1)
    y = moe.grouped_matmul(x.view(M, 256).cuda(), weight, i32([0, M]), gated=True)
    want = (silu * up).numpy()[None]
    gone = (gate < -126 * np.log(2) + 1e-4).numpy()     # the reciprocal instruction has no result below 2^-126: 0
    bound = np.abs(want) * np.where(gone, 1, (1.23 * gate.abs().numpy() + 7.01) * ref.U)
    close(y[:1], want, bound)
    got = f64(y[:1])                                    # and no other value than the two ends' roundings allow
    assert ((nearest(want - bound, dtype) <= got) & (got <= nearest(want + bound, dtype))).all()
    assert torch.equal(y, y[:1].expand(M, I))


@pytest.mark.parametrize("fmt", ["mx4", "int8"])
@pytest.mark.parametrize("E,n,N,K,gated", [(3, 90, 96, 528, False), (64, 500, 64, 144, True), (3, 1500, 10272, 272, False)])
def test_grouped_in_a_workspace_of_the_callers(E, n, N, K, gated, fmt):
    """Exactly as large as the helper says, filled with anything, nothing written around it."""
    announce(f"grouped in a workspace, E={E} rows={n} N={N} K={K} {fmt}")
    x, (weight, _) = activations(40, K, F16, n), weights_of(E, N, K, fmt, F16, E)
    off, rows = i32(np.arange(E + 1) * n // E), i32(np.arange(n) % 40)
    need = moe.grouped_workspace_bytes(40, K, n, E, N, int(fmt == "mx4"))
    guard = torch.full((need + 512,), 0xa5, dtype=torch.uint8, device="cuda")
    y = moe.grouped_matmul(x, weight, off, rows, gated, workspace=guard[256:256 + need])
    assert torch.equal(y, moe.grouped_matmul(x, weight, off, rows, gated))
    assert bool((guard[:256] == 0xa5).all()) and bool((guard[256 + need:] == 0xa5).all())


@pytest.mark.parametrize("dtype", [F16, B16])
def test_grouped_strided_rows(dtype):
    announce(f"grouped mx4, strided X {dtype}")
    big = activations(70, 400, dtype, 10)
    x = big[:, 64:64 + 272]
    weight, _ = weights_of(4, 64, 272, "mx4", dtype, 11)
    off, rows = i32([0, 20, 20, 90, 100]), i32(np.arange(100) % 70)
    assert torch.equal(moe.grouped_matmul(x, weight, off, rows), moe.grouped_matmul(x.contiguous(), weight, off, rows))


# ---- back to tokens ----

@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("T,k,D", [(1, 1, 16), (7, 3, 1040), (33, 16, 4112), (200, 8, 2048), (5, 2, 48), (9, 11, 8208)])
def test_combine(T, k, D, dtype):
    announce(f"combine T={T} k={k} D={D} {dtype}")
    n = max(1, T * k - 3)
    p = torch.randn((n, D), generator=gen(T)).to(dtype)
    p[0] = float("nan")                # a row that no token has
    slots = torch.randint(1 if n > 1 else 0, n, (T, k), generator=gen(k)) if n > 1 else torch.full((T, k), -1)
    slots[torch.rand((T, k), generator=gen(D)) < 0.2] = -1
    slots[0, 0] = n                    # past the last row
    w = torch.randn((T, k), generator=gen(2))
    y = moe.combine(p.cuda(), slots.int().cuda(), w.cuda())
    close(y, *ref.combine(f64(p), slots.numpy(), w.double().numpy()))


@pytest.mark.parametrize("T", [(1 << 24) - 1, 1 << 24])
def test_combine_of_as_many_tokens_as_there_may_be(T):
    announce(f"combine T={T}")
    p = torch.randn((1000, 16), generator=gen(4)).half().cuda()
    slots = (torch.arange(T, dtype=torch.int32, device="cuda") * 7 % 1003).view(T, 1)   # 1000 .. 1002: no row
    w = torch.ones((T, 1), device="cuda")
    y = moe.combine(p, slots, w)
    want = torch.cat((p, torch.zeros((3, 16), dtype=F16, device="cuda")))
    for part in range(0, T, 1 << 22):
        at = slots[part:part + (1 << 22), 0].long()
        assert torch.equal(y[part:part + (1 << 22)], want[at])


# ---- the layer ----

@pytest.mark.parametrize("fmt,dtype", [("mx4", F16), ("mx4", B16), ("int8", F16)])
@pytest.mark.parametrize("T,D,I,E,k", [(1, 64, 32, 3, 2), (37, 272, 144, 10, 3), (300, 528, 272, 5, 2)])
def test_layer(T, D, I, E, k, fmt, dtype):
    """The parts after each other, each against the oracle on what the one before gave, and
    moe_prompt the same bits."""
    announce(f"moe_prompt T={T} D={D} I={I} E={E} k={k} {fmt} {dtype}")
    x = activations(T, D, dtype, T)
    gu, gu_values = weights_of(E, 2 * I, D, fmt, dtype, D)
    dn, dn_values = weights_of(E, D, I, fmt, dtype, I)
    logits = torch.randn((T, E), generator=gen(E))
    logits[torch.rand((T, E), generator=gen(k)) < 0.3] = -float("inf")
    logits[0] = -float("inf")          # a padding row
    r = check_route(logits.cuda(), k, True)
    offsets, rows = r.offsets.cpu().numpy(), r.rows.cpu().numpy()
    h = moe.grouped_matmul(x, gu, r.offsets, r.rows, gated=True)
    close(h, *want_grouped(x, gu_values, fmt, offsets, rows, T * k, True))
    p = moe.grouped_matmul(h, dn, r.offsets)
    close(p, *want_grouped(h, dn_values, fmt, offsets, None, T * k, False))
    y = moe.combine(p, r.slots, r.weights)
    close(y, *ref.combine(f64(p), r.slots.cpu().numpy(), f64(r.weights)))
    assert int(torch.count_nonzero(y[0])) == 0
    whole, ids, weights = moe.moe_prompt(x, logits.cuda(), gu, dn, k)
    assert torch.equal(whole, y) and torch.equal(ids, r.ids) and torch.equal(weights, r.weights)


# ---- adapters ----

def lora_case(M, K, N, R, S, dtype, seed, ranked):
    g = gen(seed)
    t = dict(Y=torch.randn((M, N), generator=g).to(dtype), X=torch.randn((M, K), generator=g).to(dtype),
             A=(torch.randn((S, R, K), generator=g) / K ** 0.5).to(dtype),
             B=(torch.randn((S, N, R), generator=g) / R ** 0.5).to(dtype),
             ids=torch.randint(-1, S, (M,), generator=g).int(), scales=torch.randn(S, generator=g), ranks=None)
    if ranked:
        t["ranks"] = torch.randint(0, R + 1, (S,), generator=g).int()
        t["ranks"][0] = 0
        for a in range(S):             # what lies beyond a rank is not looked at
            t["A"][a, t["ranks"][a]:] = float("nan")
            t["B"][a, :, t["ranks"][a]:] = float("inf")
    return {k: v if v is None else v.cuda() for k, v in t.items()}


def want_lora(t):
    return ref.lora(f64(t["Y"]), f64(t["X"]), np.nan_to_num(f64(t["A"])), f64(t["B"]), t["ids"].cpu().numpy(),
                    None if t["scales"] is None else f64(t["scales"]),
                    None if t["ranks"] is None else t["ranks"].cpu().numpy(), t["X"].dtype == B16)


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M,K,N,R,S", [
    (1, 16, 16, 8, 1), (1, 4096, 272, 16, 3), (8, 1040, 528, 16, 20), (17, 144, 4112, 24, 2), (64, 528, 144, 64, 5),
    (65, 528, 144, 64, 5), (64, 2064, 48, 128, 64), (200, 272, 1040, 40, 1), (333, 1040, 528, 72, 9),
    (1000, 144, 80, 104, 1000), (700, 4112, 272, 96, 3), (2050, 64, 64, 8, 2), (130, 48, 16, 120, 1024)])
def test_lora(M, K, N, R, S, dtype):
    announce(f"lora M={M} K={K} N={N} R={R} S={S} {dtype}")
    for ranked in (False, True):
        t = lora_case(M, K, N, R, S, dtype, M + K + ranked, ranked)
        guard = torch.full((M * N + 64,), 3.0, dtype=dtype, device="cuda")
        y = lora.apply(**t, out=guard[:M * N].view(M, N))
        close(y, *want_lora(t))
        assert bool((guard[M * N:] == 3.0).all())
        none = (t["ids"] < 0).nonzero().squeeze(1)
        assert torch.equal(y[none], t["Y"][none])
        assert torch.equal(y, lora.apply(**t))                       # the same bits
        inplace = t["Y"].clone()
        assert lora.apply(**{**t, "Y": inplace}, out=inplace) is inplace and torch.equal(inplace, y)
    t["scales"] = None
    close(lora.apply(**t), *want_lora(t))


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("ranked", [False, True])
@pytest.mark.parametrize("M,K,N,R,S", [
    (65, 4112, 272, 8, 1), (200, 4608, 1040, 72, 2), (300, 4112, 528, 128, 3),     # K in 8 parts
    (700, 2576, 272, 24, 9),                                                       # in 5, tiles for each XCD
    (1500, 1040, 144, 104, 40), (2100, 1552, 272, 64, 6), (4000, 2064, 144, 24, 100),  # in 2, 3 and 1
])
def test_lora_many_rows_in_parts(M, K, N, R, S, dtype, ranked):
    """Beyond 64 rows: K in few and in many parts, one step of a wave and several, a last step past K's
    end, tiles that do not divide by the XCDs."""
    announce(f"lora {M} x {K} x {N} rank {R} of {S} {dtype} ranked={ranked}")
    t = lora_case(M, K, N, R, S, dtype, M + R, ranked)
    y = lora.apply(**t)
    close(y, *want_lora(t))
    assert torch.equal(y, lora.apply(**t))


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M,R,S,ranked", [(1, 8, 1, False), (9, 24, 2, True), (30, 48, 1, False), (64, 128, 3, True),
                                          (65, 16, 2, False), (200, 56, 3, True), (130, 88, 1, True), (700, 128, 4, False)])
def test_lora_keeps_all_of_a_sum(M, R, S, ranked, dtype):
    """V of 24 bits whose first nine cancel between two ranks: whole numbers below 2^24 all along (V, its parts, and
    the sums of one rank less another), so bf16 has one rounding, the output's. Two fp16 parts leave out at most
    one unit of a number below 2^24 (11 bits, and 11 of the 12 of what they leave), so 1 each of two ranks."""
    announce(f"lora of 24-bit sums M={M} R={R} S={S} {dtype} ranked={ranked}")
    g, K, N = gen(M + R), 48, 80
    whole = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=g)  # noqa: E731
    X, A = whole(-127, 127, M, K), whole(0, 1, S, R, K) * 2 - 1
    X[:, 0] = (whole(64, 126, M) << 7) * (whole(0, 1, M) * 2 - 1)
    A[:, :, 0], A[:, :, 1] = 1 << 10, whole(-127, 127, S, R)   # V: 64 .. 126 times 2^17, and up to 173 * 127 beside it
    ranks = whole(2, R, S) if ranked else torch.full((S,), R)
    B = torch.zeros((S, N, R), dtype=torch.int64)
    for a in range(S):
        for n in range(N):
            i, j = torch.randperm(int(ranks[a]), generator=g)[:2].tolist()
            B[a, n, i], B[a, n, j] = 1, -1
    Y, ids = whole(-64, 64, M, N), whole(0, S - 1, M)
    V = torch.einsum("mk,mrk->mr", X, A[ids])
    assert int(V.abs().min()) > 1 << 22 and int(V.abs().max()) < 1 << 24
    want = (Y + torch.einsum("mr,mnr->mn", V, B[ids])).double().numpy()
    t = [v.to(dtype) for v in (Y, X, A, B)]
    assert all(torch.equal(a.long(), b) for a, b in zip(t, (Y, X, A, B)))
    got = lora.apply(*(v.cuda() for v in t), ids.int().cuda(), ranks=ranks.int().cuda() if ranked else None)
    close(got, want, np.full(want.shape, 2.0 if dtype == F16 else 0.0))


@pytest.mark.parametrize("M", [3, 90])
def test_lora_the_largest_sum_in_bf16(M):
    """V of fp32's largest value, 2^128 - 2^104, whose rounding to 8 bits would be infinite: brought down by B
    it is 2^108 - 2^84, which rounds to 2^108."""
    announce(f"lora, V of 2^128 - 2^104, M={M}")
    X = torch.zeros((M, 32), dtype=B16)
    X[:, :24] = torch.exp2(127.0 - torch.arange(24)).to(B16)
    A, B = torch.ones((1, 8, 32), dtype=B16), torch.zeros((1, 48, 8), dtype=B16)
    B[0, :, 5] = 2.0 ** -20
    got = lora.apply(torch.zeros((M, 48), dtype=B16, device="cuda"), X.cuda(), A.cuda(), B.cuda(),
                     torch.zeros(M, dtype=torch.int32, device="cuda"))
    assert bool((got == 2.0 ** 108).all())


@pytest.mark.parametrize("M", [3, 90])
def test_lora_small_values_beside_a_large_one_in_fp16(M):
    """A value of V far below its row's largest is off by at most 2^-39 of the largest."""
    announce(f"lora, V from 2^-10 to 2^30, M={M}")
    X, A, B = torch.zeros((M, 16)), torch.zeros((1, 16, 16)), torch.zeros((1, 32, 16))
    X[:, 0], X[:, 1] = 2.0 ** 15, (1024 + torch.arange(M) % 1024) * 2.0 ** -15
    A[0, 0, 0] = 2.0 ** 15
    small = torch.arange(1, 16)
    A[0, small, 1] = torch.exp2(5.0 - small)            # V: 2^30, and 11 bits from 1 down to 2^-14
    B[0, small, small] = 1.0
    got = lora.apply(torch.zeros((M, 32), dtype=F16, device="cuda"), X.half().cuda(), A.half().cuda(), B.half().cuda(),
                     torch.zeros(M, dtype=torch.int32, device="cuda"))
    want = (X.double() @ A[0].double().T) @ B[0].double().T
    assert float(want.max()) < 2 and float(want[:, 1:16].min()) > 0
    close(got, want.numpy(), np.full(want.shape, 2.0 ** -9))


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M", [1, 40, 150])
def test_lora_strided_and_ids_out_of_range(M, dtype):
    announce(f"lora strided M={M} {dtype}")
    t = lora_case(M, 272, 144, 16, 4, dtype, M, False)
    t["ids"][M // 2] = 4
    t["ids"][0] = -(1 << 31)
    t["ids"][M - 1] = 1 << 30
    want = lora.apply(**t)
    assert torch.equal(want[M // 2], t["Y"][M // 2]) and torch.equal(want[M - 1], t["Y"][M - 1])
    xb, yb, ob = (torch.full((M, w), float("nan"), dtype=dtype, device="cuda") for w in (400, 200, 176))
    xb[:, 64:336], yb[:, 8:152] = t["X"], t["Y"]
    got = lora.apply(**{**t, "X": xb[:, 64:336], "Y": yb[:, 8:152]}, out=ob[:, 16:160])
    assert torch.equal(got, want)
    assert bool(torch.isnan(ob[:, :16]).all()) and bool(torch.isnan(ob[:, 160:]).all())


@pytest.mark.parametrize("M,K,R,S", [(1, 16, 8, 1), (9, 1040, 24, 3), (64, 528, 128, 7), (65, 4112, 72, 2), (700, 272, 40, 20)])
def test_lora_in_a_workspace_of_the_callers(M, K, R, S):
    """Exactly as large as the helper says, filled with anything, nothing written around it."""
    announce(f"lora in a workspace, M={M} K={K} R={R} S={S}")
    t = lora_case(M, K, 144, R, S, B16, M, True)
    need = lora.workspace_bytes(M, K, S, R)
    guard = torch.full((need + 512,), 0xa5, dtype=torch.uint8, device="cuda")
    assert torch.equal(lora.apply(**t, workspace=guard[256:256 + need]), lora.apply(**t))
    assert bool((guard[:256] == 0xa5).all()) and bool((guard[256 + need:] == 0xa5).all())


@pytest.mark.parametrize("M", [5, 100])
def test_lora_wide_ranges_in_fp16(M):
    """V's rows far above and below what fp16 holds: each has a power of two of its own."""
    announce(f"lora, rows of very different sizes, M={M}")
    t = lora_case(M, 1040, 272, 32, 2, F16, M, False)
    t["ids"] = (torch.arange(M) % 2).int().cuda()
    t["X"] = (t["X"].float() * torch.exp2((torch.arange(M) % 25 - 14).float()).cuda()[:, None]).half()
    t["A"] = (t["A"].float() * 256).half()
    t["B"] = (t["B"].float() / 4096).half()
    close(lora.apply(**t), *want_lora(t))


def test_lora_of_rows_that_are_not_finite():
    announce("lora, rows with NaN and infinities")
    for M in (6, 90):
        t = lora_case(M, 272, 144, 16, 3, F16, M, False)
        t["ids"].fill_(1)
        want = lora.apply(**t)
        t["X"][2, 5], t["X"][4, 271] = float("nan"), float("inf")
        got = lora.apply(**t)
        bad = torch.zeros(M, dtype=torch.bool)
        bad[2] = bad[4] = True
        assert bool(torch.isnan(got[bad.cuda()]).all()) and torch.equal(got[~bad.cuda()], want[~bad.cuda()])


@pytest.mark.parametrize("dtype", [F16, B16])
def test_lora_whole_batch_of_one_adapter_and_of_none(dtype):
    announce(f"lora, one adapter and none, {dtype}")
    for M in (33, 64, 640):
        t = lora_case(M, 528, 272, 32, 2, dtype, M, False)
        t["ids"].fill_(1)
        close(lora.apply(**t), *want_lora(t))
        t["ids"].fill_(-1)
        assert torch.equal(lora.apply(**t), t["Y"])


def test_lora_many_rows_and_offsets_beyond_32_bits():
    """Over 4 GB of X and of Y: the last rows are right, and rows far apart share a tile."""
    M, K, N = 140000, 16384, 16400
    announce(f"lora M={M} K={K} N={N}")
    Y, X = (torch.zeros((M, w), dtype=B16, device="cuda") for w in (N, K))
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    pick = [0, 1, M // 2, M - 2, M - 1]
    small = lora_case(5, K, N, 16, 2, B16, 7, False)
    X[pick], Y[pick] = small["X"], small["Y"]
    small["ids"] = torch.tensor([1, 0, 1, 0, 1], dtype=torch.int32, device="cuda")
    ids[pick] = small["ids"]
    got = lora.apply(Y, X, small["A"], small["B"], ids, scales=small["scales"], out=Y)
    close(got[pick], *want_lora(small))
    assert int(torch.count_nonzero(got)) <= 5 * N


# ---- streams, graphs, large operands ----

def test_streams_and_calls_at_once():
    announce("grouped operators on two streams")
    x = activations(300, 528, F16, 20)
    gu, _ = weights_of(6, 288, 528, "mx4", F16, 21)
    dn, _ = weights_of(6, 528, 144, "mx4", F16, 22)
    logits = torch.randn((300, 6), generator=gen(23)).cuda()
    t = lora_case(200, 272, 528, 16, 5, F16, 24, False)
    want = moe.moe_prompt(x, logits, gu, dn, 2)[0], lora.apply(**t)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = moe.moe_prompt(x, logits, gu, dn, 2)[0]
        with torch.cuda.stream(s2):
            b, c = lora.apply(**t), moe.moe_prompt(x, logits, gu, dn, 2)[0]
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[0])


@pytest.mark.parametrize("fmt", ["mx4", "int8"])
@pytest.mark.parametrize("T", [20, 150])
def test_graph_capture_and_replay(T, fmt):
    """The layer and adapters beside it in one graph, with routing that changes between replays."""
    announce(f"graph T={T} {fmt}")
    x, logits = activations(T, 272, F16, 30), torch.randn((T, 6), generator=gen(31)).cuda()
    gu, _ = weights_of(6, 288, 272, fmt, F16, 32)
    dn, _ = weights_of(6, 272, 144, fmt, F16, 33)
    t = lora_case(T, 272, 272, 16, 5, F16, 34, False)
    t["X"] = x

    def step():
        y = moe.moe_prompt(x, logits, gu, dn, 3)[0]
        return y, lora.apply(**{**t, "Y": y})
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for seed in range(4):
        x.copy_(activations(T, 272, F16, 40 + seed))
        logits.copy_(torch.randn((T, 6), generator=gen(50 + seed)).cuda())
        logits[seed] = -float("inf")
        t["ids"].copy_(torch.randint(-1, 5, (T,), generator=gen(60 + seed)).int())
        for o in got:
            o.zero_()
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_route_of_as_many_tokens_as_there_may_be():
    T, E, k = 1 << 24, 3, 2
    announce(f"route T={T}")
    x = torch.randn((T, E), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    x[::5, 1] = -float("inf")
    x[::35] = -float("inf")
    r = moe.route(x, k)
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    ids = torch.where(top > -float("inf"), ids, E)[:, :k].reshape(-1)
    key, order = torch.sort(ids, stable=True)
    n = int((key < E).sum())
    assert torch.equal(r.ids.view(-1).long(), torch.where(ids < E, ids, -1))
    assert torch.equal(r.offsets.long(), torch.searchsorted(key, torch.arange(E + 1, device="cuda")))
    assert torch.equal(r.rows[:n].long(), order[:n] // k) and bool((r.rows[n:] == -1).all())
    slots = torch.full((T * k,), -1, device="cuda")
    slots[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(r.slots.view(-1).long(), slots)


@pytest.mark.parametrize("fmt", ["mx4", "int8"])
def test_grouped_of_as_many_rows_as_there_may_be(fmt):
    """2^24 rows of Y, and as many of X: each as in a product of a few."""
    P = 1 << 24
    announce(f"grouped P={P} {fmt}")
    x, (weight, values) = activations(8, 16, F16, 90, 0), weights_of(3, 16, 16, fmt, F16, 91)
    small = torch.cat([moe.grouped_matmul(x, weight, i32([8 * (i > e) for i in range(4)])) for e in range(3)])
    close(small, *want_grouped(x, values, fmt, [0, 8, 16, 24], np.arange(24) % 8, 24, False))
    offsets = [0, 100, (1 << 23) + 1, P - 9]
    at = torch.arange(P, device="cuda")
    want = small[(at >= offsets[1]) * 8 + (at >= offsets[2]) * 8 + at % 8]
    want[offsets[3]:] = 0
    many = x.repeat(P // 8, 1)
    for got in (moe.grouped_matmul(x, weight, i32(offsets), (at % 8).int()), moe.grouped_matmul(many, weight, i32(offsets))):
        assert torch.equal(got, want)


def test_lora_of_as_many_rows_as_there_may_be():
    M = 1 << 24
    announce(f"lora M={M}")
    t = lora_case(4096, 16, 16, 8, 2, B16, 92, False)
    want = lora.apply(**t)
    close(want, *want_lora(t))
    big = {n: v.repeat(M // 4096, *[1] * (v.dim() - 1)) if n in ("X", "Y", "ids") else v for n, v in t.items()}
    got = lora.apply(**big)
    assert torch.equal(got.view(-1, 4096, 16), want.expand(M // 4096, 4096, 16))


def test_grouped_offsets_beyond_32_bits():
    """Over 4 GB of expert weights and over 4 GB of outputs: the last expert's rows are right."""
    E, N, K = 1024, 4112, 2048
    announce(f"grouped mx4 with {E} x {N} x {K} weights")
    codes = torch.zeros((E * N // 16, K // 128, 16, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((E * N // 16, K // 512, 64, 4), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 1 << 32
    w, values = weights_of(1, N, K, "mx4", B16, 70)
    codes[-(N // 16):], scales[-(N // 16):] = w
    x = activations(4, K, B16, 71)
    n = 700000
    offsets = np.concatenate((np.zeros(E), [n]))
    rows = np.arange(n) % 4
    y = moe.grouped_matmul(x, (codes, scales), i32(offsets), i32(rows))
    assert y.numel() > 1 << 31
    close(y[-4:], *ref.grouped_mx4(f64(x), values, [0, 4], None, 4, False))
    assert torch.equal(y[:4], y[-4:]) and torch.equal(y[n // 2:n // 2 + 4], y[-4:])
