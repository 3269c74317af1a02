"""GPU tests of the MX4 operators against the float64 oracle.

Tolerances (derived, not fitted): quantization, its inverse and the layouts are exact. A
product's fp32 sum is rounded at most once per matrix instruction and once per wave or block
that joins it, each time by at most 2^-23 of the sum of magnitudes S (half a step, doubled
for an alignment that truncates); its output once more by half a step of its type.
"""

import numpy as np
import pytest
import torch

from int8_mixed_precision_col_amd import mx4
from oracle import mx4_oracle as ref
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

F16, B16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F16: 2.0 ** -25, B16: 2.0 ** -134}  # half the smallest subnormal


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(M, K, dtype, seed, spread=6):
    """Normal rows whose blocks have widely different magnitudes, some of them zero."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    e = torch.randint(-spread, spread + 1, (M, (K + 15) // 16), generator=g)
    x = x * torch.exp2(e.float()).repeat_interleave(16, 1)[:, :K]
    x[torch.rand((M, (K + 15) // 16), generator=g).repeat_interleave(16, 1)[:, :K] < 0.05] = 0
    return x.to(dtype).cuda()


def raw(M, K, dtype, seed, nonfinite=True):
    """Every kind of bit pattern."""
    g = torch.Generator().manual_seed(seed)
    bits = torch.randint(0, 65536, (M, K), generator=g)
    if not nonfinite:
        top = 0x7c00 if dtype == F16 else 0x7f80
        bits = torch.where((bits & top) == top, bits & ~top, bits)
    return bits.to(torch.uint16).view(torch.int16).view(dtype).cuda()


def check_sum(y, want, S, dtype, roundings):
    y = f64(y)
    bound = S * roundings * 2.0 ** -23
    bound = bound + (np.abs(want) + bound) * torch.finfo(dtype).eps / 2 + TINY[dtype]
    assert np.isfinite(y).all()
    worst = (np.abs(y - want) / bound).max()
    assert worst <= 1, worst


def oracle_pair(x):
    codes, scales = ref.mx4_quantize(f64(x))
    return ref.mx4_pack(codes), scales


def check_pair(codes, scales, x):
    """Tiled codes and scales of x against the oracle's, and zeros in all padding."""
    M, K = x.shape
    packed, bytes_ = mx4.untile(codes, scales, M, K)
    want, want_scale = oracle_pair(x)
    assert np.array_equal(bytes_.cpu().numpy(), want_scale)
    assert np.array_equal(packed.cpu().numpy(), want)
    Mp, Kp = codes.shape[0] * 16, codes.shape[1] * 128
    all_codes, _ = mx4.untile(codes, scales, Mp, Kp)
    all_scales = scales.view(codes.shape[0], -1, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(Mp, -1)
    assert int(all_codes[M:].sum()) == 0 and int(all_codes[:, 16 * ((K + 31) // 32):].sum()) == 0
    assert int(all_scales[M:].sum()) == 0 and int(all_scales[:, (K + 31) // 32:].sum()) == 0


SHAPES = [(1, 16), (1, 4096), (5, 48), (16, 128), (17, 528), (33, 1040), (3, 4112), (64, 2048)]


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize(M, K, dtype):
    announce(f"mx4.quantize {M}x{K} {dtype}")
    for x in (rows(M, K, dtype, M + K), raw(M, K, dtype, K), raw(M, K, dtype, M, False)):
        check_pair(*mx4.quantize(x), x)


@pytest.mark.parametrize("dtype", [F16, B16])
def test_quantize_every_value_under_every_maximum(dtype):
    """Each finite 16-bit value in a block whose largest magnitude has each exponent."""
    v = torch.arange(65536).to(torch.uint16).view(torch.int16).view(dtype)
    v = v[torch.isfinite(v)]
    tops = torch.exp2(torch.arange(-24, 16).double()) if dtype == F16 else torch.exp2(torch.arange(-133, 128).double())
    # for a maximum 1.5 * 2^e (2^e where that is not a value) the values around it and far below
    x = []
    mag = v.double().abs()
    for top in tops[::3].tolist():
        near = v[(mag <= 1.5 * top) & (mag >= top / 64)]
        near = near[torch.linspace(0, len(near) - 1, min(len(near), 31 * 16)).long()]
        near = torch.nn.functional.pad(near.float(), (0, -len(near) % 31)).to(dtype).view(-1, 31)
        x.append(torch.cat((torch.full((len(near), 1), top, dtype=torch.float64).to(dtype), near), 1))
    x = torch.cat(x).cuda()
    announce(f"mx4.quantize {tuple(x.shape)} {dtype}")
    check_pair(*mx4.quantize(x), x)


@pytest.mark.parametrize("dtype", [F16, B16])
def test_quantize_strided(dtype):
    big = rows(40, 1200, dtype, 3)
    for x in (big[:, 64:64 + 528], big[3:20:2, 16:1056], big[7:8, 8:56]):
        announce(f"mx4.quantize strided {tuple(x.shape)} {x.stride()}")
        check_pair(*mx4.quantize(x), x.contiguous())


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("N,K", [(16, 16), (48, 144), (272, 528), (144, 4112), (16, 2048)])
def test_prepare_weight_both_layouts(N, K, dtype):
    W = rows(N, K, dtype, N * K)
    W[N // 2, K // 2] = float("nan")
    announce(f"mx4.prepare_weight N={N} K={K} {dtype}")
    a, b = mx4.prepare_weight(W, 1), mx4.prepare_weight(W.T.contiguous(), 0)
    check_pair(*a, W)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("N,K", [(16, 16), (48, 144), (272, 528), (32, 4112)])
def test_tile_and_untile(N, K):
    W = rows(N, K, F16, N + K)
    packed, scales = (torch.from_numpy(a).cuda() for a in oracle_pair(W))
    announce(f"mx4.tile_weight N={N} K={K}")
    tiled = mx4.tile_weight(packed, scales, K)
    want = mx4.prepare_weight(W, 1)
    assert torch.equal(tiled[0], want[0]) and torch.equal(tiled[1], want[1])
    if K % 32:   # codes that a checkpoint has past K are dropped
        packed[:, -8:] = 0x77
        tiled = mx4.tile_weight(packed, scales, K)
        assert torch.equal(tiled[0], want[0])
    back = mx4.untile(*tiled, N, K)
    assert torch.equal(back[1], scales)


@pytest.mark.parametrize("dtype", [F16, B16, F32])
@pytest.mark.parametrize("M,K", [(1, 16), (5, 528), (33, 1040)])
def test_dequantize(M, K, dtype):
    """Every scale byte and code; fp16 rounds once outside its range."""
    g = torch.Generator().manual_seed(M)
    Mp, nb = (M + 15) // 16 * 16, (K + 31) // 32
    packed = torch.randint(0, 256, (Mp, 16 * nb), generator=g, dtype=torch.uint8).cuda()
    scales = torch.randint(0, 256, (Mp, nb), generator=g, dtype=torch.uint8).cuda()
    announce(f"mx4.dequantize {M}x{K} {dtype}")
    tiled = mx4.tile_weight(packed, scales, K)
    codes = np.stack((packed.cpu().numpy() & 15, packed.cpu().numpy() >> 4), -1).reshape(Mp, -1)[:, :K]
    want = torch.from_numpy(ref.mx4_values(codes, scales.cpu().numpy())[:M]).to(dtype)
    out = mx4.dequantize(*tiled, M, K, dtype).cpu()
    assert torch.equal(out.double().nan_to_num(1e300), want.double().nan_to_num(1e300))
    # into a strided window: what lies beside it stays
    wide = torch.full((M + 2, K + 32), 7.0, dtype=dtype, device="cuda")
    mx4.dequantize(*tiled, M, K, dtype, out=wide[1:M + 1, 16:K + 16])
    inside = wide[1:M + 1, 16:K + 16].cpu()
    assert torch.equal(inside.double().nan_to_num(1e300), want.double().nan_to_num(1e300))
    wide[1:M + 1, 16:K + 16] = 7.0
    assert bool((wide == 7.0).all())


def product_case(M, K, N, dtype, seed):
    x, w = rows(M, K, dtype, seed, 3), rows(N, K, dtype, seed + 1, 3)
    xv, wv = ref.mx4_round(f64(x)), ref.mx4_round(f64(w))
    return x, w, xv, wv


PRODUCTS = [(1, 16, 16), (1, 4096, 256), (3, 1040, 48), (16, 128, 16), (16, 1024, 1024), (17, 528, 272),
            (40, 2064, 144), (64, 4096, 512), (65, 144, 4112), (100, 16, 800), (256, 1024, 256), (300, 1040, 528),
            (513, 2048, 272), (1000, 640, 1296),
            # K split over few tiles: 8 of 24 quads, 5 of 16 with a short last one, 2
            (65, 12288, 272), (130, 7760, 528), (140, 8208, 4112),
            # two launches: whole waves of 256 x 256 tiles, then the rest; 128 x 256 tiles
            (2048, 272, 10000), (512, 144, 16384),
            # few rows: long K, and two and four groups of features per workgroup
            (16, 12304, 48), (40, 12304, 144), (32, 1040, 272), (64, 512, 528), (48, 1024, 8208), (33, 96, 16400),
            (17, 2048, 144), (64, 1040, 8208), (5, 272, 8208), (5, 272, 16400), (20, 272, 16400), (50, 144, 16400),
            (4, 1552, 4112), (12, 2064, 4112), (9, 1552, 8208), (30, 2064, 4112), (20, 2064, 16400)]


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M,K,N", PRODUCTS)
def test_matmul(M, K, N, dtype):
    announce(f"mx4.matmul {M}x{K}x{N} {dtype}")
    x, w, xv, wv = product_case(M, K, N, dtype, M + N)
    W = mx4.prepare_weight(w, 1)
    want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    roundings = -(-K // 128) + 32   # 32: the waves or splits that are joined
    guard = torch.full((M * N + 64,), 3.0, dtype=dtype, device="cuda")
    y = mx4.matmul(x, *W, out=guard[:M * N].view(M, N))
    check_sum(y, want, S, dtype, roundings)
    assert bool((guard[M * N:] == 3.0).all())
    q = mx4.quantize(x)
    for out_dtype in (dtype, B16 if dtype == F16 else F16):
        check_sum(mx4.matmul_q(*q, M, K, *W, dtype=out_dtype), want, S, out_dtype, roundings)
    assert torch.equal(y, mx4.matmul(x, *W))   # the same bits again


@pytest.mark.parametrize("M", [5, 30, 200])
def test_matmul_nonfinite_rows_and_columns(M):
    x, w, xv, wv = product_case(M, 528, 272, F16, 9)
    x[2, 100], w[37, 300], w[40, 527] = float("inf"), float("nan"), float("-inf")
    announce(f"mx4.matmul with non-finite blocks M={M}")
    y = mx4.matmul(x, *mx4.prepare_weight(w, 1))
    bad = torch.zeros((M, 272), dtype=torch.bool)
    bad[2], bad[:, 37], bad[:, 40] = True, True, True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert bool(torch.isfinite(y[~bad.cuda()]).all())


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M", [7, 48, 130])
def test_matmul_strided_rows(M, dtype):
    big = rows(M, 1200, dtype, 5)
    x = big[:, 80:80 + 1040]
    W = mx4.prepare_weight(rows(144, 1040, dtype, 6), 1)
    announce(f"mx4.matmul strided M={M}")
    assert torch.equal(mx4.matmul(x, *W), mx4.matmul(x.contiguous(), *W))


WEIGHT_ONLY = [(1, 16, 16), (1, 4096, 512), (2, 144, 272), (5, 528, 48), (8, 1040, 4112), (13, 8192, 272), (16, 4112, 16),
               (16, 2048, 1040), (9, 512, 8208), (3, 528, 16400), (16, 12304, 48), (16, 528, 16400),
               (2, 8208, 4112), (12, 1040, 4112), (4, 2064, 5136)]


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M,K,N", WEIGHT_ONLY)
def test_weight_only(M, K, N, dtype):
    announce(f"mx4.weight_only_matmul {M}x{K}x{N} {dtype}")
    x, w, _, wv = product_case(M, K, N, dtype, M * K + N)
    W = mx4.prepare_weight(w, 1)
    xv = f64(x)
    guard = torch.full((M * N + 64,), 3.0, dtype=dtype, device="cuda")
    y = mx4.weight_only_matmul(x, *W, out=guard[:M * N].view(M, N))
    # at most one rounding for every four products (an instruction adds eight or more)
    check_sum(y, xv @ wv.T, np.abs(xv) @ np.abs(wv).T, dtype, K // 4 + 32)
    assert bool((guard[M * N:] == 3.0).all())
    wide = torch.zeros((M, K + 24), dtype=dtype, device="cuda")
    wide[:, 8:K + 8] = x
    assert torch.equal(y, mx4.weight_only_matmul(wide[:, 8:K + 8], *W))


@pytest.mark.parametrize("dtype", [F16, B16])
def test_weight_only_scales_over_their_whole_range(dtype):
    """Random scale bytes: with fp16 X, values below 2^-23 of their row's largest power of two
    within 512 elements are off by at most 2^-25 of it."""
    M, K, N = 4, 1040, 64
    g = torch.Generator().manual_seed(1)
    packed = torch.randint(0, 256, (N, 16 * 33), generator=g, dtype=torch.uint8)
    packed[:, -8:] = 0
    scales = torch.randint(90, 165, (N, 33), generator=g, dtype=torch.uint8)
    scales[5, 3] = 255
    x = rows(M, K, dtype, 2, 1) * 2.0 ** -12
    announce(f"mx4.weight_only_matmul wide scales {dtype}")
    y = f64(mx4.weight_only_matmul(x, *mx4.tile_weight(packed.cuda(), scales.cuda(), K)).float())
    codes = np.stack((packed.numpy() & 15, packed.numpy() >> 4), -1).reshape(N, -1)[:, :K]
    wv = ref.mx4_values(codes, scales.numpy())
    assert np.isnan(y[:, 5]).all()
    wv, y = np.delete(wv, 5, 0), np.delete(y, 5, 1)
    top = np.exp2(np.delete(scales.numpy(), 5, 0).astype(np.float64) - 127).max(1)
    xv = f64(x)
    S = np.abs(xv) @ np.abs(wv).T
    flush = 2.0 ** -25 * np.abs(xv).sum(1)[:, None] * top[None] if dtype == F16 else 0.0
    bound = S * (K // 4 + 32) * 2.0 ** -23 + flush
    want = xv @ wv.T
    big = np.abs(want) > torch.finfo(dtype).max * 0.99
    bound = bound + (np.abs(want) + bound) * torch.finfo(dtype).eps / 2 + TINY[dtype]
    assert (np.abs(y - want)[~big] <= bound[~big]).all()


def test_weight_only_values_of_x_that_are_not_finite():
    x, w = rows(6, 528, B16, 1), rows(48, 528, B16, 2)
    x[1, 7], x[4, 500] = float("inf"), float("nan")
    y = mx4.weight_only_matmul(x, *mx4.prepare_weight(w, 1))
    ok = torch.isfinite(y).all(1).cpu()
    assert ok.tolist() == [True, False, True, True, False, True]


def test_streams_and_two_calls_at_once():
    x1, x2 = rows(200, 1040, F16, 1), rows(40, 1040, F16, 2)
    W = mx4.prepare_weight(rows(528, 1040, F16, 3), 1)
    want = mx4.matmul(x1, *W), mx4.matmul(x2, *W), mx4.weight_only_matmul(x2[:9], *W)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    announce("mx4 on two streams")
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = mx4.matmul(x1, *W)
        with torch.cuda.stream(s2):
            b, c = mx4.matmul(x2, *W), mx4.weight_only_matmul(x2[:9], *W)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[2])


@pytest.mark.parametrize("M,K", [(9, 1040), (40, 1040), (200, 1040), (100, 8192)])
def test_graph_capture_and_replay(M, K):
    x = rows(M, K, F16, 1)
    W = mx4.prepare_weight(rows(528, K, F16, 3), 1)
    out = torch.empty((M, 528), dtype=F16, device="cuda")
    work = mx4.make_workspace(M, K, 528)
    mx4.matmul(x, *W, workspace=work, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx4.matmul(x, *W, workspace=work, out=out)
    for seed in range(3):
        x.copy_(rows(M, K, F16, 10 + seed))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx4.matmul(x, *W))


def test_offsets_beyond_32_bits():
    """A weight of over 4 GB of codes and activations of over 4 GB: the last rows are right."""
    N, K, M = 131088, 65536, 3
    announce(f"mx4 with {N} x {K} weights")
    w = rows(32, K, B16, 1, 2)
    tail = mx4.prepare_weight(w, 1)
    codes = torch.zeros((N // 16, K // 128, 16, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((N // 16, K // 512, 64, 4), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 1 << 32
    codes[-1], scales[-1] = tail[0][1], tail[1][1]
    codes[0], scales[0] = tail[0][0], tail[1][0]
    wv = ref.mx4_round(f64(w))
    for f, m, roundings in ((mx4.matmul, M, K // 128 + 32), (mx4.matmul, 70, K // 128 + 32),
                            (mx4.weight_only_matmul, M, K // 4 + 32)):
        x = rows(m, K, B16, 2, 2)
        xv = f64(x) if f is mx4.weight_only_matmul else ref.mx4_round(f64(x))
        y = f(x, codes, scales)
        want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
        check_sum(torch.cat((y[:, :16], y[:, -16:]), 1), want, S, B16, roundings)
        assert int(torch.count_nonzero(y[:, 16:-16])) == 0
    del codes, scales
    big = torch.zeros((32784, K + 64), dtype=B16, device="cuda")
    big[-5:, :K] = rows(5, K, B16, 3)
    q = mx4.quantize(big[:, :K])
    last = mx4.quantize(big[-16:, :K])
    assert torch.equal(q[0][-1], last[0][0]) and torch.equal(q[1][-1], last[1][0])
    back = mx4.dequantize(*q, 32784, K, B16)
    assert np.array_equal(f64(back[-5:]), ref.mx4_round(f64(big[-5:, :K])))
    assert int(torch.count_nonzero(back[:-5])) == 0


def test_quantize_once_for_three_weights():
    """Q, K and V of one input: MX4 activations once, three products, the values of each."""
    x = rows(77, 1040, B16, 4)
    ws = [rows(n, 1040, B16, n) for n in (528, 144, 144)]
    q = mx4.quantize(x)
    xv = mx4.dequantize(*q, 77, 1040, F32)
    for w in ws:
        W = mx4.prepare_weight(w, 1)
        wv = mx4.dequantize(*W, w.shape[0], 1040, F32)
        a, b = f64(xv), f64(wv)
        check_sum(mx4.matmul_q(*q, 77, 1040, *W, dtype=B16), a @ b.T, np.abs(a) @ np.abs(b).T, B16, 9 + 32)


def spread_weight(N, K, seed, at_most):
    """Tiled pair and values of N rows whose blocks' powers of two lie up to 2^at_most apart: in
    every 512 elements a few blocks far above the others (row n: by n % at_most), and the others
    24 bits apart. Also the columns of the far blocks."""
    g = torch.Generator().manual_seed(seed)
    nb = (K + 31) // 32
    packed = torch.randint(0, 256, (N, 16 * nb), generator=g, dtype=torch.uint8)
    if K % 32:
        packed[:, -8:] = 0
    scales = torch.randint(100, 124, (N, nb), generator=g)
    far = torch.rand((nb,), generator=g) < 0.25
    far[0] = True
    scales[:, far] = 123 + (torch.arange(N) % at_most)[:, None]
    scales = scales.to(torch.uint8)
    codes = np.stack((packed.numpy() & 15, packed.numpy() >> 4), -1).reshape(N, -1)[:, :K]
    return mx4.tile_weight(packed.cuda(), scales.cuda(), K), ref.mx4_values(codes, scales.numpy()), \
        far.repeat_interleave(32)[:K]


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("M,K,N", [(1, 528, 128), (4, 1040, 128), (16, 2064, 112), (12, 1040, 4208), (16, 528, 16496)])
def test_weight_only_small_blocks_beside_far_larger_ones(M, K, N, dtype):
    """X is zero where the weight is largest, so that what is left of every sum comes from blocks
    far below: nothing of them is lost. (A block more than 26 powers of two below the
    largest one left takes another pass; each pass over 512 elements is one more rounding.)"""
    announce(f"mx4.weight_only_matmul spread blocks {M}x{K}x{N} {dtype}")
    W, wv, far = spread_weight(N, K, K + N, 100)
    x = rows(M, K, dtype, M, 2)
    x[:, far] = 0
    xv = f64(x)
    want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert np.abs(want).max() < 30000 and (np.abs(want) > 2.0 ** -14).mean() > 0.95
    check_sum(mx4.weight_only_matmul(x, *W), want, S, dtype, K // 4 + 32 + 10 * -(-K // 512))


def test_weight_only_subnormal_activations():
    """fp16 X down to its smallest values against weights that bring the sums back."""
    M, K, N = 5, 1040, 48
    x, w = rows(M, K, F16, 1, 2).float() * 2.0 ** -20, rows(N, K, B16, 2, 2) * 2.0 ** 16
    x = x.half()
    assert int(((x.abs() < 2.0 ** -14) & (x != 0)).sum()) > K
    W, wv, xv = mx4.prepare_weight(w, 1), ref.mx4_round(f64(w)), f64(x)
    want = xv @ wv.T
    announce("mx4.weight_only_matmul subnormal X")
    check_sum(mx4.weight_only_matmul(x, *W), want, np.abs(xv) @ np.abs(wv).T, F16, K // 4 + 32)


def test_weight_only_nan_blocks_and_values_beside_spread_blocks():
    """NaN blocks, and an infinity or a NaN in X, in rows that take several passes."""
    M, K, N = 6, 1040, 64
    W, wv, far = spread_weight(N, K, 3, 60)
    x = rows(M, K, F16, 4, 2)
    x[:, far] = 0
    near = int((~far).nonzero()[3])
    x[1, near], x[4, near] = float("inf"), float("nan")
    W[1].view(-1)[:4] = 255                    # feature 0, block 0 of the first four units
    announce("mx4.weight_only_matmul spread blocks, not finite")
    y = mx4.weight_only_matmul(x, *W).cpu()
    assert bool(torch.isnan(y[:, 0]).all())
    assert torch.isfinite(y[:, 1:]).all(1).tolist() == [True, False, True, True, False, True]
    assert not torch.isfinite(y[1]).any() and bool(torch.isnan(y[4]).all())


@pytest.mark.parametrize("M,K,N", [(3, 1040, 144), (16, 528, 48), (30, 1040, 272), (64, 2064, 144), (200, 1040, 272),
                                   (70, 8208, 144)])
def test_matmul_of_opposite_scales(M, K, N):
    """Blocks from 2^-100 to 2^100 against blocks that bring the products back: neither scale is
    applied alone. And both at an end: zeros, or infinities."""
    announce(f"mx4.matmul opposite scales {M}x{K}x{N}")
    g = torch.Generator().manual_seed(K)
    x, w = rows(M, K, B16, M, 1), rows(N, K, B16, N, 1)
    e = torch.randint(-100, 101, (K // 16 + 1,), generator=g).repeat_interleave(32)[:K].cuda()
    x, w = x * torch.exp2(e.float()).to(B16), w * torch.exp2(-e.float()).to(B16)
    xv, wv = ref.mx4_round(f64(x)), ref.mx4_round(f64(w))
    W = mx4.prepare_weight(w, 1)
    want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    check_sum(mx4.matmul(x, *W), want, S, B16, -(-K // 128) + 32)
    check_sum(mx4.matmul_q(*mx4.quantize(x), M, K, *W, dtype=B16), want, S, B16, -(-K // 128) + 32)
    if M <= 16:
        check_sum(mx4.weight_only_matmul(x, *W), f64(x) @ wv.T, np.abs(f64(x)) @ np.abs(wv).T, B16, K // 4 + 32)
    one = torch.ones((M, K), dtype=B16, device="cuda")
    for s in (-120, 120):
        v = one * 2.0 ** s
        y = mx4.matmul(v, *mx4.prepare_weight(v[:1].expand(N, K).contiguous(), 1)).float()
        assert bool((y == (0.0 if s < 0 else float("inf"))).all())
