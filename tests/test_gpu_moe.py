"""GPU tests of the mixture-of-experts layer against the float64 oracle, whose bound on what
the fp32 sums and the 16-bit hidden values can do is derived in ``mx4_oracle.moe_layer``;
the output's own rounding is half a step of its type."""

import numpy as np
import pytest
import torch

import oracle
from int8_mixed_precision_col_amd import binding, moe, mx4
from oracle import mx4_oracle as ref
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

F16, B16, F32 = torch.float16, torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def prepared(w, fmt):
    """(prepared pair, float64 values) of weight rows w."""
    if fmt == "mx4":
        return mx4.prepare_weight(w, 1), ref.mx4_round(f64(w))
    Wq, aw = binding.prepare_weight(w.half().contiguous(), 1)
    q, a = oracle.prepare_weight(w.half().cpu().numpy().T.copy())
    assert np.array_equal(binding.untile_weight(Wq, w.shape[1]).cpu().numpy(), q)
    return (Wq, aw), oracle.dequantize(q, a[:, None])


def case(T, D, I, E, dtype, fmt, seed, scale=0.05):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn((T, D), generator=g).to(dtype).cuda()
    logits = torch.randn((T, E), generator=g) * 2
    w13 = (torch.randn((E * 2 * I, D), generator=g) * scale).to(dtype).cuda()
    w2 = (torch.randn((E * D, I), generator=g) * scale).to(dtype).cuda()
    p13, v13 = prepared(w13, fmt)
    p2, v2 = prepared(w2, fmt)
    return X, logits, (p13, p2), (v13.reshape(E, 2 * I, D), v2.reshape(E, D, I))


def check(X, logits, pairs, values, k, renorm, **kw):
    dtype = X.dtype
    y, ids, w = moe.moe_layer(X, logits.cuda(), *pairs, k, renormalize=renorm, **kw)
    Y, want_ids, want_w, bound = ref.moe_layer(f64(X), f64(logits), *values, k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.abs(f64(w) - want_w).max() <= 1e-6
    tiny = 2.0 ** -25 if dtype == F16 else 2.0 ** -134
    bound = bound + (np.abs(Y) + bound) * torch.finfo(dtype).eps / 2 + tiny
    err = np.abs(f64(y) - Y)
    assert np.isfinite(err).all() and (err <= bound).all(), (err / bound).max()
    return y


@pytest.mark.parametrize("fmt", ["int8", "mx4"])
@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("T,D,I,E,k,renorm", [
    (1, 16, 16, 1, 1, True), (1, 512, 256, 8, 2, True), (5, 528, 144, 10, 3, False), (16, 1040, 528, 4, 4, True),
    (16, 256, 128, 70, 8, False), (9, 144, 48, 500, 16, True), (2, 2064, 32, 3, 1, False), (16, 128, 1040, 2, 2, False),
    (13, 640, 272, 64, 6, True),
    # X past, at and within what the first launch holds in LDS at once; long hidden rows
    (16, 4224, 32, 3, 2, True), (16, 4096, 48, 4, 2, False), (3, 12304, 32, 4, 2, True), (4, 64, 4112, 3, 2, True),
])
def test_layer(T, D, I, E, k, renorm, dtype, fmt):
    announce(f"moe T={T} D={D} I={I} E={E} k={k} {dtype} {fmt}")
    X, logits, pairs, values = case(T, D, I, E, dtype, fmt, T * D + E)
    y = check(X, logits, pairs, values, k, renorm)
    for ld in (F16, B16):
        check(X, logits.to(ld), pairs, values, k, renorm)
    assert torch.equal(y, moe.moe_layer(X, logits.cuda(), *pairs, k, renormalize=renorm)[0])


@pytest.mark.parametrize("fmt", ["int8", "mx4"])
@pytest.mark.parametrize("T,k", [(1, 4), (1, 8), (16, 8)])
def test_eight_four_and_two_waves_on_a_rows_quads(T, k, fmt):
    """33 groups of features of 4, 8 or all 24 experts, five quads a row: the first launch's
    list of steps fits its workgroups once with 8, 4 and 2 waves on a row."""
    D, I, E = 1040 if fmt == "int8" else 2064, 528, 24
    announce(f"moe T={T} D={D} I={I} E={E} k={k} {fmt}")
    X, logits, pairs, values = case(T, D, I, E, F16, fmt, 10 * T + k)
    if T > 1:
        logits[torch.arange(E) % T, torch.arange(E)] += 20  # every expert has a token
    check(X, logits, pairs, values, k, True)


@pytest.mark.parametrize("T,E,I", [(3, 4, 2064), (1, 2, 2064), (2, 2, 2048)])
def test_two_workgroups_per_cu(T, E, I):
    """Long int8 rows of few tokens: more steps than 512 workgroups take once, than 256, and as
    many as 256."""
    announce(f"moe T={T} D=3600 I={I} E={E}")
    X, logits, pairs, values = case(T, 3600, I, E, B16, "int8", T + E)
    check(X, logits, pairs, values, 2, False)


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("T,D,I,E,k", [(16, 1040, 1040, 16, 4), (4, 272, 1040, 8, 4), (9, 2048, 784, 12, 3),
                                       (16, 1024, 1024, 8, 8), (16, 16, 4112, 4, 2)])
def test_down_product_of_several_workgroups(T, D, I, E, k, dtype):
    """int8, few features and many items: two or four workgroups share 16 features."""
    announce(f"moe T={T} D={D} I={I} E={E} k={k} {dtype}")
    X, logits, pairs, values = case(T, D, I, E, dtype, "int8", T + D)
    logits[T // 2] = -float("inf")       # a padding row
    y = check(X, logits, pairs, values, k, True)
    lg = logits.cuda()
    ws = torch.full((moe.workspace_bytes(T, I, k),), 255, dtype=torch.uint8, device="cuda")
    want, alone = y.clone(), torch.zeros_like(y)
    for _ in range(3):                   # the workspace's contents do not matter
        assert torch.equal(moe.moe_layer(X, lg, *pairs, k, workspace=ws)[0], want)
        ws.fill_(85)
    off = torch.full_like(lg, -float("inf"))
    assert torch.equal(moe.moe_layer(X, off, *pairs, k, workspace=ws)[0], alone)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_layer(X, lg, *pairs, k, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        a = moe.moe_layer(X, lg, *pairs, k, workspace=ws)[0]
        b = moe.moe_layer(X, lg, *pairs, k, workspace=ws)[0]
    for _ in range(4):
        a.zero_()
        b.zero_()
        g.replay()
        eager = moe.moe_layer(X, lg, *pairs, k)[0]
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(eager, want)


@pytest.mark.parametrize("T", [7, 8, 9])
def test_many_experts_and_the_edge_of_one_token_per_wave(T):
    for E in (64, 65, 130):
        announce(f"moe T={T} D=272 I=80 E={E}")
        X, logits, pairs, values = case(T, 272, 80, E, F16, "mx4", T + E)
        check(X, logits, pairs, values, 5, True)


@pytest.mark.parametrize("fmt", ["int8", "mx4"])
def test_masks_ties_and_padding_tokens(fmt):
    X, logits, pairs, values = case(6, 272, 80, 12, F16, fmt, 1)
    inf = float("inf")
    logits[0] = -inf                    # a padding row
    logits[1, :11] = -inf               # one expert left
    logits[2] = 0.5                     # all tied
    logits[3, 4:] = logits[3, 3]        # tied in part
    logits[4] = torch.finfo(F32).min    # the lowest value is no mask
    logits[4, 7] = -inf
    logits[5, 2], logits[5, 9] = 0.0, -0.0
    logits[5, [0, 1, 3, 4, 5, 6, 7, 8, 10, 11]] = -1.0
    announce(f"moe masks {fmt}")
    for renorm in (True, False):
        y = check(X, logits, pairs, values, 4, renorm)
        assert int(torch.count_nonzero(y[0])) == 0
    logits[:] = -inf
    y, ids, w = moe.moe_layer(X, logits.cuda(), *pairs, 4)
    assert int(torch.count_nonzero(y)) == 0 and int((ids != -1).sum()) == 0 and int(torch.count_nonzero(w)) == 0


def test_padding_tokens_are_not_read():
    """What an off token's row of X holds reaches nobody's output."""
    X, logits, pairs, values = case(5, 272, 80, 8, F16, "mx4", 2)
    logits[3] = -float("inf")
    want = moe.moe_layer(X, logits.cuda(), *pairs, 2)[0]
    X[3] = float("nan")
    got = moe.moe_layer(X, logits.cuda(), *pairs, 2)[0]
    assert torch.equal(got, want) and int(torch.count_nonzero(got[3])) == 0


def test_nan_and_inf_reach_their_own_token_only():
    X, logits, pairs, values = case(6, 272, 80, 8, B16, "int8", 3)
    logits[1, 5] = float("nan")
    logits[2, 3] = float("inf")
    X[4, 100] = float("inf")
    y, ids, _ = moe.moe_layer(X, logits.cuda(), *pairs, 2)
    assert torch.isfinite(y).all(1).cpu().tolist() == [True, False, False, True, False, True]
    assert int(ids[1, 0]) == 5 and int(ids[2, 0]) == 3


@pytest.mark.parametrize("fmt", ["int8", "mx4"])
@pytest.mark.parametrize("dtype", [F16, B16])
def test_every_token_chooses_the_same_experts(dtype, fmt):
    X, logits, pairs, values = case(16, 528, 144, 6, dtype, fmt, 4)
    logits[:] = logits[0]
    announce(f"moe all tokens at the same experts {dtype} {fmt}")
    check(X, logits, pairs, values, 3, True)


def test_hidden_values_beyond_fp16():
    """|h| passes 65504 while the output stays in range: no infinity in between."""
    X, logits, pairs, values = case(3, 512, 64, 4, F16, "mx4", 5, scale=0.25)
    X *= 64
    w2 = (torch.randn((4 * 512, 64), generator=torch.Generator().manual_seed(9)) * 2.0 ** -12).half().cuda()
    p2, v2 = prepared(w2, "mx4")
    h = np.abs(np.einsum("eid,td->tei", values[0], f64(X))).max()
    assert h ** 2 > 65504
    check(X, logits, (pairs[0], p2), (values[0], v2.reshape(4, 512, 64)), 2, True)


def test_strides_workspace_out_and_guard():
    X, logits, pairs, values = case(7, 272, 80, 8, F16, "mx4", 6)
    wide = torch.zeros((7, 400), dtype=F16, device="cuda")
    wide[:, 64:336] = X
    want = check(X, logits, pairs, values, 2, True)
    guard = torch.full((7 * 272 + 64,), 3.0, dtype=F16, device="cuda")
    work = torch.randint(0, 256, (moe.workspace_bytes(7, 80, 2),), dtype=torch.uint8, device="cuda")
    y, _, _ = moe.moe_layer(wide[:, 64:336], logits.cuda(), *pairs, 2, workspace=work, out=guard[:7 * 272].view(7, 272))
    assert torch.equal(y, want) and bool((guard[7 * 272:] == 3.0).all())
    with pytest.raises(binding.Int8mmError):
        moe.moe_layer(X, logits.cuda(), *pairs, 2, workspace=work[:256])
    with pytest.raises(binding.Int8mmError):
        moe.moe_layer(X, logits.cuda(), *pairs, 9)


def test_streams_and_graph():
    X, logits, pairs, _ = case(7, 272, 80, 8, F16, "int8", 7)
    X2, logits2, pairs2, _ = case(16, 272, 80, 8, B16, "mx4", 8)
    l1, l2 = logits.cuda(), logits2.cuda()
    want = moe.moe_layer(X, l1, *pairs, 2)[0], moe.moe_layer(X2, l2, *pairs2, 3)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = moe.moe_layer(X, l1, *pairs, 2)[0]
        with torch.cuda.stream(s2):
            b = moe.moe_layer(X2, l2, *pairs2, 3)[0]
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    work = torch.empty(moe.workspace_bytes(7, 80, 2), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(X)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, ids, w = moe.moe_layer(X, l1, *pairs, 2, workspace=work, out=out)
    for seed in range(3):
        l1.copy_(torch.randn((7, 8), generator=torch.Generator().manual_seed(seed)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = moe.moe_layer(X, l1, *pairs, 2)
        assert torch.equal(out, want[0]) and torch.equal(ids, want[1]) and torch.equal(w, want[2])


def test_a_decode_step_with_the_operators_together():
    """A few tokens: router logits by the MX4 weight-only product, the layer on MX4 experts,
    its output quantized for the next product; each stage against its oracle on its own input."""
    T, D, I, E, k = 6, 528, 144, 16, 4
    X, _, pairs, values = case(T, D, I, E, B16, "mx4", 11)
    g = torch.Generator().manual_seed(12)
    router = (torch.randn((E, D), generator=g) * 0.2).to(B16).cuda()
    logits = mx4.weight_only_matmul(X, *mx4.prepare_weight(router, 1))
    y = check(X, logits.cpu(), pairs, values, k, True)
    nxt = (torch.randn((272, D), generator=g) * 0.05).to(B16).cuda()
    W = mx4.prepare_weight(nxt, 1)
    z = f64(mx4.matmul(y, *W))
    a, b = ref.mx4_round(f64(y)), ref.mx4_round(f64(nxt))
    S = np.abs(a) @ np.abs(b).T
    assert (np.abs(z - a @ b.T) <= S * (5 + 32) * 2.0 ** -23 + np.abs(a @ b.T) * 2.0 ** -8 * 1.01 + 1e-30).all()


@pytest.mark.parametrize("fmt", ["int8", "mx4"])
@pytest.mark.parametrize("T", [1, 3, 16])
def test_hidden_values_keep_their_24_bits(T, fmt):
    """Gate rows that all read X[0], up rows that read one element each, and down rows that
    subtract neighbouring hidden values, which differ in their last fp16 bit: y = silu(X[0])
    (X[1 + 2 d] - X[2 + 2 d]). What the layer rounds, with s = |silu(X[0])| and hidden values
    below 2 s: each hidden value twice by half an fp32 step (the column constant's product and
    the product with silu), so four times 2^-24 of 2 s in a difference; silu, the constants and
    the sums by a few units that both values share; Y by half a step."""
    I = 144
    D = I + 16
    X = torch.zeros((T, D))
    g = torch.Generator().manual_seed(T)
    X[:, 0] = torch.linspace(0.75, 3, T)
    even = 1 + torch.randint(0, 512, (T, I // 2), generator=g) * 2.0 ** -9
    X[:, 1:1 + I:2], X[:, 2:2 + I:2] = even + 2.0 ** -10, even
    X = X.half().cuda()
    w13, w2 = torch.zeros((2 * I, D)), torch.zeros((D, I))
    w13[:I, 0] = 1
    w13[torch.arange(I) + I, torch.arange(I) + 1] = 1
    d = torch.arange(I // 2)
    w2[d, 2 * d], w2[d, 2 * d + 1] = 1, -1
    pairs = tuple(prepared(w.half().cuda(), fmt)[0] for w in (w13, w2))
    announce(f"moe hidden values T={T} {fmt}")
    y = f64(moe.moe_layer(X, torch.zeros((T, 1), device="cuda"), *pairs, 1)[0])
    x = f64(X)
    s = x[:, :1] / (1 + np.exp(-x[:, :1]))
    h = s * x[:, 1:1 + I]
    want = h[:, 0::2] - h[:, 1::2]
    bound = 4 * 2.0 ** -24 * 2 * s + np.abs(want) * (16 * 2.0 ** -24 + 2.0 ** -11) + 2.0 ** -25
    # hidden values of 16 bits would not do
    bf = lambda a: torch.from_numpy(a).float().bfloat16().double().numpy()  # noqa: E731
    pair = bf(h) + bf(h - bf(h))
    assert (np.abs(pair[:, 0::2] - pair[:, 1::2] - want) > bound).mean() > 0.3
    assert (np.abs(y[:, :I // 2] - want) <= bound).all(), (np.abs(y[:, :I // 2] - want) / bound).max()
    assert int(np.count_nonzero(y[:, I // 2:])) == 0


def test_infinite_hidden_values_stay_infinite():
    """|h| past fp32's range: an infinity of its sign in Y, not a NaN, and only for its token."""
    D, I = 64, 32
    w13, w2 = torch.zeros((2 * I, D)), torch.zeros((D, I))
    w13[0, 0], w13[I, 1], w2[:, 0] = 1, 4, 1
    X = torch.zeros((3, D))
    X[:, 0] = 2
    X[:, 1] = torch.tensor([1.0, 3e38, -3e38])
    pairs = mx4.prepare_weight(w13.bfloat16().cuda(), 1), mx4.prepare_weight(w2.bfloat16().cuda(), 1)
    y = moe.moe_layer(X.bfloat16().cuda(), torch.zeros((3, 1), device="cuda"), *pairs, 1)[0].float().cpu()
    assert bool(torch.isfinite(y[0]).all()) and bool((y[1] == float("inf")).all()) and bool((y[2] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [F16, B16])
@pytest.mark.parametrize("T,D,I,E,k", [(1, 528, 32, 4, 2), (6, 1040, 48, 6, 3), (16, 4224, 32, 3, 2)])
def test_mx4_blocks_far_below_others(T, D, I, E, k, dtype):
    """Gate and up rows whose blocks lie up to 2^80 apart, X zero where they are largest: the
    oracle's bound, which knows no loss, holds. X in LDS and read by the waves."""
    from tests.test_gpu_mx4 import spread_weight
    announce(f"moe spread blocks T={T} D={D} I={I} E={E} {dtype}")
    X, logits, pairs, values = case(T, D, I, E, dtype, "mx4", T + D)
    W, wv, far = spread_weight(E * 2 * I, D, T + D, 80)
    X[:, far] = 0
    wv = wv.reshape(E, 2 * I, D)
    assert np.abs(np.einsum("eid,td->tei", wv, f64(X))).max() < 2000
    check(X, logits, (W, pairs[1]), (wv, values[1]), k, True)


@pytest.mark.parametrize("fmt", ["int8", "mx4"])
def test_most_experts_and_longest_lists(fmt):
    """16 tokens of 16 experts each out of 512: 256 list entries, nearly as many experts."""
    T, D, I, E, k = 16, 48, 16, 512, 16
    announce(f"moe T={T} E={E} k={k} {fmt}")
    X, logits, pairs, values = case(T, D, I, E, F16, fmt, 21)
    check(X, logits, pairs, values, k, True)
    logits[:] = -float("inf")
    logits[torch.arange(T).repeat_interleave(k), torch.arange(T * k) * 2 + 1] = 1.0  # every expert has one token
    check(X, logits, pairs, values, k, False)


def test_lists_are_optional_in_the_c_call():
    X, logits, pairs, _ = case(5, 272, 80, 8, F16, "mx4", 22)
    lg = logits.cuda()
    want = moe.moe_layer(X, lg, *pairs, 2)[0]
    y = torch.zeros_like(X)
    work = torch.empty(moe.workspace_bytes(5, 80, 2), dtype=torch.uint8, device="cuda")
    announce("moe_layer without lists")
    mx4._launch("moe_layer", X, X.data_ptr(), 5, 272, 272, 0, lg.data_ptr(), 8, 2, 2, 1, 1, pairs[0][0].data_ptr(),
                pairs[0][1].data_ptr(), pairs[1][0].data_ptr(), pairs[1][1].data_ptr(), 80, y.data_ptr(), None, None,
                work.data_ptr(), work.numel())
    assert torch.equal(y, want)


def test_on_a_stream_of_its_own_behind_the_inputs():
    """Captured twice in one graph beside an MX4 product that shares no buffer; replayed with eager
    calls of both between the replays."""
    X, logits, pairs, _ = case(9, 528, 144, 12, B16, "mx4", 23)
    lg = logits.cuda()
    W = mx4.prepare_weight((torch.randn((272, 528), generator=torch.Generator().manual_seed(1)) * 0.05).to(B16).cuda(), 1)

    def step(x):
        y = moe.moe_layer(x, lg, *pairs, 3)[0]
        return y, mx4.matmul(moe.moe_layer(y, lg, *pairs, 3)[0], *W)
    want = step(X)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(X)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step(X)
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        eager = step(X)
        torch.cuda.synchronize()
        for a, b, c in zip(got, want, eager):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_one_experts_rows_are_a_weight_of_their_own():
    """What a prompt of more than 16 tokens uses: the products on one expert's slice of the prepared
    weights, both formats, as on the expert prepared alone."""
    E, I, D, e = 4, 48, 272, 2
    g = torch.Generator().manual_seed(31)
    w13 = (torch.randn((E * 2 * I, D), generator=g) * 0.05).half().cuda()
    X = torch.randn((40, D), generator=g).half().cuda()
    part = slice(e * 2 * I // 16, (e + 1) * 2 * I // 16)
    announce("one expert's slice")
    rows_ = w13[e * 2 * I:(e + 1) * 2 * I].contiguous()
    codes, scales = mx4.prepare_weight(w13, 1)
    assert torch.equal(mx4.matmul(X, codes[part], scales[part]), mx4.matmul(X, *mx4.prepare_weight(rows_, 1)))
    Wq, aw = binding.prepare_weight(w13, 1)
    assert torch.equal(binding.mixed_matmul(X, Wq[part], aw[e * 2 * I:(e + 1) * 2 * I]),
                       binding.mixed_matmul(X, *binding.prepare_weight(rows_, 1)))
