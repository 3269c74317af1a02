"""Cases and plain forms of the microscaled 4-bit operators and of the mixture-of-experts
layer for a few tokens.

A microscaled 4-bit row ("MX4") is cut into blocks of 32 consecutive elements. A block
holds one power of two 2^s, s = floor(log2 max|x|) - 2 in [-127, 127], stored as the byte
s + 127, and 32 four-bit codes of x / 2^s: a sign and a magnitude of
{0, 0.5, 1, 1.5, 2, 3, 4, 6}, to the nearest, ties to the even code, beyond 6 to 6.

The operators, by case["op"]:
  quantize     rows of X [M, K] to MX4 and back to their values
  prepare      a weight [K, N] or [N, K] to MX4 (one row per output feature) and back
  matmul       Y [M, N] = MX4(X) . W^T with an MX4 weight
  weight_only  Y [M, N] = X . W^T with X as it is, M <= 16
  moe          routing, gate and up products, SiLU, down product and weighted sum of the
               chosen experts, int8 or MX4 weights, T <= 16 tokens
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ----

def listed():
    return [
        # one decode step's activations: latency
        dict(name="quantize 8x4096", op="quantize", M=8, K=4096, dtype="fp16"),
        # a ragged prompt of the 13B-like down projection: odd row count, a half-full last block
        dict(name="quantize 1333x20464", op="quantize", M=1333, K=20464, dtype="bf16"),
        # a weight at load, input features first: blocks run down its columns
        dict(name="prepare 4096x16384", op="prepare", K=4096, N=16384, layout=0, dtype="fp16"),
        # the smallest product: a few tokens, latency
        dict(name="matmul 16x1024x1024", op="matmul", M=16, K=1024, N=1024, dtype="fp16"),
        # odd and ragged everywhere
        dict(name="matmul 333x1040x528", op="matmul", M=333, K=1040, N=528, dtype="bf16"),
        # the 6.7B-like up projection of a prompt
        dict(name="matmul 2048x4096x16384", op="matmul", M=2048, K=4096, N=16384, dtype="fp16"),
        # one GPU's share of a 175B layer, the largest
        dict(name="matmul 4096x12288x49152", op="matmul", M=4096, K=12288, N=49152, dtype="fp16"),
        # decode with 16-bit activations: one token, and a ragged batch
        dict(name="weight_only 1x4096x4096", op="weight_only", M=1, K=4096, N=4096, dtype="bf16"),
        dict(name="weight_only 13x8192x8192", op="weight_only", M=13, K=8192, N=8192, dtype="fp16"),
        # one token through small experts: latency
        dict(name="moe 1 token int8", op="moe", T=1, D=2048, I=768, E=64, k=8, dtype="fp16",
             weights="int8", renormalize=True, masked=0.0),
        # a ragged batch with a padding token and masked experts
        dict(name="moe 5 tokens mx4 masked", op="moe", T=5, D=1040, I=528, E=10, k=3, dtype="fp16",
             weights="mx4", renormalize=False, masked=0.3),
        # a full batch over large experts: nearly every expert is read
        dict(name="moe 16 tokens mx4", op="moe", T=16, D=4096, I=1280, E=64, k=8, dtype="bf16",
             weights="mx4", renormalize=True, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "prepare", "matmul", "matmul", "weight_only", "moe", "moe"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "quantize":
        return dict(op=op, M=_log_int(rng, 1, 4096), K=16 * _log_int(rng, 1, 1280), dtype=dtype)
    if op == "prepare":
        return dict(op=op, K=16 * _log_int(rng, 1, 512), N=16 * _log_int(rng, 1, 1024),
                    layout=rng.choice([0, 1]), dtype=dtype)
    if op == "matmul":
        return dict(op=op, M=_log_int(rng, 1, 4096), K=16 * _log_int(rng, 1, 768),
                    N=16 * _log_int(rng, 1, 1024), dtype=dtype)
    if op == "weight_only":
        return dict(op=op, M=rng.randint(1, 16), K=16 * _log_int(rng, 1, 1024),
                    N=16 * _log_int(rng, 1, 1024), dtype=dtype)
    E, T = _log_int(rng, 2, 128), rng.randint(1, 16)
    return dict(op=op, T=T, D=16 * _log_int(rng, 4, 256),
                I=16 * _log_int(rng, 2, 64), E=E, k=rng.randint(1, min(E, 8)), dtype=dtype,
                weights=rng.choice(["int8", "mx4"]), renormalize=rng.random() < 0.5,
                masked=rng.choice([0.0, 0.3]) if T > 1 and E >= 8 else 0.0)


def work(case):
    """Bytes and operations of one pass: each input once, each output once."""
    c = case
    if c["op"] in ("quantize", "prepare"):
        # 16-bit values in, 4-bit codes and scales out and in again, 16-bit values out
        n = c["K"] * (c["M"] if c["op"] == "quantize" else c["N"])
        return {"bytes": 4 * n + 2 * (n / 2 + n / 32), "flops": 4 * n}
    if c["op"] in ("matmul", "weight_only"):
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": 2 * M * K + N * (K / 2 + K / 32) + 2 * M * N, "flops": 2 * M * N * K}
    T, D, I, E, k = c["T"], c["D"], c["I"], c["E"], c["k"]
    # experts that at least one of T tokens, each with k of E, is expected to choose
    experts = E * (1 - (1 - k / E) ** T)
    per = 1 if c["weights"] == "int8" else 0.5 + 1 / 32
    return {"bytes": experts * 3 * D * I * per + 4 * T * D + 4 * T * E + 8 * T * k,
            "flops": 6 * T * k * D * I}


# ---- inputs ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, M, K, dtype):
    """Hidden states of a large transformer: a normal background and, in about 0.1% of the
    features, magnitudes far above it in most rows."""
    x = torch.randn((M, K), generator=g, device="cuda")
    dims = torch.randint(0, K, (max(1, K // 1000),), generator=g, device="cuda")
    far = 15 + 10 * torch.rand((M, len(dims)), generator=g, device="cuda")
    keep = torch.rand((M, len(dims)), generator=g, device="cuda") < 0.75
    sign = torch.randint(0, 2, (M, len(dims)), generator=g, device="cuda") * 2 - 1
    x[:, dims] = torch.where(keep, far * sign, x[:, dims])
    return x.to(dtype)


def _weight(g, shape, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * 0.02).to(dtype)


def _inputs(case, seed):
    """The 16-bit tensors a case starts from: made from the seed alone."""
    g, c, dt = _gen(seed), case, DTYPES[case["dtype"]]
    if c["op"] == "quantize":
        return {"X": _activations(g, c["M"], c["K"], dt)}
    if c["op"] == "prepare":
        return {"W": _weight(g, (c["K"], c["N"]) if c["layout"] == 0 else (c["N"], c["K"]), dt)}
    if c["op"] in ("matmul", "weight_only"):
        return {"X": _activations(g, c["M"], c["K"], dt), "W": _weight(g, (c["N"], c["K"]), dt)}
    T, D, I, E = c["T"], c["D"], c["I"], c["E"]
    logits = torch.randn((T, E), generator=g, device="cuda")
    if c["masked"]:
        # experts that are off for a token, and the first token a padding row with none left
        off = torch.rand((T, E), generator=g, device="cuda") < c["masked"]
        off[0] = True
        logits = logits.masked_fill(off, -math.inf)
    return {"X": _activations(g, T, D, dt), "logits": logits,
            "W13": _weight(g, (E * 2 * I, D), dt), "W2": _weight(g, (E * D, I), dt)}


def _rows_in_parts(f, W):
    """f over row ranges of W, so that its 32-bit intermediates stay small."""
    step = max(1, (1 << 27) // W.shape[1])
    parts = [f(W[i:i + step]) for i in range(0, W.shape[0], step)]
    return tuple(torch.cat(p) for p in zip(*parts))


def _held(W, fmt):
    """A weight as a checkpoint holds it: MX4 packed codes [N, K / 2] and scale bytes
    [N, ceil(K / 32)], or int8 codes [N, K] and constants [N]."""
    if fmt == "mx4":
        return _rows_in_parts(lambda w: _pack(*_codes(w.float())), W)
    a = W.abs().amax(1).float()
    q = _rows_in_parts(lambda w: (torch.round(w.float() * 127 / w.abs().amax(1, True).float()),), W)
    return q[0].to(torch.int8), a


def prepare(case, seed):
    c, t = case, _inputs(case, seed)
    if c["op"] in ("quantize", "prepare"):
        return {"case": c, **t}
    names = ("W13", "W2") if c["op"] == "moe" else ("W",)
    state = {"case": c, "X": t["X"]}
    if c["op"] == "moe":
        state["logits"] = t["logits"]
    for n in names:
        held = _held(t.pop(n), c.get("weights", "mx4"))
        # the framework keeps a weight in its own layout from load on
        state[n] = _laid_out(held, c.get("weights", "mx4")) if own else held
    return state


def _laid_out(held, fmt):
    if fmt == "mx4":
        from int8_mixed_precision_col_amd import mx4
        return mx4.tile_weight(*held)
    from int8_mixed_precision_col_amd import binding
    return binding.tile_weight(held[0]), held[1]


# ---- one pass ----

def run(state):
    c = state["case"]
    return (_run_own if own else _run_plain)(c, state)


def _run_own(c, s):
    from int8_mixed_precision_col_amd import moe, mx4
    if c["op"] == "quantize":
        codes, scales = mx4.quantize(s["X"])
        return mx4.dequantize(codes, scales, c["M"], c["K"], s["X"].dtype)
    if c["op"] == "prepare":
        codes, scales = mx4.prepare_weight(s["W"], c["layout"])
        return mx4.dequantize(codes, scales, c["N"], c["K"], s["W"].dtype)
    if c["op"] == "matmul":
        return mx4.matmul(s["X"], *s["W"])
    if c["op"] == "weight_only":
        return mx4.weight_only_matmul(s["X"], *s["W"])
    y, ids, weights = moe.moe_layer(s["X"], s["logits"], s["W13"], s["W2"], c["k"],
                                    renormalize=c["renormalize"])
    return {"y": y, "ids": ids, "weights": weights}


def _codes(x):
    """Codes [rows, K padded to 32] (uint8, 0 .. 15) and scale bytes [rows, K / 32] of fp32 x."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 32)).view(rows, -1, 32)
    top = x.abs().amax(2)
    s = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    s = torch.where(top > 0, s, -127)
    a = torch.ldexp(x, -s.unsqueeze(2))
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0))
    code = code + 8 * torch.signbit(a)
    return code.view(rows, -1).to(torch.uint8), (s + 127).to(torch.uint8)


def _pack(code, scale):
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def _values(packed, scale):
    """fp32 values of packed codes [..., K / 2] under scale bytes [..., ceil(K / 32)]."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=packed.device)
    v = torch.stack((table[(packed & 15).int()], table[(packed >> 4).int()]), -1).flatten(-2)
    v = v.unflatten(-1, (-1, 32)) * torch.exp2(scale.float() - 127).unsqueeze(-1)
    return v.flatten(-2)


def _weight_values(held, K, fmt):
    if fmt == "mx4":
        return _values(*held)[..., :K]
    return held[0].float() * (held[1] / 127).unsqueeze(-1)


def _run_plain(c, s):
    if c["op"] == "quantize":
        return _values(*_pack(*_codes(s["X"].float())))[:, :c["K"]].to(s["X"].dtype)
    if c["op"] == "prepare":
        W = s["W"].T if c["layout"] == 0 else s["W"]
        return _values(*_pack(*_codes(W.float())))[:, :c["K"]].to(s["W"].dtype)
    X, dt = s["X"], s["X"].dtype
    if c["op"] == "matmul":
        x = _values(*_pack(*_codes(X.float())))[:, :c["K"]]
        return (x @ _weight_values(s["W"], c["K"], "mx4").T).to(dt)
    if c["op"] == "weight_only":
        return (X.float() @ _weight_values(s["W"], c["K"], "mx4").T).to(dt)
    return _moe_plain(c, s)


def _moe_plain(c, s):
    T, D, I, E, k, fmt = c["T"], c["D"], c["I"], c["E"], c["k"], c["weights"]
    logits = s["logits"]
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    on = top > -math.inf
    most = torch.where(on[:, :1], top[:, :1], 0.0)
    e = torch.exp(top - most)
    w = e / (e if c["renormalize"] else torch.exp(logits - most)).sum(1, keepdim=True).clamp(min=1e-30)
    w = torch.where(on, w, 0.0)
    pick = ids.reshape(-1)
    W13 = _weight_values([t.unflatten(0, (E, 2 * I))[pick] for t in s["W13"]], D, fmt)
    gu = torch.matmul(W13, s["X"].float().repeat_interleave(k, 0).unsqueeze(2)).squeeze(2)
    del W13
    gate, up = gu[:, :I], gu[:, I:]
    h = gate / (1 + torch.exp(-gate)) * up
    W2 = _weight_values([t.unflatten(0, (E, D))[pick] for t in s["W2"]], I, fmt)
    y = torch.matmul(W2, h.unsqueeze(2)).view(T, k, D)
    y = (y * w.unsqueeze(2)).sum(1).to(s["X"].dtype)
    return {"y": y, "ids": torch.where(on, ids, -1).to(torch.int32), "weights": w}


# ---- the definition in 64 bits ----

def _exact_values(x):
    """What the rows of x become when they are held in MX4: each block over its power of two
    is rounded half-even to the spacing of its magnitude (0.5 below 2, 1 below 4, 2 above)."""
    rows, K = x.shape
    full = torch.zeros((rows, -(-K // 32) * 32), dtype=torch.float64, device=x.device)
    full[:, :K] = x.double()
    full = full.reshape(rows, -1, 32)
    top = full.abs().max(2, keepdim=True).values
    s = torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2
    unit = torch.pow(2.0, s.clamp(-127, 127))
    a = (full / unit).abs()
    gap = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = torch.clamp(torch.round(a / gap) * gap, max=6.0)
    return (torch.sign(full) * q * unit).reshape(rows, -1)[:, :K]


def _exact_weight(W, fmt):
    """fp64 values that the weight rows are held as."""
    if fmt == "mx4":
        step = max(1, (1 << 26) // W.shape[1])
        return torch.cat([_exact_values(W[i:i + step]) for i in range(0, W.shape[0], step)])
    W = W.double()
    a = W.abs().max(1, keepdim=True).values
    return torch.round(W * 127 / a) * a / 127


def exact(case, seed):
    c, t = case, _inputs(case, seed)
    if c["op"] == "quantize":
        return _exact_values(t["X"])
    if c["op"] == "prepare":
        return _exact_values(t["W"] if c["layout"] == 1 else t["W"].T)
    if c["op"] in ("matmul", "weight_only"):
        W = _exact_weight(t.pop("W"), "mx4")
        x = _exact_values(t["X"]) if c["op"] == "matmul" else t["X"].double()
        return x @ W.T
    T, D, I, E, k = c["T"], c["D"], c["I"], c["E"], c["k"]
    W13 = _exact_weight(t.pop("W13"), c["weights"]).reshape(E, 2 * I, D)
    W2 = _exact_weight(t.pop("W2"), c["weights"]).reshape(E, D, I)
    X, logits = t["X"].double(), t["logits"].double().cpu()
    y = torch.zeros((T, D), dtype=torch.float64, device=X.device)
    weights = torch.zeros((T, k), dtype=torch.float64)
    for i in range(T):
        row = logits[i].tolist()
        live = sorted((e for e in range(E) if row[e] > -math.inf), key=lambda e: (-row[e], e))
        p = {e: math.exp(row[e] - row[live[0]]) for e in live}
        chosen = live[:k]
        norm = sum(p[e] for e in (chosen if c["renormalize"] else live))
        for j, e in enumerate(chosen):
            weights[i, j] = p[e] / norm
            g, u = (W13[e] @ X[i]).split(I)
            y[i] += weights[i, j].item() * (W2[e] @ (g * torch.sigmoid(g) * u))
    return {"y": y, "ids": None, "weights": weights.to(X.device)}
