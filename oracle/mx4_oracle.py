"""CPU oracle for the microscaled 4-bit operators and the mixture-of-experts layer.

TEST INFRASTRUCTURE, with the same standing as ``int8mm_oracle``: plain numpy in float64,
sharing no code with the HIP library or its binding. Values are passed as float64 arrays
that hold exact fp16 / bf16 / fp32 numbers.
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize(x: np.ndarray):
    """float64 [R, K] -> codes uint8 [R, K] (0 .. 15) and scale bytes uint8 [R, ceil(K / 32)]."""
    R, K = x.shape
    nb = (K + 31) // 32
    full = np.zeros((R, nb * 32))
    full[:, :K] = x
    blocks = full.reshape(R, nb, 32)
    bad = ~np.isfinite(blocks).all(2)
    clean = np.where(bad[..., None], 0.0, blocks)
    top = np.abs(clean).max(2)
    exponent = np.frexp(np.where(top > 0, top, 1.0))[1] - 1          # floor(log2 top)
    s = np.where(top > 0, np.clip(exponent - 2, -127, 127), -127)
    a = np.abs(clean) / np.exp2(s.astype(np.float64))[..., None]
    # nearest grid value; at a midpoint the even index; past the last one the last
    hi = np.clip(np.searchsorted(GRID, a, side="left"), 1, 7)
    lo = hi - 1
    mid = (GRID[lo] + GRID[hi]) / 2
    code = np.where(a > mid, hi, np.where(a < mid, lo, np.where(lo % 2 == 0, lo, hi)))
    code = code + 8 * np.signbit(clean)
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    byte = np.where(bad, 255, s + 127).astype(np.uint8)
    return code.reshape(R, -1)[:, :K], byte


def mx4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of codes [R, K] under scale bytes [R, ceil(K / 32)]."""
    K = codes.shape[1]
    unit = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(unit, 32, axis=1)[:, :K]


def mx4_pack(codes: np.ndarray) -> np.ndarray:
    """codes [R, K] -> packed uint8 [R, 16 ceil(K / 32)]."""
    R, K = codes.shape
    full = np.zeros((R, (K + 31) // 32 * 32), np.uint8)
    full[:, :K] = codes
    return full[:, 0::2] | (full[:, 1::2] << 4)


def mx4_round(x: np.ndarray) -> np.ndarray:
    """The values that rows of x become in MX4."""
    return mx4_values(*mx4_quantize(x))


def moe_route(logits: np.ndarray, top_k: int, renormalize: bool):
    """(ids [T, top_k], weights [T, top_k]); -inf is off, ties go to the lowest index."""
    T, E = logits.shape
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        row = logits[t]
        key = np.where(np.isnan(row), np.inf, row)
        order = [e for e in np.lexsort((np.arange(E), -key, ~np.isnan(row))) if row[e] != -np.inf]
        if not order:
            continue
        with np.errstate(invalid="ignore"):
            p = np.exp(row - row[order[0]])
        chosen = order[:top_k]
        norm = p[chosen].sum() if renormalize else p[order].sum()
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = p[chosen] / norm
    return ids, weights


def moe_layer(X, logits, gate_up, down, top_k, renormalize):
    """X [T, D], gate_up values [E, 2 I, D], down values [E, D, I] -> (Y, ids, weights, bound):
    bound [T, D] is what rounding the sums in fp32, keeping the hidden values to 16 bits and
    evaluating the weights and SiLU in fp32 can move Y by, before Y's own rounding."""
    T, D = X.shape
    I = down.shape[2]
    u = 2.0 ** -24
    ids, weights = moe_route(logits, top_k, renormalize)
    Y, bound = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j in range(top_k):
            e = ids[t, j]
            if e < 0:
                continue
            g, up = np.split(gate_up[e] @ X[t], 2)
            sg, su = np.split(np.abs(gate_up[e]) @ np.abs(X[t]), 2)
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            h = silu * up
            # fp32 sums of D terms in at most D / 4 + 32 roundings; |silu'| <= 1.1; a few
            # units of fp32 for exp and the quotient; 16 significant bits for h
            n = D / 4 + 32
            dh = 1.1 * n * u * sg * np.abs(up) + np.abs(silu) * n * u * su + np.abs(h) * (2.0 ** -16 + 8 * u)
            a = np.abs(down[e])
            y = down[e] @ h
            Y[t] += weights[t, j] * y
            # the weight itself: exp of a difference and a quotient of sums, 1e-6 relative
            bound[t] += weights[t, j] * (a @ dh + (I / 4 + 32) * u * (a @ np.abs(h)) + 1e-6 * np.abs(y))
    return Y, ids, weights, bound
