"""CPU oracle for the operators whose rows have weights of their own.

TEST INFRASTRUCTURE, with the same standing as ``int8mm_oracle``: plain numpy in float64,
sharing no code with the HIP library or its binding. Values are passed as float64 arrays that
hold exact fp16 / bf16 / fp32 numbers. Functions that return a bound give what rounding in fp32
(and the documented fewer bits) can move the result by, before the output's own rounding.
"""

from __future__ import annotations

import numpy as np

from . import int8mm_oracle as int8
from . import mx4_oracle as mx4

U = 2.0 ** -24


def group_order(ids: np.ndarray, groups: int):
    """ids [T, k] (-1: none) -> offsets [groups + 1], rows [T k], slots [T, k]."""
    T, k = ids.shape
    offsets = np.zeros(groups + 1, np.int64)
    rows, slots = np.full(T * k, -1, np.int64), np.full((T, k), -1, np.int64)
    at = 0
    for e in range(groups):
        for t, j in zip(*np.nonzero(ids == e)):
            rows[at], slots[t, j] = t, at
            at += 1
        offsets[e + 1] = at
    return offsets, rows, slots


def _gate(v, dv):
    """silu(gate) * up of halves of v, and what errors dv of v move it by."""
    (g, u), (dg, du) = np.split(v, 2, 1), np.split(dv, 2, 1)
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    # |silu'| <= 1.1; a few units of fp32 for exp, the quotient and the product
    return silu * u, 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + np.abs(silu * u) * 8 * U


def _grouped(x_rows, offsets, rows, P, N, gated, product):
    Y, bound = np.zeros((P, N // 2 if gated else N)), np.zeros((P, N // 2 if gated else N))
    for e in range(len(offsets) - 1):
        p = np.arange(offsets[e], offsets[e + 1])
        src = p if rows is None else rows[p]
        p, src = p[(src >= 0) & (src < x_rows)], src[(src >= 0) & (src < x_rows)]
        if len(p) == 0:
            continue
        v, dv = product(e, src)
        Y[p], bound[p] = _gate(v, dv) if gated else (v, dv)
    return Y, bound


def grouped_mx4(X, W, offsets, rows, P, gated):
    """X [M, K] values, W [E, N, K] values as held -> (Y, bound)."""
    x, K = mx4.mx4_round(X), X.shape[1]

    def product(e, src):
        # a rounding per 128 elements of K, and as many again for sums inside the instruction
        return x[src] @ W[e].T, (np.abs(x[src]) @ np.abs(W[e]).T) * (-(-K // 128) + 32) * 2 * U
    return _grouped(len(X), offsets, rows, P, W.shape[1], gated, product)


def grouped_int8(X, Wq, a_w, threshold, offsets, rows, P, gated):
    """X [M, K] fp16, codes Wq [E, N, K], constants a_w [E, N] -> (Y, bound)."""
    q = int8.quant_rows(X, threshold)
    xo = X[:, q["idx"]].astype(np.float64)

    def product(e, src):
        acc = q["Xq"][src].astype(np.float64) @ Wq[e].astype(np.float64).T
        y8 = int8.dequant_outer(acc, q["a_x"][src], a_w[e])
        # the outlier columns' weights are fp16 values, by this expression in fp32
        held = (Wq[e][:, q["idx"]].astype(np.float32) * a_w[e][:, None].astype(np.float32) / np.float32(127))
        held = held.astype(np.float16).astype(np.float64)
        yo, so = xo[src] @ held.T, np.abs(xo[src]) @ np.abs(held).T
        # the int8 part: the sum, two constants' products, 1 / 127^2; then a rounding per term
        return y8 + yo, np.abs(y8) * 6 * U + (np.abs(y8) + so) * (len(q["idx"]) + 2) * U
    return _grouped(len(X), offsets, rows, P, Wq.shape[1], gated, product)


def combine(P, slots, weights):
    Y, bound = np.zeros((len(slots), P.shape[1])), np.zeros((len(slots), P.shape[1]))
    for j in range(slots.shape[1]):
        on = (slots[:, j] >= 0) & (slots[:, j] < len(P))
        term = weights[on, j:j + 1] * P[slots[on, j]]
        Y[on] += term
        bound[on] += np.abs(term) * (slots.shape[1] + 1) * U
    return Y, bound


def lora(Y, X, A, B, ids, scales, ranks, bf16):
    """out values and bound: V = A X in fp32, held in 16 (bf16) or 21 bits and more (fp16, under a
    row's own power of two), then B V and the sum with Y in fp32."""
    M, K = X.shape
    out, bound = Y.copy(), np.zeros_like(Y)
    for a in range(len(A)):
        m = np.nonzero(ids == a)[0]
        r = A.shape[1] if ranks is None else int(ranks[a])
        if len(m) == 0 or r == 0:
            continue
        s = 1.0 if scales is None else scales[a]
        Aa, Ba = A[a, :r], B[a, :, :r]
        V = X[m] @ Aa.T
        dV = (np.abs(X[m]) @ np.abs(Aa).T) * (K / 4 + 96) * U
        top = np.abs(V).max(1, keepdims=True)
        dV += np.abs(V) * 2.0 ** -16 if bf16 else np.abs(V) * 2.0 ** -21 + top * 2.0 ** -38
        L, S = V @ Ba.T, np.abs(V) @ np.abs(Ba).T
        out[m] += s * L
        bound[m] = np.abs(s) * (dV @ np.abs(Ba).T + S * (r / 2 + 8) * U) + (np.abs(s * L) + np.abs(out[m])) * 2 * U
    return out, bound
