"""Plain, slow CPU oracle for the MXFP4 path and the mixture-of-experts layer (NumPy).

TEST INFRASTRUCTURE ONLY: only ``tests/`` imports this module, and nothing here imports,
calls or links the product path.

* MXFP4 is the 4-bit member of the Open Compute Project's microscaling formats: E2M1
  elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), 32-element blocks along K that
  share an E8M0 scale byte (value 2^(byte - 127), 0xFF is NaN). Two elements per byte,
  element 2j in the low nibble.
* Shared exponent of a block: e = floor(log2(amax)) - 2 clamped to [-127, 127]; an all-zero
  block takes byte 0. A block with a NaN or an infinity takes byte 0xFF and codes 0.
* Elements: the E2M1 value nearest to x / 2^e, ties to the even code, saturating at 6, sign
  copied.

Parity unpinned (conventions with no external reference): the nibble order, the scale byte
of an all-zero block and the codes of a NaN block.
"""
from __future__ import annotations

import numpy as np

from .mxfp8_oracle import e8m0_decode, floor_log2
from .nvfp4_oracle import _nearest_code_ties_even, bf16_bits_to_f32

BLOCK = 32
EMAX = 2  # exponent of the largest E2M1 value, 6 = 1.5 * 2^2
E2M1_POS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x_bits: np.ndarray):
    """(packed uint8 [rows, K/2], scales uint8 [rows, K/32]) of a bf16 tensor [rows, K]."""
    x_bits = np.asarray(x_bits, dtype=np.uint16)
    R, K = x_bits.shape
    if K % BLOCK:
        raise ValueError("K must be a multiple of 32")
    x = bf16_bits_to_f32(x_bits).astype(np.float64).reshape(R, K // BLOCK, BLOCK)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(axis=-1)
    e = np.clip(floor_log2(np.where(amax > 0, amax, 1.0)) - EMAX, -127, 127)
    e = np.where(amax > 0, e, -127)
    y = np.ldexp(x, -e[..., None])
    code = _nearest_code_ties_even(np.abs(y), E2M1_POS).astype(np.uint8)
    code = np.where(np.signbit(y), code | np.uint8(8), code).astype(np.uint8).reshape(R, K)
    scales = np.where(bad, 0xFF, e + 127).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scales


def dequantize(packed: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of packed [..., K/2] and scales [..., K/32]."""
    code = np.stack((packed & 15, packed >> 4), axis=-1).reshape(*packed.shape[:-1], -1)
    v = E2M1_POS[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.repeat(e8m0_decode(scales), BLOCK, axis=-1)
    return v * s


def gemm_ref(a_packed, a_scales, w_packed, w_scales):
    """(out, sum of magnitudes) of A_hat @ W_hat^T in float64."""
    A, W = dequantize(a_packed, a_scales), dequantize(w_packed, w_scales)
    return A @ W.T, np.abs(A) @ np.abs(W).T


def route(logits: np.ndarray, top_k: int, renormalize: bool):
    """(ids int32, weights float64) [T, top_k] of float32 logits [T, E]: the largest first,
    ties to the lowest index, NaN above +inf, -inf never chosen (id -1, weight 0)."""
    T, E = logits.shape
    ids = np.full((T, top_k), -1, dtype=np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        row = logits[t].astype(np.float64)
        able = [i for i in range(E) if not np.isneginf(row[i])]
        able.sort(key=lambda i: (0, 0.0, i) if np.isnan(row[i]) else (1, -row[i], i))
        pick = able[:top_k]
        if not pick:
            continue
        with np.errstate(invalid="ignore"):
            p = np.exp(row - (np.nan if np.isnan(row).any() else row.max()))
        total = p[pick].sum() if renormalize else p[able].sum()
        ids[t, : len(pick)] = pick
        weights[t, : len(pick)] = p[pick] / total
    return ids, weights


def moe_ref(x, ids, weights, w13, w2, h_error=2.0**-8):
    """(out, tol) [T, H] of activations x [T, H] under a routing, with decoded weights w13
    [E, 2I, H] and w2 [E, H, I], all float64.

    ``tol`` bounds a correct result's error, to first order: a sum of n products in fp32 is
    off by at most n 2^-24 of its terms' magnitudes (any order), |silu'| <= 1.1 and
    |silu(g)| <= |g|; h is held to ``h_error`` of its value (2^-8: rounded to bf16 once) after an
    exponential and a division good to 2^-20; routing weights are good to 2^-20; out is rounded
    to bf16."""
    T, H = x.shape
    I = w2.shape[2]
    out, tol = np.zeros((T, H)), np.zeros((T, H))
    eh, ei = (H + 8) * 2.0**-24, (I + 64) * 2.0**-24
    for t in range(T):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if e < 0:
                continue
            g, u = w13[e, :I] @ x[t], w13[e, I:] @ x[t]
            with np.errstate(over="ignore"):
                h = g / (1.0 + np.exp(-g)) * u
            out[t] += weights[t, j] * (w2[e] @ h)
            sg, su = np.abs(w13[e, :I]) @ np.abs(x[t]), np.abs(w13[e, I:]) @ np.abs(x[t])
            dh = 1.1 * eh * sg * np.abs(u) + eh * np.abs(g) * su + (h_error + 2.0**-19) * np.abs(h)
            tol[t] += np.abs(weights[t, j]) * (np.abs(w2[e]) @ (dh + (ei + 2.0**-19) * np.abs(h)))
    return out, tol + 2.0**-8 * (np.abs(out) + tol)
