"""MXFP4: quantization, dequantization, the grouped product, the backward's
re-quantization to MXFP8, and the expert layer for a few tokens on 4-bit
weights.

TEST INFRASTRUCTURE ONLY (see the package docstring).

MXFP4 (OCP Microscaling) is E2M1 elements in NVFP4's nibble order with one E8M0
scale per 32 consecutive elements of a row. The pages do not use it; readings:
* block exponent: the smallest e with max|x_block| <= 6 * 2^e, clamped to
  [-127, 127] (0 gives -127): the MXFP8 rule with E2M1's largest value;
* codes E2M1_RNE(x * 2^-e), sign kept;
* the backward of a saved MXFP4 tensor is mxfp8.requant_sr's on its values.
The few-token layer is route.py's selection and gates and, in float64, the
projections of the dequantized weights; its activations are not quantized.
"""

import numpy as np

from . import formats as F
from . import mxfp8 as MX
from . import nvfp4 as Q
from . import route as R

BLOCK = 32


def block_exponents(x):
    """Smallest e with amax <= 6 * 2^e for each block of 32 of float32 x, by trial."""
    a = np.abs(np.asarray(x, np.float64)).reshape(x.shape[0], -1, BLOCK).max(axis=2)
    with np.errstate(divide="ignore"):
        e = np.where(a > 0, np.floor(np.log2(np.where(a > 0, a, 1.0))) - 4, -127).astype(np.int64)
    for _ in range(4):                                   # the guess is at most three below
        e = np.where(a > 6.0 * np.exp2(e.astype(np.float64)), e + 1, e)
    return np.clip(e, -127, 127)


def quantize(x):
    """x [rows, cols] (float32 or bfloat16 bits) -> (codes [rows, cols/2], scales [rows, cols/32])."""
    x = Q._as_f32(x)
    e = block_exponents(x)
    y = x.astype(np.float64).reshape(x.shape[0], -1, BLOCK) * np.exp2(-e.astype(np.float64))[:, :, None]
    return Q.pack_codes(F.e2m1_rne(y.reshape(x.shape))), (e + 127).astype(np.uint8)


def dequantize(codes, scales):
    """float64 values [rows, cols] (exact)."""
    codes = np.asarray(codes)
    v = F.e2m1_decode(Q.unpack_codes(codes)).astype(np.float64)
    s = np.exp2(np.asarray(scales).astype(np.float64) - 127)
    return (v.reshape(codes.shape[0], -1, BLOCK) * s[:, :, None]).reshape(v.shape)


def weight(w):
    """float64 values of a weight in MXFP4 (codes, scales) or NVFP4 (codes, scales, outer of each expert)."""
    if len(w) == 2:
        return dequantize(*w)
    v = F.e2m1_decode(Q.unpack_codes(w[0])).astype(np.float64)
    v = v.reshape(v.shape[0], -1, 16) * F.e4m3_decode(np.asarray(w[1])).astype(np.float64)[:, :, None]
    return v.reshape(v.shape[0], -1) * np.repeat(np.asarray(w[2], np.float64), v.shape[0] // len(w[2]))[:, None]


def fwd_grouped(a, b, offsets, N, row_token=None):
    """(y, magnitude) float64 [M, N]: the product, and the same sum over
    magnitudes (what a rounding error bound scales with)."""
    A, B = dequantize(*a), dequantize(*b)
    off = np.asarray(offsets, np.int64)
    M = int(off[-1])
    rows = np.arange(M) if row_token is None else np.asarray(row_token, np.int64)[:M]
    y, mag = np.zeros((M, N)), np.zeros((M, N))
    for g in range(off.shape[0] - 1):
        s = slice(int(off[g]), int(off[g + 1]))
        w = B[g * N:(g + 1) * N]
        y[s] = A[rows[s]] @ w.T
        mag[s] = np.abs(A[rows[s]]) @ np.abs(w).T
    return y, mag


def requant_sr(codes, scales, offsets, padded_offsets, P, seed, tag, row_token=None):
    """(E4M3 [cols, P], E8M0 [cols, P/32]) of saved MXFP4 rows (through row_token)."""
    v = dequantize(codes, scales).astype(np.float32)
    if row_token is not None:
        M = int(np.asarray(offsets)[-1])
        v = v[np.asarray(row_token, np.int64)[:M]]
    return MX.quantize_sr(MX.transpose_grouped(v, offsets, padded_offsets, P), seed, tag)


def activate(v, act):
    if act == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    return np.maximum(v, 0.0) ** 2 if act == "relu2" else v


def _slope(v, act):
    """A bound of the activation's slope near v."""
    return {"silu": 1.1, "relu2": 2.0 * np.abs(v), "none": 1.0}[act] + 0.0 * v


def ffn_tokens(x, logits, k, w1, w2, act="silu", gated=False, score="softmax", renorm=True,
               scale=1.0, bias=None, token_mask=None, e0=0, n_local=1, u=2.0 ** -23, gate_rel=0.0):
    """dict(out, topk_ids, gate, bound): float64 results, and how far out may be
    when sums of n terms lose n u of their magnitude, h is a float32 and gates are
    right to a relative gate_rel."""
    r = R.route(logits, k, score, renorm, scale, bias, token_mask)
    xv = Q._as_f32(x).astype(np.float64)
    W1, W2 = weight(w1), weight(w2)
    T, K = xv.shape
    Fw = W2.shape[1]
    rows = W1.shape[0] // n_local
    out, bound = np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for j in range(k):
            e = int(r["topk_ids"][t, j]) - e0
            if r["topk_ids"][t, j] < 0 or not 0 <= e < n_local:
                continue
            a1, a2 = W1[e * rows:(e + 1) * rows], W2[e * K:(e + 1) * K]
            v, dv = a1 @ xv[t], (K + 4) * u * (np.abs(a1) @ np.abs(xv[t]))
            h = activate(v[:Fw], act)
            # the activation's own arithmetic: exp of |v| loses |v| u, quotient and products a few more
            dh = _slope(v[:Fw], act) * dv[:Fw] + dv[:Fw] ** 2 + np.abs(h) * (np.abs(v[:Fw]) + 16) * u
            if gated:
                dh = dh * np.abs(v[Fw:]) + np.abs(h) * dv[Fw:] + dh * dv[Fw:]
                h = h * v[Fw:]
            g = r["gate"][t, j]
            dh = dh + np.abs(h) * (gate_rel + 4 * u)
            out[t] += g * (a2 @ h)
            bound[t] += g * (np.abs(a2) @ (dh + (Fw * k + 4) * u * np.abs(h)))
    return dict(out=out, topk_ids=r["topk_ids"], gate=r["gate"], bound=bound)
