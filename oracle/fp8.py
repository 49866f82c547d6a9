"""FP8 block format, its product, the block norm and the experts' layer, in FP64.

TEST INFRASTRUCTURE ONLY: a plain restatement used to check the GPU library.  The steps
that decide a code (the scale, its reciprocal, the product with it) are FP32, as the
format defines them; everything else is FP64.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128
TINY = np.float32(2.0 ** -100)


def _decode_table() -> np.ndarray:
    """Values of the 256 E4M3 codes from their fields (bias 7, no infinity)."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (c & 0x7F) == 0x7F else (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 0x80 else v
    return out


E4M3 = _decode_table()


def decode(codes: np.ndarray) -> np.ndarray:
    return E4M3[codes]


def encode(v: np.ndarray) -> np.ndarray:
    """To the nearest code, ties to the even one, saturating at 448; NaN to 0x7F."""
    v = np.asarray(v, dtype=np.float64)
    mags = E4M3[:127]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    c = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    c = np.where(a >= 448, 126, c) | (np.signbit(v) * 128)
    return np.where(np.isnan(v), 0x7F, c).astype(np.uint8)


def block_scale(amax: np.ndarray):
    """FP32 block maxima -> (scale, reciprocal) as FP32."""
    a = np.where(amax < TINY, TINY, amax).astype(np.float32)
    with np.errstate(invalid="ignore"):
        return a / np.float32(448), np.float32(448) / a


def quant_rows(x: np.ndarray):
    """float32 [M, K] -> (codes uint8 [M, K], scales float32 [ceil(K/128), M])."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    codes = np.zeros((M, K), np.uint8)
    scales = np.zeros((kb, M), np.float32)
    for b in range(kb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float32)
        s, inv = block_scale(np.abs(v).max(axis=1))
        with np.errstate(invalid="ignore"):
            codes[:, b * BLOCK:(b + 1) * BLOCK] = encode(v * inv[:, None])
        scales[b] = s
    return codes, scales


def quant_tiles(w: np.ndarray):
    """float32 [N, K] -> (codes uint8 [N, K], scales float32 [ceil(N/128), ceil(K/128)])."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((nb, kb), np.float32)
    for i in range(nb):
        for b in range(kb):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            v = w[at].astype(np.float32)
            s, inv = block_scale(np.abs(v).max())
            with np.errstate(invalid="ignore"):
                codes[at] = encode(v * inv)
            scales[i, b] = s
    return codes, scales


def dequant_rows(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    K = codes.shape[1]
    return decode(codes) * np.repeat(scales.T.astype(np.float64), BLOCK, axis=1)[:, :K]


def dequant_tiles(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, axis=0)[:N], BLOCK, axis=1)[:, :K]
    return decode(codes) * s


def gemm(xc, xs, wc, ws):
    """(y, sum of the products' magnitudes) of the block-scaled product."""
    x, w = dequant_rows(xc, xs), dequant_tiles(wc, ws)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def rms(v, w, offset, eps):
    return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps) * (w + offset)


def block_norm(y, h, post_weight=None, gate=None, res_scale=1.0, pre_weight=None, offset=0.0, eps=1e-6):
    """(h', x or None); gate is [G, D]."""
    M, D = (h if y is None else y).shape
    u = np.zeros((M, D)) if y is None else y.astype(np.float64)
    if post_weight is not None:
        u = rms(u, post_weight, offset, eps)
    if gate is not None:
        u = u * np.repeat(gate, M // gate.shape[0], axis=0)
    h2 = u if h is None else res_scale * h + u
    return h2, None if pre_weight is None else rms(h2, pre_weight, offset, eps)


def route(x, router, k, score="softmax", bias=None, renorm=True, route_scale=1.0):
    """(ids [T, k], weights [T, k]) of the router, ties to the lowest index."""
    logits = x @ router.T
    if score == "softmax":
        p = np.exp(logits - logits.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
    else:
        p = 1 / (1 + np.exp(-logits))
    key = logits if bias is None else p + bias
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, axis=1)
    if renorm:
        w = w / w.sum(axis=1, keepdims=True)
    return ids, w * route_scale


def moe(x, ids, weights, w13, w2, shared=0):
    """sum of the picked experts' outputs for dequantised weights [n, 2F, D], [n, D, F]; the
    last `shared` experts serve every token with weight 1."""
    n, F = w13.shape[0], w13.shape[1] // 2
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        picks = list(zip(ids[t], weights[t])) + [(e, 1.0) for e in range(n - shared, n)]
        for e, w in picks:
            g, u = w13[e, :F] @ x[t], w13[e, F:] @ x[t]
            y[t] += w * (w2[e] @ (g / (1 + np.exp(-g)) * u))
    return y
