"""fp64 reference of the rotary rows and of the 8-bit key/value cache.

TEST INFRASTRUCTURE ONLY. Plain numpy in float64, one (row, block, head) rule at a time:

* rope_rows -- every row turned by rope_rotate to the (t, x, y) position of its token;
* e4m3 (4 exponent bits with bias 7, 3 mantissa bits, largest 448, codes 0x7F / 0xFF NaN,
  no infinities): decode from the bits, round to nearest with ties to even;
* kv_sync_q8 -- the block-scaled cache update;
* attn_bound -- what the arithmetic of an f16-probability, fp32-sum attention over such a
  cache may be off by.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from .tps_oracle import f64, rope_rotate

__all__ = ["rope_rows", "e4m3_decode", "e4m3_round", "q8_scale", "q8_values", "kv_sync_q8", "q8_attn_bound"]

BLOCK = 128


def rope_rows(x, idx, dims, grid, origin=(0, 0, 0), base: float = 10000.0, inverse: bool = False) -> np.ndarray:
    """x [A, H, d]; row j turned to token idx[j] = (f*Hs + y)*Ws + x on the grid (F, Hs, Ws), or back."""
    F, Hs, Ws = grid
    out = f64(x).copy()
    sign = -1 if inverse else 1
    for j, n in enumerate(np.asarray(idx, np.int64)):
        pos = (n // (Hs * Ws) + origin[0], n % Ws + origin[1], (n // Ws) % Hs + origin[2])
        out[j] = rope_rotate(out[j], dims, [sign * int(p) for p in pos], base)
    return out


def e4m3_decode(codes) -> np.ndarray:
    """uint8 codes -> float64 values, from the bit fields."""
    c = np.asarray(codes, np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def e4m3_round(x) -> np.ndarray:
    """float64 -> the nearest e4m3 value (ties to even), saturated at 448; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0) - 3.0)
    return np.copysign(np.round(a / step) * step, x)        # numpy rounds halves to even


def q8_scale(amax: float) -> float:
    """The smallest 2^e, -100 <= e <= 100, with amax <= 448 * 2^e; 0 for 0."""
    if amax == 0:
        return 0.0
    e = -100
    while e < 100 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def q8_values(codes, scale) -> np.ndarray:
    """codes uint8 [N, H, d], scale [nb, H] -> float64 values [N, H, d]."""
    v = e4m3_decode(codes)
    return v * np.repeat(f64(scale), BLOCK, axis=0)[: v.shape[0], :, None]


def kv_sync_q8(values, scale, fresh, idx):
    """One tensor of the cache: values float64 [N, H, d] (unscaled e4m3 values), scale [nb, H]; fresh float64
    [A, H, d] (keys already turned), idx ascending. Returns (values, scale) after the update."""
    values, scale = values.copy(), f64(scale).copy()
    N, H, _ = values.shape
    idx = np.asarray(idx, np.int64)
    for b in np.unique(idx // BLOCK):
        lo, hi = b * BLOCK, min(N, (b + 1) * BLOCK)
        rows = np.flatnonzero((idx >= lo) & (idx < hi))
        stale = np.setdiff1d(np.arange(lo, hi), idx[rows])
        for h in range(H):
            x = fresh[rows, h]
            fin = np.abs(x[np.isfinite(x)])
            need = q8_scale(float(fin.max()) if fin.size else 0.0)
            old = scale[b, h] if scale[b, h] > 0 else 0.0
            new = need if len(stale) == 0 else max(old, need)
            if len(stale) and new != scale[b, h]:
                values[stale, h] = e4m3_round(values[stale, h] * (old / new if new else 0.0))
            values[idx[rows], h] = e4m3_round(x / (new if new else 1.0))
            scale[b, h] = new
    return values, scale


def q8_attn_bound(q, k, v, vs, idx, scale: float, blockmask=None, floor=None):
    """(tolerance of o [A, H, d], tolerance of lse [A, H]) for float64 k, v [N, H, d] and V's scales vs [nb, H].

    With E the mean over the softmax weights p, and e the relative error of an unrounded probability:
      e    <= scale * (2^-17 max|q| sum|k| + 2 d 2^-23 sum|q||k|)   (q's two 8-bit parts: at most 2^-17 of the
              row's largest where they are not exact; products summed in fp32, 2 d terms, truncated sums)
              + 2^-22 (|x| + 4)                                       (the fp32 exponent, exp2, reciprocals),
      o:   (2^-11 + 2 e) E|v| + N 2^-25 448 max vs + 2^-8 |o|         (f16 probabilities, normal and below
              2^-14 of the reference; bf16 output),
      lse: e + 2^-22 (|lse| + 1).
    floor: a tighter second term, for scales far apart and for long caches. What f16 cannot hold is below `floor` of
    the row's largest p vs, so the term is N floor 448 max_n(p_n vs_n)."""
    A, H, d = q.shape
    N = k.shape[0]
    o_tol, l_tol = np.zeros((A, H, d)), np.zeros((A, H))
    kb = np.arange(N) // BLOCK
    for h in range(H):
        Q, K, V = f64(q[:, h]), f64(k[:, h]), f64(v[:, h])
        x = Q @ K.T * scale
        ab = np.abs(Q) @ np.abs(K).T
        if blockmask is not None:
            keep = (np.asarray(blockmask) != 0)[np.asarray(idx, np.int64) // BLOCK][:, kb]
            x, ab = np.where(keep, x, -np.inf), np.where(keep, ab, 0.0)
        top = x.max(1, keepdims=True)
        live = np.isfinite(top)
        p = np.exp(x - np.where(live, top, 0.0))
        l = p.sum(1, keepdims=True)
        p = np.where(live, p / np.where(l > 0, l, 1.0), 0.0)
        big = np.where(np.isfinite(x), np.abs(x), 0.0).max(1) * math.log2(math.e)
        e = scale * (2.0 ** -17 * np.abs(Q).max(1) * np.abs(K).sum(1).max() + 2 * d * 2.0 ** -23 * ab.max(1))
        e = e + 2.0 ** -22 * (big + 4)
        o = p @ V
        if floor is None:
            lost = N * 2.0 ** -25 * 448 * f64(vs)[:, h].max()
        else:
            lost = (N * floor * 448 * (p * f64(vs)[kb, h]).max(1))[:, None]
        o_tol[:, h] = (2.0 ** -11 + 2 * e)[:, None] * (p @ np.abs(V)) + lost + 2.0 ** -8 * np.abs(o)
        lse = np.where(live[:, 0], np.where(live, top, 0.0)[:, 0] + np.log(np.where(l > 0, l, 1.0))[:, 0], 0.0)
        l_tol[:, h] = e + 2.0 ** -22 * (np.abs(lse) + 1)
    return o_tol, l_tol


def codes_of(values: np.ndarray) -> torch.Tensor:
    """float64 e4m3 values -> uint8 codes (the exact cast of torch)."""
    return torch.from_numpy(np.ascontiguousarray(values)).float().to(torch.float8_e4m3fn).view(torch.uint8)
