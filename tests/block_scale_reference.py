"""64-bit definitions of the norm + rotation, the block-scaled 8-bit scatter and
the attention over it, in numpy, with the error bounds the GPU tests use.

Bounds count: half a step of the output type for its one rounding
(finfo(t).eps / 2 of the value), the fp32 arithmetic before it, and for
attention the fp16 rounding of a weight (2^-11).
"""

import math

import numpy as np

EPS = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}          # half a step, relative
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}       # half the smallest step
CODE_MAX = 448.0
MIN_EXP = -64


def code_values() -> np.ndarray:
    """float64 value of every E4M3 code."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


CODES = code_values()


def decode(codes: np.ndarray) -> np.ndarray:
    return CODES[codes]


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even fraction, saturating; NaN to a NaN code of its sign."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), CODE_MAX)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    n = np.rint(np.where(np.isnan(a), 0.0, a) / 2.0 ** (e - 3))  # fraction steps of binade e
    carry = n == 16
    e, n = np.where(carry, e + 1, e), np.where(carry, 8, n)
    bits = np.where(n < 8, n, ((e + 7) * 8 + n - 8)).astype(np.int64)
    bits = np.where(np.isnan(x), 0x7F, bits)
    return (bits | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def needed_exp(amax: float) -> int:
    """Smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    e = MIN_EXP
    if amax > 0:
        e = max(e, math.frexp(amax)[1] - 11)
        while amax > CODE_MAX * 2.0 ** e:
            e += 1
    return e


def block_scatter(rows, cache, scales, tables, lens, starts, bs):
    """One cache (K or V): rows float64 [T, Hkv, D], cache uint8 and scales float64 updated in place."""
    hkv = rows.shape[1]
    for b in range(len(lens)):
        t0, t1, L = int(starts[b]), int(starts[b + 1]), int(lens[b])
        ctx = L - (t1 - t0)
        if t1 == t0:
            continue
        for page in range(ctx // bs, (L - 1) // bs + 1):
            lo, hi = max(ctx, page * bs), min(L, (page + 1) * bs)
            phys, r0 = int(tables[b, page]), lo - page * bs
            x = rows[t0 + lo - ctx:t0 + hi - ctx]
            for h in range(hkv):
                fin = x[:, h][np.isfinite(x[:, h])]
                need = 2.0 ** needed_exp(float(np.abs(fin).max()) if fin.size else 0.0)
                old = float(scales[phys, h]) if r0 > 0 else 0.0
                if not (np.isfinite(old) and old > 0):
                    old = 0.0
                new = max(old, need)
                if r0 > 0 and new != old:
                    cache[phys, :r0, h] = encode(decode(cache[phys, :r0, h]) * (old / new))
                cache[phys, r0:r0 + hi - lo, h] = encode(x[:, h] / new)
                scales[phys, h] = new


def attention(q, kc, vc, ks, vs, tables, lens, starts, bs, scale):
    """Outputs and their bound, float64 [T, H, D]; q float64, caches uint8, scales [NB, Hkv]."""
    T, H, D = q.shape
    hkv = kc.shape[2]
    G = H // hkv
    out, bound = np.zeros((T, H, D)), np.zeros((T, H, D))
    for b in range(len(lens)):
        t0, t1, L = int(starts[b]), int(starts[b + 1]), int(lens[b])
        if t1 == t0:
            continue
        pages = tables[b, :(L + bs - 1) // bs].astype(np.int64)
        for h in range(hkv):
            k = (decode(kc[pages, :, h]) * ks[pages, h][:, None, None]).reshape(-1, D)[:L]
            v = (decode(vc[pages, :, h]) * vs[pages, h][:, None, None]).reshape(-1, D)[:L]
            vs_key = np.repeat(vs[pages, h], bs)[:L]
            qq = q[t0:t1, h * G:(h + 1) * G]                     # [n, G, D]
            s = np.einsum("ngd,kd->ngk", qq, k) * scale
            mag = np.einsum("ngd,kd->ngk", np.abs(qq), np.abs(k)) * abs(scale)
            seen = np.arange(L)[None, :] <= (L - (t1 - t0) + np.arange(t1 - t0))[:, None]
            s = np.where(seen[:, None, :], s, -np.inf)
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            p /= p.sum(-1, keepdims=True)
            o = np.einsum("ngk,kd->ngd", p, v)
            a = np.einsum("ngk,kd->ngd", p, np.abs(v))
            # a score: D products and sums in fp32 (relative to the sum of
            # magnitudes), the exponent's rounding (relative to the largest
            # exponent, log2 of the V scale included) and 2^x itself
            big = np.where(seen[:, None, :], mag, 0).max(-1, keepdims=True)
            lv = np.abs(np.log2(vs_key)).max()
            delta = D * 2.0 ** -24 * big + (1.5 * big + lv + 4) * 2.0 ** -22 + 2.0 ** -21
            # weights: fp16 half step, or half of fp16's smallest step against the largest weight times V scale
            floor = 2.0 ** -25 * CODE_MAX * L * (p * vs_key).max(-1, keepdims=True)
            out[t0:t1, h * G:(h + 1) * G] = o
            bound[t0:t1, h * G:(h + 1) * G] = (2.0 ** -11 + 2 * delta) * a + floor
    return out, bound


def norm_rope(x, w, eps, positions, table, rot, neox):
    """Rows float64 [T, heads, D]; returns (rotated rows, magnitude that an fp32 error is relative to)."""
    x = np.asarray(x, dtype=np.float64)
    y = x
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    out, mag = y.copy(), np.abs(y)
    row = table[positions].astype(np.float64)[:, None, :]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    i1 = np.arange(rot // 2) if neox else np.arange(0, rot, 2)
    i2 = i1 + rot // 2 if neox else i1 + 1
    y1, y2 = y[..., i1], y[..., i2]
    out[..., i1], out[..., i2] = y1 * c - y2 * s, y2 * c + y1 * s
    mag[..., i1] = mag[..., i2] = np.abs(y1) + np.abs(y2)
    return out, mag


def norm_rope_bound(ref, mag, dtype):
    """One rounding of the type, and fp32 before it: a sum of D squares in chains of 16 and a tree (half of
    whose relative error, at most 24 steps of 2^-24, reaches the norm), the reciprocal root, two products and
    the rotation's two roundings: at most 20 steps of 2^-24 of the magnitude."""
    return EPS[dtype] * np.abs(ref) * (1 + 2.0 ** -7) + 20 * 2.0 ** -24 * mag + TINY[dtype]
