"""Plain 64-bit statements of the 4-bit cache's operators and of norm_rotate, and seeded caches, for their tests.

Tolerances follow from the arithmetic. Records and rows read back are compared exactly. Attention
is compared as the 8-bit cache's (see cache8_helpers): queries and weights enter as 22 bits, values exactly;
with 16-bit queries chunks of many rows round the weights to fp16 once, 2^-11. The weights' fp16 pairs have the
largest at 2^14 (prefill: 2^8 at least) and end in steps of 2^-24: 2^-39 (2^-33) of the largest weight
whatever a weight's size.
norm_rotate, with u = 2^-24: a sum of D squares by eights and shuffles 12 u, halved by the root, its root 4 u, three
products 3 u: 13 u of a normed element; an angle's rounding and its sine 2^-25 + 2^-23, the sum 2 u: with all of it
below 2^-19 (|a| + |b|). The transform adds u per stage of sum |y| / sqrt(D), and its scale 4 u. Then half a step
of the output's type.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

from kv_cache_quantization_token_gb300 import kvarn
from tests.cache8_helpers import DEV, HALF_STEP, T, attend, check, rows  # noqa: F401

MAX4 = 14336.0
INV_2PI = Fraction(15915494309189533576888376337251436203445964574045644874766734405889679763422653509011380276,
                   10 ** 92)  # 1 / (2 pi) to 92 digits


def quantise(x):
    """Rows [..., D] fp32 -> codes [..., D], scales [..., D/32]. The scale by search over candidates around the
    quotient in 64 bits (7 s is exact there), the code by comparing exact products."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(y).max(-1)
    with np.errstate(divide="ignore"):
        e = np.where(amax > 0, np.floor(np.log2(np.maximum(amax, 1e-300) / 7)), -200)
    step = 2.0 ** np.maximum(e - 7, -24)
    s = (np.floor(amax / 7 / step) - 2) * step
    for _ in range(6):  # up to the first that reaches it
        s = np.where(7 * s < amax, s + step, s)
    s = np.maximum(s, 2.0 ** -24)
    n = np.floor(np.abs(y) / s[..., None])
    n = np.where((n + 1) * s[..., None] <= np.abs(y), n + 1, n)
    n = np.where(n * s[..., None] > np.abs(y), n - 1, n)
    rest, half = np.abs(y) - n * s[..., None], s[..., None] / 2
    n = n + ((rest > half) | ((rest == half) & (n % 2 == 1)))
    return (np.sign(y) * n).reshape(x.shape), s


def poisoned(k, v):
    """Which rows [...] of k, v [..., D] are poison."""
    with np.errstate(invalid="ignore"):
        return ~((np.abs(k) <= MAX4).all(-1) & (np.abs(v) <= MAX4).all(-1))


def put_token(rec, D, t, kc, ks, vc, vs):
    """Token t of one record (uint8 [144 D]): codes [D] and fp16 scales [D/32] of K and of V."""
    run = rec[36 * D * (t // 32):36 * D * (t // 32 + 1)]
    words, halves, r, W = run.view(np.uint16), run.view(np.float16), t % 32, min(D, 128)
    for codes, k in ((kc, True), (vc, False)):
        u = (np.asarray(codes) + 8).astype(np.int64)
        for c in range(0, D, 4):
            a, b, d, e = u[c:c + 4]
            unit = a << 6 | b << 10 | d << 2 | (e & 3) << 14 | e >> 2
            if k:
                words[(c // W) * 32 * (W // 4) + r * (W // 4) + c % W // 4] = unit
            else:
                words[8 * D + (c // 32) * 256 + r * 8 + c % 32 // 4] = unit
    for i in range(D // 32):
        halves[16 * D + r * (D // 32) + i] = ks[i]
        halves[17 * D + i * 32 + 8 * (r % 8 // 2) + 2 * (r // 8) + r % 2] = vs[i]


class Cache4:
    """A batch of 4-bit caches built here, byte by byte, in a shuffled pool whose unwritten bytes are `fill`; k[b], v[b]
    are the values, [Hkv][tokens][D] in 64 bits (NaN for poison). Its table has `beyond` columns behind the tiles, each
    an offset that must not be followed."""

    beyond = 0

    def __init__(self, seed, lens, Hkv, D, max_tiles=None, fill=0xFF, change=None, spare=0):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.D, self.lens_of = len(lens), Hkv, D, list(lens)
        self.lay = kvarn.layout4(D)
        self.rb = rb = self.lay.record_bytes
        n_of = [-(-n // T) for n in lens]
        self.max_tiles = max(max(n_of), 1) if max_tiles is None else max_tiles
        units = Hkv * self.B * self.max_tiles
        place = rng.permutation(units + spare)[:units]
        pool = np.full((units + spare, rb), fill, np.uint8)
        table = (place * rb).reshape(self.B, Hkv, self.max_tiles).astype(np.int64)
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            kb, vb = np.zeros((Hkv, n, D)), np.zeros((Hkv, n, D))
            for h in range(Hkv):
                if not n:
                    continue
                k, v = rows(rng, n, D)
                if change:
                    change(b, h, k, v)
                bad = poisoned(k, v)
                k[bad] = v[bad] = 0
                (kc, ks), (vc, vs) = quantise(k), quantise(v)
                kb[h], vb[h] = kc * ks.repeat(32, -1), vc * vs.repeat(32, -1)
                ks[bad], vs[bad], kb[h, bad], vb[h, bad] = np.nan, 0, np.nan, np.nan
                for t in range(n):
                    put_token(pool[place[(b * Hkv + h) * self.max_tiles + t // T]], D, t % T, kc[t],
                              ks[t].astype(np.float16), vc[t], vs[t].astype(np.float16))
            self.k.append(kb)
            self.v.append(vb)
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
        self.pool = pool
        self.max_tiles += self.beyond
        table = np.concatenate([table, np.full((self.B, Hkv, self.beyond), -16)], 2)
        self.tiles, self.table = dev(pool.reshape(-1)), dev(table)
        self.lens = torch.tensor(list(lens), dtype=torch.int32, device=DEV)

    def decode(self, q, **kw):
        return kvarn.decode_attention4(q, self.tiles, self.table, self.lens, self.lay, **kw)

    def prefill(self, q, pos0, b=0, **kw):
        return kvarn.prefill_attention4(q, pos0, self.tiles, self.table[b], self.lay, **kw)


def turned(pos, freq):
    """cos and sin of pos * freq for integers pos [n] and a double freq: the turns taken off exactly."""
    out = []
    for p in pos:
        t = Fraction(float(freq)) * int(p) * INV_2PI
        t -= t.numerator // t.denominator
        out.append(2 * np.pi * float(t))
    return np.cos(out), np.sin(out)


def norm_rotate(x, weight, eps, pos, inv_freq, axis, adjacent, hadamard):
    """x [T, H, D] -> the result and the bound on its error before the output's rounding, in 64 bits; pos
    [axes][T] integers or None."""
    y = np.asarray(x, np.float64)
    D = y.shape[-1]
    if eps is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (1 if weight is None else np.asarray(weight, np.float64))
    bound = 13 * 2.0 ** -24 * np.abs(y)
    if pos is not None:
        n = len(inv_freq)
        y, bound, src = y.copy(), bound.copy(), y
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
            c, s = (z[:, None] for z in turned(pos[axis[i]], inv_freq[i]))
            y[..., a], y[..., b] = src[..., a] * c - src[..., b] * s, src[..., a] * s + src[..., b] * c
            bound[..., a] = bound[..., b] = 2.0 ** -19 * (np.abs(src[..., a]) + np.abs(src[..., b]))
    if hadamard:
        h = np.ones((1, 1))
        while h.shape[0] < D:
            h = np.block([[h, h], [h, -h]])
        size = np.abs(y).sum(-1, keepdims=True) / np.sqrt(D)
        y = y @ h / np.sqrt(D)
        bound = bound.sum(-1, keepdims=True) / np.sqrt(D) + (np.log2(D) + 4) * 2.0 ** -24 * size + 0 * y
    return y, bound
