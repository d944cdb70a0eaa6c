"""Plain 64-bit statements of the 8-bit cache's operators, and seeded caches, for its tests.

Tolerances follow from the arithmetic. A record's bytes are compared exactly (the
quotients are decided exactly on both sides). Attention is compared per element
against sum_t p_t |v_t|, the size of the terms of that output:
  scores   q enters as 22 bits or exactly, codes exactly, and each of the at most
           2 D / 16 + 2 accumulation steps loses up to 2^-23 of sum_c |q_c k_tc|, so a
           score is off by at most 2^-18 of that (times the softmax scale), and the
           ratio of two weights by twice that: 2^-17;
  weights  exponential and 22-bit split, 2^-20 together, then one 2^-23 per 16 tokens
           summed, and for 16-bit prefill one fp16 rounding, 2^-11;
  floor    the weighted probabilities w_t = p_t vscale_t are fp16 pairs with a common power
           of two that puts the largest at 2^14 (prefill: 2^8 at least), and fp16 ends in
           steps of 2^-24: each is off by up to 2^-25 in those units whatever its size,
           2^-39 (2^-33) of the largest. With a value row of zeros under the largest weight
           (a row far below its block's scale) nothing larger covers that.
  output   half a step of its type.
"""
from __future__ import annotations

import numpy as np
import torch

from kv_cache_quantization_token_gb300 import kvarn

DEV = "cuda:0"
T = 128
QMAX = {"i8": 127.0, "e4m3": 448.0}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def e4m3_values():
    """The 127 non-negative finite e4m3 values, by code."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def quantise(x, code, block):
    """x [128, D] fp32 -> stored bytes [128, D], values of the codes, scales [8]."""
    x = np.asarray(x, np.float32)
    D = x.shape[1]
    b = x.reshape(T // block, block, D)
    good = np.isfinite(b).all((1, 2))
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(b).max((1, 2))
        s = np.maximum(amax / np.float32(QMAX[code]), np.float32(2.0 ** -100)).astype(np.float32)
    s = np.where(good, s, np.float32(np.nan)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        y = np.where(good[:, None, None], b.astype(np.float64) / s.astype(np.float64)[:, None, None], 0.0)
    y = y.reshape(T, D)
    if code == "i8":
        v = np.rint(y)
        byte = (v + 128).astype(np.uint8)
    else:
        vals = e4m3_values()
        mid = (vals[1:] + vals[:-1]) / 2
        at = np.searchsorted(mid, np.abs(y), side="left")   # at a middle: the lower value
        tie = (at < 126) & (np.abs(y) == mid[np.minimum(at, 125)])
        at = at + (tie & (at % 2 == 1))
        neg = np.signbit(np.where(good.repeat(block)[:, None], x, 0))  # -0 and what rounds to it keep the sign
        v = np.where(neg, -vals[at], vals[at])
        byte = (at + 128 * neg).astype(np.uint8)
    return byte, v, s.repeat(block // 16)


def pack(kb, ks, vb, vs):
    """Stored bytes [128, D] and scales [8] of K and V -> one record."""
    D = kb.shape[1]
    rec = np.zeros(256 * D + 128, np.uint8)
    t, c = np.meshgrid(np.arange(T), np.arange(D), indexing="ij")
    rec[(t // 8) * 8 * D + (c // 64) * 512 + (t % 8) * 64 + c % 64] = kb
    rec[128 * D + (c // 8) * 1024 + (t // 64) * 512 + (c % 8) * 64 + t % 64] = vb
    rec[256 * D:256 * D + 32] = np.ascontiguousarray(ks, np.float32).view(np.uint8)
    rec[256 * D + 32:256 * D + 64] = np.ascontiguousarray(vs, np.float32).view(np.uint8)
    return rec


def rows(rng, n, D):
    """K with outlier channels, V with heavy-tailed token scales."""
    ch = np.exp(rng.standard_normal(D))
    ch[rng.choice(D, max(1, D // 50), replace=False)] *= 20
    k = (rng.standard_normal((n, D)) * ch).astype(np.float32)
    v = (rng.standard_normal((n, D)) * np.abs(rng.standard_t(4, (n, 1)))).astype(np.float32)
    return k, v


class Cache8:
    """A batch of caches: records written by kvarn.compress_tile8 into a shuffled pool, windows
    in rings; k[b], v[b] are what attention sees, [Hkv][tokens][D] in 64 bits."""

    def __init__(self, seed, tiles, windows, Hkv, D, code="i8", block=64, cap=None, starts=None,
                 max_tiles=None):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.D = len(tiles), Hkv, D
        self.tiles_of, self.windows = list(tiles), list(windows)
        self.lay = kvarn.layout8(D, code, block)
        rb = self.lay.record_bytes
        self.max_tiles = max(tiles) if max_tiles is None else max_tiles
        self.cap = cap if cap is not None else max(T, -(-max(windows) // T) * T)
        self.starts = starts if starts is not None else [int(rng.integers(0, self.cap)) for _ in tiles]
        n_units = Hkv * sum(tiles)
        place = rng.permutation(n_units)
        raw_k, raw_v = np.zeros((n_units * T, D), np.float32), np.zeros((n_units * T, D), np.float32)
        table = np.full((self.B, Hkv, self.max_tiles), -1, np.int64)
        wk = rng.standard_normal((self.B, Hkv, self.cap, D)).astype(np.float32) * 1e30  # unused slots: junk
        wv = wk.copy()
        self.k, self.v, self.vs, u = [], [], [], 0
        for b in range(self.B):
            n = T * tiles[b] + windows[b]
            kb, vb, sb = np.zeros((Hkv, n, D)), np.zeros((Hkv, n, D)), np.zeros((Hkv, n))
            for h in range(Hkv):
                k, v = rows(rng, n, D)
                for i in range(tiles[b]):
                    sl = slice(T * i, T * i + T)
                    raw_k[u * T:u * T + T], raw_v[u * T:u * T + T] = k[sl], v[sl]
                    table[b, h, i] = place[u] * rb
                    for x, dst in ((k, kb), (v, vb)):
                        _, val, s = quantise(x[sl], code, block)
                        dst[h, sl] = val * s.astype(np.float64).repeat(16)[:, None]
                    sb[h, sl] = s.repeat(16)  # of V, the last one quantised
                    u += 1
                w0 = T * tiles[b]
                for j in range(w0, n, 16):  # prefill's power of two of 16 window rows: 2^8 .. 2^9 at the top
                    sb[h, j:j + 16] = np.abs(v[j:j + 16]).max() / 256
                kb[h, w0:], vb[h, w0:] = k[w0:], v[w0:]
                slots = (self.starts[b] + np.arange(windows[b])) % self.cap
                wk[b, h, slots], wv[b, h, slots] = k[w0:], v[w0:]
            self.k.append(kb)
            self.v.append(vb)
            self.vs.append(sb)
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
        self.tiles = torch.zeros(max(n_units, 1) * rb, dtype=torch.uint8, device=DEV)
        if n_units:
            kvarn.compress_tile8(dev(raw_k), dev(raw_v), torch.arange(n_units, device=DEV) * T, self.tiles,
                                 dev(place.astype(np.int64) * rb), self.lay)
        self.table = dev(table)
        self.n_tiles = torch.tensor(tiles, dtype=torch.int32, device=DEV)
        self.win_k, self.win_v = dev(wk), dev(wv)
        self.win_start = torch.tensor(self.starts, dtype=torch.int32, device=DEV)
        self.win_len = torch.tensor(windows, dtype=torch.int32, device=DEV)

    def args(self):
        return (self.tiles, self.table, self.n_tiles, self.win_k, self.win_v, self.win_start, self.win_len,
                self.lay)

    def decode(self, q, **kw):
        return kvarn.decode_attention8(q, *self.args(), **kw)

    def prefill(self, q, pos0, b=0, **kw):
        return kvarn.prefill_attention8(q, pos0, self.tiles, self.table[b], self.tiles_of[b], self.win_k[b],
                                        self.win_v[b], self.starts[b], self.windows[b], self.lay, **kw)


def attend(q, k, v, scale, visible, vs, floor):
    """q [R, D], k, v [n, D], visible [R] keys per row, vs [n] the scales under v -> out, weights, and the tolerance
    without the output's own half step, all in 64 bits."""
    s = scale * (q @ k.T)
    hide = np.arange(k.shape[0])[None, :] >= np.asarray(visible)[:, None]
    s[hide] = -np.inf
    m = s.max(1, keepdims=True)
    p = np.exp(s - m)
    p /= p.sum(1, keepdims=True)
    size = abs(scale) * (np.abs(q) @ np.abs(k).T)
    size[hide] = 0
    a = 2.0 ** -17 * size.max(1, keepdims=True)
    n = k.shape[0]
    bound = (a + 2.0 ** -20 + (n / 16 + 2) * 2.0 ** -23) * (p @ np.abs(v))
    bound = bound + floor * (p * vs).max(1, keepdims=True) * (np.abs(v) / vs[:, None]).sum(0)
    return p @ v, p, bound


def check(got, want, bound, dtype, extra=0.0, terms=None):
    """got within bound (+ extra of the terms) + half a step of its type around want."""
    got = got.detach().double().cpu().numpy() if torch.is_tensor(got) else got
    tiny = {torch.float32: 1e-37, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-37}[dtype]
    tol = bound + HALF_STEP[dtype] * (np.abs(want) + bound) + tiny
    if extra:
        tol = tol + extra * terms
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} outside, worst "
                           f"{float((np.abs(got - want) / tol)[bad].max()):.3g} x the tolerance at "
                           f"{np.argwhere(bad)[0].tolist()}")
