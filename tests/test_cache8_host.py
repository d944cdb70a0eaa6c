"""What the 8-bit cache's calls and eviction refuse, on the host: nothing reaches a GPU."""
import ctypes
import os
import random
import re

import pytest
import torch

from kv_cache_quantization_token_gb300 import _build, kvarn

f32 = ctypes.c_float
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvarn._L()


def test_layout(lib):
    for D in (64, 128, 256):
        L = kvarn.layout8(D, "e4m3", 32)
        assert L.record_bytes == 256 * D + 128 and L.record_bytes % 128 == 0
        assert (L.off_k_codes, L.off_v_codes, L.off_k_scale, L.off_v_scale) == (0, 128 * D, 256 * D, 256 * D + 32)
        assert (L.version, L.head_dim, L.tile_tokens, L.code_format, L.block_tokens) == (1, D, 128, 1, 32)
    L = kvarn.Layout8()
    for D, f, b in ((96, 0, 64), (512, 0, 64), (128, 2, 64), (128, -1, 64), (128, 0, 8), (128, 0, 256), (128, 0, 48)):
        assert lib.kvarn_layout8(D, f, b, ctypes.byref(L)) == -3
    assert lib.kvarn_layout8(128, 0, 64, None) == -1
    with pytest.raises(ValueError, match="code must be one of"):
        kvarn.layout8(128, "e5m2")
    with pytest.raises(kvarn.KvarnError):
        kvarn.layout8(128, "i8", 20)


def test_compress_and_expand_refusals(lib):
    L = kvarn.layout8(128)
    rb, lay = L.record_bytes, ctypes.byref(L)
    bad = kvarn.layout8(128)
    bad.record_bytes += 16
    ok = [P, P, 128, 256, P, P, rb, P, 1, lay, None]

    def both(i, x, want):
        a = list(ok)
        a[i] = x
        assert lib.kvarn_compress_tile8(*a) == want
        k, v, stride, n, rows, tiles, size, recs, units, y, st = a
        assert lib.kvarn_expand_tile8(tiles, size, recs, k, v, stride, n, rows, units, y, st) == want
    for i in (0, 1, 4, 5, 7):
        both(i, None, -1)
    for i in (0, 1, 5):
        both(i, ODD, -2)
    both(2, 130, -2)
    for i, x in ((2, 64), (2, -128), (3, 127), (3, -1), (6, rb - 1), (6, -1), (8, -1), (8, 1 << 30)):
        both(i, x, -4)
    both(8, 0, 0)
    both(9, None, -1)
    both(9, ctypes.byref(bad), -3)


def _decode(lib, **kw):
    L = kvarn.layout8(128)
    a = dict(q=P, io=0, tiles=P, tiles_bytes=1 << 30, table=P, n=P, wk=P, wv=P, ws_=P, wl=P, cap=128, B=1, Hq=32, Hkv=8,
             D=128, mt=8, scale=f32(0.1), lay=ctypes.byref(L), mi=None, mo=None, ws=P, wsb=1 << 30, out=P, flags=0,
             st=None)
    a.update(kw)
    return lib.kvarn_decode_attention8(*a.values())


def test_decode_refusals(lib):
    for k in ("q", "tiles", "table", "n", "wk", "wv", "ws_", "wl", "lay", "ws", "out"):
        assert _decode(lib, **{k: None}) == -1, k
    for k in ("q", "tiles", "wk", "wv", "out"):
        assert _decode(lib, **{k: ODD}) == -2, k
    assert _decode(lib, ws=ctypes.c_void_p((1 << 20) + 128)) == -2
    for k in ("table", "n", "ws_", "wl"):
        assert _decode(lib, **{k: ctypes.c_void_p((1 << 20) + 2)}) == -2, k
    assert _decode(lib, table=ctypes.c_void_p((1 << 20) + 4)) == -2
    assert _decode(lib, mo=ctypes.c_void_p((1 << 20) + 2)) == -2
    assert _decode(lib, mt=(1 << 29) + 1) == -4 and _decode(lib, cap=(1 << 29) + 1) == -4
    for kw in (dict(io=3), dict(io=-1), dict(tiles_bytes=-1), dict(cap=-1), dict(B=-1), dict(B=65536), dict(Hq=30),
               dict(Hq=0), dict(Hkv=0), dict(mt=-1), dict(flags=4), dict(flags=2), dict(scale=f32(float("nan"))),
               dict(mi=P), dict(mi=P, mo=ctypes.c_void_p((1 << 20) + 4))):
        assert _decode(lib, **kw) == -4, kw
    assert _decode(lib, Hq=72) == -3 and _decode(lib, D=96) == -3 and _decode(lib, D=64) == -3
    assert _decode(lib, wsb=256) == -5
    assert _decode(lib, B=0) == 0
    n = ctypes.c_size_t()
    q = lib.kvarn_decode8_workspace_bytes
    assert q(1, 32, 8, 128, 8, 128, None) == -1 and q(1, 32, 8, 96, 8, 128, ctypes.byref(n)) == -3
    assert q(2, 32, 8, 128, 8, 128, ctypes.byref(n)) == 0 and n.value % 256 == 0
    # every (head, item) row and every tile's eight (maximum, sum) pairs have room
    assert n.value >= 2 * 32 * (8 + 2) * (128 * 4 + 8) + 2 * 8 * 8 * 64


def _prefill(lib, **kw):
    L = kvarn.layout8(128)
    a = dict(q=P, io=0, C=16, pos0=100, tiles=P, tiles_bytes=1 << 30, table=P, stride=4, nt=2, wk=P, wv=P, start=0, wl=16,
             cap=128, Hq=32, Hkv=8, D=128, scale=f32(0.1), lay=ctypes.byref(L), ws=P, wsb=1 << 30, out=P, st=None)
    a.update(kw)
    return lib.kvarn_prefill_attention8(*a.values())


def test_prefill_refusals(lib):
    for k in ("q", "tiles", "table", "wk", "wv", "lay", "ws", "out"):
        assert _prefill(lib, **{k: None}) == -1, k
    for k in ("q", "tiles", "wk", "wv", "out"):
        assert _prefill(lib, **{k: ODD}) == -2, k
    for kw in (dict(io=3), dict(C=-1), dict(pos0=-1), dict(pos0=257), dict(pos0=(1 << 63) - 1), dict(stride=1), dict(nt=-1),
               dict(wl=-1), dict(wl=129), dict(cap=-1), dict(Hq=30), dict(tiles_bytes=-1), dict(scale=f32(float("nan")))):
        assert _prefill(lib, **kw) == -4, kw
    assert _prefill(lib, Hq=72) == -3 and _prefill(lib, D=64) == -3 and _prefill(lib, D=100) == -3
    assert _prefill(lib, wsb=1 << 10) == -5
    assert _prefill(lib, table=ctypes.c_void_p((1 << 20) + 4)) == -2
    many, most = (1 << 29) + 1, ctypes.c_size_t()
    assert _prefill(lib, nt=many, stride=many) == -4 and _prefill(lib, cap=many) == -4
    query = lib.kvarn_prefill8_workspace_bytes
    assert query(512, many, 0, 32, 8, 128, ctypes.byref(most)) == -4 and query(512, 0, many, 32, 8, 128, ctypes.byref(most)) == -4
    # the largest sizes are counted without wrapping: images of every tile, fp16 K and V
    assert query(512, 1 << 29, 1 << 29, 32, 8, 256, ctypes.byref(most)) == 0 and most.value > 8 * 2 * 128 * 512 << 29
    assert _prefill(lib, C=0) == 0


def test_the_largest_chunks_are_counted_without_wrapping(lib):
    n, below = ctypes.c_size_t(), ctypes.c_size_t()
    query = lib.kvarn_prefill8_workspace_bytes
    assert query((1 << 31) - 1, 1 << 24, 0, 8, 8, 64, ctypes.byref(n)) == 0
    assert query((1 << 31) - 128, 1 << 24, 0, 8, 8, 64, ctypes.byref(below)) == 0
    assert below.value <= n.value < 2 * below.value


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 8), (4, 3), (8, 4), (40, 2)])
def test_a_workspace_serves_every_smaller_chunk(lib, Hkv, G, D):
    """What the query gives is not refused for fewer positions, tiles or window rows, on either kind of kernels: an
    unaligned output, looked at after the workspace, is."""
    L, rng = kvarn.layout8(D), random.Random(Hkv * D)
    log = lambda top: min(top, int(round(2 ** rng.uniform(0, 12)))) if rng.random() < 0.9 else 0
    for _ in range(400):
        n, w = log(900), log(3500)
        C = max(1, min(log(2000), 128 * n + w))
        size = kvarn.prefill8_workspace_bytes(C, n, w, Hkv * G, Hkv, D)
        for _ in range(12):
            n1, w1 = rng.choice([n, log(n)]), rng.choice([w, log(w)])
            C1 = min(rng.choice([C, max(1, log(C)), rng.randint(1, C)]), 128 * n1 + w1)
            if C1 == 0:
                continue
            rc = _prefill(lib, C=C1, pos0=128 * n1 + w1 - C1, nt=n1, stride=n1, wl=w1, cap=w1, Hq=Hkv * G, Hkv=Hkv, D=D,
                          lay=ctypes.byref(L), wsb=size, out=ODD)
            assert rc == -2, (rc, (C, n, w), (C1, n1, w1))


def test_the_window_counts_in_the_choice_of_kernels(lib):
    """A chunk of 512 rows per KV head over a long window alone runs on images of it, whose size the workspace shows
    (fp16 pairs of K and V in blocks of 32 keys), not on kernels that read the window again for every eight rows."""
    images = lambda w: 8 * -(-w // 64) * 2 * 2 * 2 * 64 * 128
    assert images(3000) <= kvarn.prefill8_workspace_bytes(128, 0, 3000, 32, 8, 128) < 2 * images(3000)
    # few rows do without them
    assert kvarn.prefill8_workspace_bytes(2, 0, 3000, 32, 8, 128) < images(3000) // 4


def _evict(lib, **kw):
    a = dict(t=ctypes.c_void_p(1 << 20), m=ctypes.c_void_p(2 << 20), n=ctypes.c_void_p(3 << 20), to=ctypes.c_void_p(4 << 20),
             mo=ctypes.c_void_p(5 << 20), no=ctypes.c_void_p(6 << 20), ev=ctypes.c_void_p(7 << 20), B=0, Hkv=2, mt=10, keep=5,
             sinks=1, recent=1, flags=0, st=None)
    a.update(kw)
    return lib.kvarn_evict_tiles(*a.values())


def test_evict_refusals(lib):
    assert _evict(lib) == 0  # no sequences
    for k in ("t", "m", "n", "to", "mo", "no"):
        assert _evict(lib, B=1, **{k: None}) == -1, k
    for kw in (dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(sinks=3, recent=3), dict(mt=-1), dict(Hkv=0), dict(B=-1),
               dict(flags=4), dict(flags=2), dict(B=1, to=ctypes.c_void_p((1 << 20) + 8)), dict(B=1, ev=ctypes.c_void_p(4 << 20)),
               dict(B=1, mo=ctypes.c_void_p(1 << 20)), dict(B=1, no=ctypes.c_void_p(3 << 20 | 4), n=ctypes.c_void_p(3 << 20)) | dict(B=2),
               dict(B=1, ev=ctypes.c_void_p(2 << 20))):
        assert _evict(lib, **kw) == -4, kw
    assert _evict(lib, B=1, t=ctypes.c_void_p((1 << 20) + 4)) == -2
    assert _evict(lib, B=65536) == -4 and _evict(lib, mt=(1 << 29) + 1) == -4
    assert _evict(lib, flags=kvarn.LAUNCH_PDL | kvarn.LAUNCH_PREFETCH) == -4


def test_evict_refuses_counts_inside_the_other_arrays(lib):
    """Read while they are written, or written over them."""
    inside = {k: ctypes.c_void_p((i << 20) + 8) for i, k in enumerate(("t", "m", "n", "to", "mo", "no", "ev"), 1)}
    for count, others in (("n", ("to", "mo", "ev")), ("no", ("t", "m", "to", "mo", "ev"))):
        for k in others:
            assert _evict(lib, B=1, **{count: inside[k]}) == -4, (count, k)


def test_compression_gives_up_as_a_whole_cta():
    """A wait can run out for some threads of a CTA alone. What each of them saw must not decide a branch before the
    CTA has joined it: the branches of the loop have barriers."""
    with open(os.path.join(_build.CSRC, "compress8.cu")) as f:
        body = f.read().split("compress8_kernel(")[1].split("\n}\n")[0]
    verdict = re.findall(r"(?:if|=|&&|\|\|)[ (!]*mbar_wait8\(", body)
    name = re.findall(r"const bool (\w+) = mbar_wait8\(", body)
    assert len(verdict) == len(name) == 1
    uses = re.findall(r"[^\n]*\b%s\b[^\n]*" % name[0], body)
    assert len(uses) == 2 and "if (!__syncthreads_and(%s)) break;" % name[0] in uses[1]


def test_decode_waits_again_for_a_copy_that_it_gave_up_on():
    """A copy whose wait ran out still writes to the CTA's shared memory: the CTA does not end before it is given as
    long again."""
    with open(os.path.join(_build.CSRC, "decode8.cu")) as f:
        body = f.read().split("split8_kernel(")[1].split("\n}\n")[0]
    end = body[body.index("const bool bad = *flag != 0;"):]
    assert re.search(r"if \(bad && tid == 0\) \{[^}]*mbar_wait8\([^}]*nullptr\);\s*\}", end)


def test_host_tensors_are_refused():
    lay = kvarn.layout8(128)
    x, i64 = torch.zeros(128, 128), torch.zeros(1, dtype=torch.int64)
    u8 = torch.zeros(lay.record_bytes, dtype=torch.uint8)
    q, tab, n, win = torch.zeros(1, 8, 128), torch.zeros(1, 2, 1, dtype=torch.int64), torch.ones(1, dtype=torch.int32), \
        torch.zeros(1, 2, 128, 128)
    for call in (lambda: kvarn.compress_tile8(x, x, i64, u8, i64, lay),
                 lambda: kvarn.expand_tile8(u8, i64, x, x, i64, lay),
                 lambda: kvarn.decode_attention8(q, u8, tab, n, win, win, n, n, lay),
                 lambda: kvarn.prefill_attention8(q, 0, u8, tab[0], 1, win[0], win[0], 0, 4, lay),
                 lambda: kvarn.evict_tiles(tab, torch.zeros(1, 2, 1), n, 1)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
