"""What the 4-bit cache's calls and norm_rotate refuse, on the host: nothing reaches a GPU."""
import ctypes
import random

import pytest
import torch

from kv_cache_quantization_token_gb300 import _build, kvarn
from tests.test_no_fallback import _fake

f32 = ctypes.c_float
P = ctypes.c_void_p(1 << 20)
Q = ctypes.c_void_p(1 << 30)
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvarn._L()


def test_layout(lib):
    for D in (64, 128, 256):
        L = kvarn.layout4(D)
        assert (L.version, L.head_dim, L.tile_tokens, L.run_tokens, L.group_channels) == (1, D, 128, 32, 32)
        assert (L.record_bytes, L.run_bytes) == (144 * D, 36 * D)
        assert (L.off_k_codes, L.off_v_codes, L.off_k_scale, L.off_v_scale) == (0, 16 * D, 32 * D, 34 * D)
    for D in (0, 32, 96, 512, -64):
        assert lib.kvarn_layout4(D, ctypes.byref(kvarn.Layout4())) == -3
    assert lib.kvarn_layout4(128, None) == -1


def _rows(lib, **kw):
    """The same arguments to both row calls."""
    L = kvarn.layout4(128)
    a = dict(k=P, ks=1024, v=Q, vs=1024, io=2, tiles=P, size=1 << 30, table=P, lens=P, counts=None, B=2, T=3, H=8, D=128,
             mt=4, lay=ctypes.byref(L), flags=0, st=None)
    a.update(kw)
    w = lib.kvarn_write_rows4(*a.values())
    r = lib.kvarn_read_rows4(*[a[n] for n in ("tiles", "size", "table", "lens", "counts", "k", "ks", "v", "vs", "io", "B",
                                              "T", "H", "D", "mt", "lay", "flags", "st")])
    assert w == r, kw
    return w


def test_row_refusals(lib):
    bad = kvarn.layout4(128)
    bad.record_bytes += 16
    for k in ("k", "v", "tiles", "table", "lens", "lay"):
        assert _rows(lib, **{k: None}) == -1, k
    for k in ("k", "v", "tiles"):
        assert _rows(lib, **{k: ODD}) == -2, k
    for kw in (dict(table=ctypes.c_void_p((1 << 20) + 4)), dict(lens=ctypes.c_void_p((1 << 20) + 2)),
               dict(counts=ctypes.c_void_p((1 << 20) + 2)), dict(ks=1028), dict(vs=1028), dict(ks=1026, io=0)):
        assert _rows(lib, **kw) == -2, kw
    for kw in (dict(io=3), dict(io=-1), dict(flags=2), dict(flags=4), dict(B=-1), dict(T=-1), dict(H=0), dict(H=65536),
               dict(mt=-1), dict(mt=1 << 24), dict(size=-1), dict(ks=1016), dict(vs=0), dict(vs=-1024), dict(ks=1 << 62),
               dict(B=1 << 30, T=1 << 30), dict(B=(1 << 31) - 1, T=(1 << 31) - 1, H=65535, ks=8388480, vs=8388480)):
        assert _rows(lib, **kw) == -4, kw
    assert _rows(lib, lay=ctypes.byref(bad)) == -3 and _rows(lib, D=64) == -3 and _rows(lib, D=96) == -3
    assert _rows(lib, B=0, k=None) == 0 and _rows(lib, T=0, lens=None) == 0


def test_read_rows_that_overlap(lib):
    L = kvarn.layout4(128)

    def read(k, ks, v, vs):
        return lib.kvarn_read_rows4(None, 0, None, P, None, ctypes.c_void_p(k), ks, ctypes.c_void_p(v), vs, 2, 2, 3, 8,
                                    128, 0, ctypes.byref(L), 2, None)  # (flags stop what is not refused earlier)
    base = 1 << 20
    for v in (base, base + 2032, base + 16):
        assert lib.kvarn_read_rows4(None, 0, None, P, None, ctypes.c_void_p(base), 1024, ctypes.c_void_p(v), 1024, 2, 2, 3,
                                    8, 128, 0, ctypes.byref(L), 0, None) == -4
    assert read(base, 1024, base + 2048, 2048) == -4


def _decode(lib, **kw):
    L = kvarn.layout4(128)
    a = dict(q=P, io=0, tiles=P, size=1 << 30, table=P, lens=P, B=1, Hq=32, Hkv=8, D=128, mt=8, scale=f32(0.1),
             lay=ctypes.byref(L), mi=None, mo=None, ws=P, wsb=1 << 30, out=P, flags=0, st=None)
    a.update(kw)
    return lib.kvarn_decode_attention4(*a.values())


def test_decode_refusals(lib):
    for k in ("q", "tiles", "table", "lens", "lay", "ws", "out"):
        assert _decode(lib, **{k: None}) == -1, k
    for k in ("q", "tiles", "out"):
        assert _decode(lib, **{k: ODD}) == -2, k
    for k, n in (("ws", 128), ("table", 4), ("lens", 2), ("mo", 2)):
        assert _decode(lib, **{k: ctypes.c_void_p((1 << 20) + n)}) == -2, k
    for kw in (dict(io=3), dict(io=-1), dict(size=-1), dict(B=-1), dict(B=65536), dict(Hq=30), dict(Hq=0), dict(Hkv=0),
               dict(mt=-1), dict(mt=1 << 24), dict(flags=2), dict(flags=4), dict(scale=f32(float("nan"))),
               dict(scale=f32(float("inf"))), dict(mi=P), dict(mi=P, mo=ctypes.c_void_p((1 << 20) + 4))):
        assert _decode(lib, **kw) == -4, kw
    assert _decode(lib, Hq=72) == -3 and _decode(lib, D=96) == -3 and _decode(lib, D=64) == -3
    assert _decode(lib, wsb=256) == -5
    assert _decode(lib, B=0) == 0
    assert _decode(lib, B=65535, Hq=8, mt=(1 << 12) + 1) == -4 and _decode(lib, B=128, mt=1 << 21) == -4  # 2^31 entries or more
    n, q = ctypes.c_size_t(), lib.kvarn_decode4_workspace_bytes
    assert q(1, 32, 8, 128, 8, None) == -1 and q(1, 32, 8, 96, 8, ctypes.byref(n)) == -3
    assert q(2, 32, 8, 128, 8, ctypes.byref(n)) == 0 and n.value % 256 == 0
    # every (head, item) row and every run's eight (maximum, sum) pairs have room
    assert n.value >= 2 * 32 * (128 * 4 + 8) + 2 * 8 * 8 * 4 * 64


def test_decode_workspaces_with_and_without_weights(lib):
    for B, Hq, Hkv, D, mt in ((1, 32, 8, 128, 8), (3, 6, 2, 64, 100), (256, 8, 8, 256, 1024)):
        L = kvarn.layout4(D)
        both = kvarn.decode4_workspace_bytes(B, Hq, Hkv, D, mt)
        plain = kvarn.decode4_workspace_bytes(B, Hq, Hkv, D, mt, weights=False)
        assert 0 < plain < both and plain % 256 == 0 and both - plain == 256 * B * Hkv * mt
        sizes = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, mt=mt, lay=ctypes.byref(L))
        assert _decode(lib, **sizes, wsb=plain - 256) == -5
        assert _decode(lib, **sizes, wsb=plain, mo=P) == -5 and _decode(lib, **sizes, wsb=both - 1, mo=P) == -5
        # enough of it: what is refused next is the workspace's alignment
        assert _decode(lib, **sizes, wsb=plain, ws=ctypes.c_void_p((1 << 20) + 128)) == -2
        assert _decode(lib, **sizes, wsb=both, mo=P, ws=ctypes.c_void_p((1 << 20) + 128)) == -2


def _prefill(lib, **kw):
    L = kvarn.layout4(128)
    a = dict(q=P, io=0, C=16, pos0=100, tiles=P, size=1 << 30, table=P, stride=2, Hq=32, Hkv=8, D=128, scale=f32(0.1),
             lay=ctypes.byref(L), ws=P, wsb=1 << 30, out=P, st=None)
    a.update(kw)
    return lib.kvarn_prefill_attention4(*a.values())


def test_prefill_refusals(lib):
    for k in ("q", "tiles", "table", "lay", "ws", "out"):
        assert _prefill(lib, **{k: None}) == -1, k
    for k in ("q", "tiles", "out"):
        assert _prefill(lib, **{k: ODD}) == -2, k
    assert _prefill(lib, table=ctypes.c_void_p((1 << 20) + 4)) == -2
    assert _prefill(lib, ws=ctypes.c_void_p((1 << 20) + 128)) == -2
    for kw in (dict(io=3), dict(C=-1), dict(pos0=-1), dict(pos0=241), dict(pos0=(1 << 63) - 1), dict(stride=0),
               dict(stride=1 << 24), dict(Hq=30), dict(size=-1), dict(scale=f32(float("nan"))),
               dict(scale=f32(float("-inf")))):
        assert _prefill(lib, **kw) == -4, kw
    assert _prefill(lib, Hq=72) == -3 and _prefill(lib, D=64) == -3 and _prefill(lib, D=100) == -3
    assert _prefill(lib, wsb=1 << 10) == -5
    assert _prefill(lib, C=0) == 0
    # tiles of all heads are counted in 32 bits, with up to 64 groups of rows
    many = dict(Hq=64, Hkv=64, C=1, stride=1 << 19, pos0=(1 << 26) - 1)
    assert _prefill(lib, **many) == -4 and _prefill(lib, **{**many, "pos0": (1 << 26) - 129, "wsb": 256}) == -5
    n = ctypes.c_size_t()
    query = lib.kvarn_prefill4_workspace_bytes
    assert query(1, 1 << 19, 64, 64, 128, ctypes.byref(n)) == -4 and query(1, (1 << 19) - 1, 64, 64, 128, ctypes.byref(n)) == 0


def test_a_prefill_workspace_serves_smaller_chunks(lib):
    rng = random.Random(3)
    for _ in range(300):
        D, Hkv, G = rng.choice([64, 128, 256]), rng.randint(1, 8), rng.randint(1, 8)
        C, n = rng.randint(1, 800), rng.randint(1, 200)
        most = kvarn.prefill4_workspace_bytes(C, n, Hkv * G, Hkv, D)
        for _ in range(20):
            assert kvarn.prefill4_workspace_bytes(rng.randint(0, C), rng.randint(0, n), Hkv * G, Hkv, D) <= most


def test_rotary(lib):
    R = kvarn.rotary(64, theta=500000.0, sections=(8, 12, 12), pairing="adjacent")
    assert (R.version, R.rotary_dim, R.pairing, R.n_axes) == (1, 64, 1, 3)
    assert list(R.axis)[:32] == [0] * 8 + [1] * 12 + [2] * 12 and not any(list(R.axis)[32:])
    # turns of 2^-64, to the last: 1 / 2 pi, a negative frequency, one of many turns, the smallest
    from fractions import Fraction
    from tests.cache4_helpers import INV_2PI
    f = [1.0, -1.0, 1000.25, 2.0 ** -60, 5e-324, 0.0, 1 / 3, 1024.0]
    R = kvarn.rotary(16, inv_freq=f)
    for x, got in zip(f, R.turn):
        t = Fraction(abs(x)) * INV_2PI * 2 ** 64
        t = t.numerator // t.denominator % 2 ** 64
        assert got == (t if x >= 0 else -t % 2 ** 64)
    C = kvarn.Rotary()
    d, u = (ctypes.c_double * 8)(*[1.0] * 8), (ctypes.c_uint8 * 8)(*[2] * 8)
    call = lambda *a: lib.kvarn_rotary(*a, ctypes.byref(C))
    assert call(16, 0, None, None, 1) == -1 and lib.kvarn_rotary(16, 0, d, None, 1, None) == -1
    for n in (0, 8, 24, 272, -16):
        assert call(n, 0, d, None, 1) == -3
    assert call(16, 2, d, None, 1) == -4 and call(16, 0, d, None, 0) == -4 and call(16, 0, d, None, 5) == -4
    assert call(16, 0, d, u, 2) == -4 and call(16, 0, d, u, 3) == 0
    for x in (float("nan"), float("inf"), 1025.0, -1e300):
        d[3] = x
        assert call(16, 0, d, None, 1) == -4
    for kw in (dict(pairing="pairs"), dict(inv_freq=[1.0] * 9), dict(sections=(4, 5)), dict(pair_axis=[0] * 7),
               dict(sections=(8,), pair_axis=[0] * 8), dict(pair_axis=[4] * 8), dict(pair_axis=[-1] * 8)):
        with pytest.raises(ValueError):
            kvarn.rotary(16, **kw)


def _rope(lib, **kw):
    R = kvarn.rotary(128)
    a = dict(q=ctypes.c_void_p(1 << 24), qs=4096, k=ctypes.c_void_p(2 << 24), ks=1024, io=2, n=5, Hq=32, Hkv=8, D=128,
             qw=P, kw=P, eps=f32(1e-6), pos=ODD, rot=ctypes.byref(R), had=1, qo=ctypes.c_void_p(3 << 24), qos=4096,
             ko=ctypes.c_void_p(4 << 24), kos=1024, flags=0, st=None)
    a.update(kw)
    return lib.kvarn_norm_rotate(*a.values())


def test_norm_rotate_refusals(lib):
    for k in ("q", "k", "qo", "ko", "pos"):
        assert _rope(lib, **{k: None}) == -1, k
    for k in ("q", "k", "qo", "ko", "qw", "kw"):
        assert _rope(lib, **{k: ODD}) == -2, k
    assert _rope(lib, pos=ctypes.c_void_p((1 << 20) + 4)) == -2
    for k in ("qs", "qos", "ks", "kos"):
        assert _rope(lib, **{k: 4100}) == -2 and _rope(lib, **{k: 512}) == -4 and _rope(lib, **{k: 1 << 62}) == -4, k
    for kw in (dict(io=3), dict(flags=2), dict(flags=8), dict(n=-1), dict(n=1 << 31), dict(Hq=0), dict(Hkv=-1), dict(Hq=65536),
               dict(eps=f32(float("nan"))), dict(eps=f32(float("inf"))), dict(eps=f32(-1)), dict(Hkv=0)):
        assert _rope(lib, **kw) == -4, kw
    assert _rope(lib, D=96) == -3 and _rope(lib, D=64, qs=4096) == -3  # the plan turns more channels than a head has
    wrong = kvarn.rotary(128)
    for field, x in (("version", 2), ("rotary_dim", 136), ("rotary_dim", 0), ("pairing", 2), ("n_axes", 0), ("n_axes", 5)):
        R = kvarn.rotary(128)
        setattr(R, field, x)
        assert _rope(lib, rot=ctypes.byref(R)) == -3, field
    wrong.axis[63] = 1
    assert _rope(lib, rot=ctypes.byref(wrong)) == -3
    assert _rope(lib, n=0, q=None) == 0


def test_norm_rotate_refuses_rows_that_meet(lib):
    at = ctypes.c_void_p
    q, k = 1 << 24, (1 << 24) + 8192  # rows of 32 + 8 + 8 heads of 128 bf16, packed: 12,288 bytes apart
    same = dict(q=at(q), qs=6144, k=at(k), ks=6144, flags=0)
    for kw in (dict(qo=at(q + 16), qos=6144), dict(qo=at(q), qos=6152), dict(qo=at(k), qos=6144), dict(ko=at(q), kos=6144),
               dict(ko=at(k - 16), kos=6144), dict(ko=at(k + 12288), kos=6144), dict(qo=at(3 << 24), ko=at(3 << 24)),
               dict(qo=at(3 << 24), qos=4096, ko=at((3 << 24) + 8192), kos=4096), dict(qo=at((1 << 20) - 16)),
               dict(ko=at((1 << 20) + 240))):
        assert _rope(lib, **{**same, **kw}) == -4, kw


def test_the_binding_refuses_what_the_kernels_cannot_use():
    lay = kvarn.layout4(128)
    x = torch.zeros(2, 3, 2, 128)
    tiles, table, n = torch.zeros(18432, dtype=torch.uint8), torch.zeros(2, 2, 1, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    for i in range(2):  # (the others are compared with the device of these)
        a = [_fake(t) for t in (x, x, tiles, table, n)]
        a[i] = (x, x, tiles, table, n)[i]
        with pytest.raises(TypeError, match="must be a CUDA tensor"):
            kvarn.write_rows4(*a, lay)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        kvarn.read_rows4(tiles, table, n, x, x, lay)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        kvarn.decode_attention4(x[0], tiles, table, n, lay)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        kvarn.prefill_attention4(x[0], 0, tiles, table[0], lay)
    with pytest.raises(TypeError, match="must be a CUDA tensor"):
        kvarn.norm_rotate(x[0], x[0], torch.zeros(3, dtype=torch.int64), kvarn.rotary(128))
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        kvarn.norm_rotate(_fake(x[0].double()), None, None, None)


def test_row_strides():
    stride = lambda t, dims: kvarn._rows_of(_fake(t), "x", dims)[0]
    x = torch.zeros(4, 6, 10, 64)
    assert stride(x, 4) == 640
    assert stride(x[:, :, 2:5], 4) == 640 and stride(x[:, 1:2, 2:5], 4) == 6 * 640 and stride(x[2:3, :, 2:5], 4) == 640
    assert stride(x[:1, :1, :3], 4) == 192 and stride(x[1], 3) == 640 and stride(x[1, :, 4:6], 3) == 640
    assert stride(x[::2, :1], 4) == 2 * 6 * 640 and stride(x[:, ::2][:1], 4) == 2 * 640
    for bad in (x[..., ::2], x[:, :, ::2], x[..., :32], x.transpose(1, 2), x[:, :5], x[:, ::2][:, :2]):
        with pytest.raises(ValueError):
            stride(bad, 4)
    with pytest.raises(ValueError):
        stride(x, 3)
