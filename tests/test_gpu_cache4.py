"""The 4-bit cache on the GPU against plain 64-bit statements of its operators."""
import numpy as np
import pytest
import torch

from kv_cache_quantization_token_gb300 import kvarn
from tests.cache4_helpers import (DEV, HALF_STEP, MAX4, T, Cache4, attend, check, poisoned, put_token, quantise,  # noqa: F401
                                  rows)

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def no_device_error():
    kvarn.device_error()
    yield
    assert kvarn.device_error() == 0


def _query(seed, shape, io):
    q = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32))
    return q.to(IO[io]).to(DEV)


def _dev(x, dtype=None):
    return torch.tensor(x, dtype=dtype, device=DEV)


# ---------------------------------------------------------------- rows in and out

class _Store:
    """An empty cache of B sequences in a pool of 0xA5 bytes."""

    def __init__(self, B, Hkv, D, max_tiles, seed=0):
        self.D, self.lay = D, kvarn.layout4(D)
        n = B * Hkv * max_tiles
        self.place = np.random.default_rng(seed).permutation(n + 1)[:n].reshape(B, Hkv, max_tiles)
        self.tiles = torch.full(((n + 1) * self.lay.record_bytes,), 0xA5, dtype=torch.uint8, device=DEV)
        self.table = torch.from_numpy(self.place * self.lay.record_bytes).to(DEV)

    def write(self, k, v, lens, counts=None, **kw):
        kvarn.write_rows4(k, v, self.tiles, self.table, _dev(lens, torch.int32), self.lay,
                          counts=None if counts is None else _dev(counts, torch.int32), **kw)

    def read(self, k, v, first, counts=None, **kw):
        kvarn.read_rows4(self.tiles, self.table, _dev(first, torch.int32), k, v, self.lay,
                         counts=None if counts is None else _dev(counts, torch.int32), **kw)

    def records(self):
        return self.tiles.cpu().numpy().reshape(-1, self.lay.record_bytes)

    def expect(self, k, v, lens, counts):
        """The pool after rows k, v (host fp32 [B, T, H, D]) were written into the pool as it is now."""
        want = self.records().copy()
        B, n, H, D = k.shape
        bad = poisoned(k, v)
        k, v = np.where(bad[..., None], 0, k), np.where(bad[..., None], 0, v)
        (kc, ks), (vc, vs) = quantise(k), quantise(v)
        ks[bad], vs[bad] = np.nan, 0
        ks, vs = ks.astype(np.float16), vs.astype(np.float16)
        for b in range(B):
            for t in range(min(max(counts[b], 0), n)):
                at = lens[b] + t
                if not 0 <= lens[b] or at >= T * self.place.shape[2]:
                    continue
                for h in range(H):
                    put_token(want[self.place[b, h, at // T]], D, at % T, kc[b, t, h], ks[b, t, h], vc[b, t, h],
                              vs[b, t, h])
        return want


def _same_bytes(got, want):
    """Equal but for which NaN a NaN scale is."""
    g, w = got.view(np.uint16), want.view(np.uint16)
    nan = np.isnan(got.view(np.float16)) & np.isnan(want.view(np.float16))
    assert ((g == w) | nan).all()


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_written_records_are_bit_exact(D, io):
    B, n, H = 3, 37, 3
    rng = np.random.default_rng(D)
    k, v = (x.reshape(B, n, H, D) for x in rows(rng, B * n * H, D))
    k[0, 3] = 0
    v[1, 5] *= np.float32(1e-6)
    k[2, 7] *= np.float32(1e-20)
    v[2, 9] = -0.0
    k, v = (torch.from_numpy(x.copy()).to(IO[io]) for x in (k, v))
    lens, counts = [0, 110, 250], [37, 20, 5]
    c = _Store(B, H, D, 2, seed=D)
    want = c.expect(k.float().numpy(), v.float().numpy(), lens, counts)
    c.write(k.to(DEV), v.to(DEV), lens, counts)
    _same_bytes(c.records(), want)
    # a second call behind the first, all rows of it, with launches chained
    want = c.expect(k.float().numpy()[:, :6], v.float().numpy()[:, :6], [37, 130, 240], [6] * 3)
    c.write(k[:, :6].contiguous().to(DEV), v[:, :6].contiguous().to(DEV), [37, 130, 240], flags=kvarn.LAUNCH_PDL)
    _same_bytes(c.records(), want)


def test_borders_of_codes_and_scales():
    """Elements on every middle of two codes and a step of fp32 to either side, under scales of many sizes, and groups
    whose largest magnitude is on or next to seven times a scale: all decided as the exact quotient is."""
    D, up = 64, np.float32(np.inf)
    out = []
    for s in [2.0 ** -24, 3 * 2.0 ** -24, 255 * 2.0 ** -24, 129 * 2.0 ** -23, 2.0 ** -17, 255 * 2.0 ** -20, 131 / 128, 0.25,
              191 / 64, 2048.0, 2040.0]:
        mids = np.float32((np.arange(7) + 0.5) * s)
        x = np.concatenate([mids, np.nextafter(mids, up), np.nextafter(mids, -up), [np.float32(7 * s)], np.zeros(10)])
        x = np.float32(x)
        for top in (np.float32(7 * s), np.nextafter(np.float32(7 * s), -up), np.nextafter(np.float32(7 * s), up)):
            if top > MAX4:
                continue
            y = x.copy()
            y[21] = top
            out.append(np.concatenate([y, -y]))
    rng = np.random.default_rng(0)
    for _ in range(400):  # largest magnitudes next to seven times a number of nine bits
        top = np.float32(7 * rng.integers(256, 512) * 2.0 ** rng.integers(-34, 2))
        for t in (top, np.nextafter(top, up), np.nextafter(top, -up)):
            y = np.float32(rng.uniform(-1, 1, 64)) * t
            y[5] = t
            out.append(y)
    k = np.minimum(np.stack(out), np.float32(MAX4)).astype(np.float32)[None, :, None]
    v = -k[:, ::-1].copy()
    c = _Store(1, 1, D, -(-k.shape[1] // T))
    want = c.expect(k, v, [0], [k.shape[1]])
    c.write(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), [0])
    _same_bytes(c.records(), want)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_read_back_are_the_values_and_nothing_else_is_written(D, io):
    B, n, H = 2, 150, 3
    k, v = (torch.from_numpy(x.reshape(B, n, H, D)).to(IO[io]) for x in rows(np.random.default_rng(D + 1), B * n * H, D))
    c = _Store(B, H, D, 3)
    c.write(k.to(DEV), v.to(DEV), [100, 7])
    packed = torch.full((B, 40, 2 * H + 1, D), 7.0, dtype=IO[io], device=DEV)
    ko, vo = packed[:, :, 1:H + 1], packed[:, :, H + 1:]
    c.read(ko, vo, [123, 9], [40, 33], flags=kvarn.LAUNCH_PDL)
    for b, first, count, len0 in ((0, 123, 40, 100), (1, 9, 33, 7)):
        for got, x in ((ko, k), (vo, v)):
            q, s = quantise(x[b, first - len0:first - len0 + count].float().numpy())
            want = torch.from_numpy(q * s.repeat(32, -1)).to(IO[io])
            assert torch.equal(got[b, :count].cpu(), want)
            assert bool((got[b, count:] == 7).all())
    assert bool((packed[:, :, 0] == 7).all())


def test_rows_of_packed_products_and_single_tokens():
    """k and v as slices of what one product makes; a batch of single tokens whose axis of one has any stride."""
    D, H, B = 128, 4, 5
    x = _query(1, (B, 7, 3 * H, D), "bf16")
    a, b = _Store(B, H, D, 1), _Store(B, H, D, 1)
    a.write(x[:, :, H:2 * H], x[:, :, 2 * H:], [3] * B)
    b.write(x[:, :, H:2 * H].contiguous(), x[:, :, 2 * H:].contiguous(), [3] * B)
    assert torch.equal(a.tiles, b.tiles)
    one = x[:, 2]                                                 # [B][3 H][D], rows 7 * 3 H * D apart
    a.write(one[:, None, H:2 * H], one[:, None, 2 * H:], [60] * B)
    b.write(one[:, None, H:2 * H].contiguous(), one[:, None, 2 * H:].contiguous(), [60] * B)
    assert torch.equal(a.tiles, b.tiles) and int((a.tiles != 0xA5).sum()) > 0


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 14344.0, -3e38])
@pytest.mark.parametrize("in_v", [False, True])
def test_a_row_that_cannot_be_held_is_poison(bad, in_v):
    D, H = 128, 2
    k, v = (x.reshape(1, 9, H, D) for x in rows(np.random.default_rng(2), 9 * H, D))
    k[0, 0, 0, 3] = MAX4  # the largest that can
    (v if in_v else k)[0, 4, 1, 77] = bad
    c = _Store(1, H, D, 1)
    want = c.expect(k, v, [30], [9])
    c.write(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), [30])
    _same_bytes(c.records(), want)
    ko, vo = (torch.zeros(1, 9, H, D, device=DEV) for _ in "kv")
    c.read(ko, vo, [30])
    nan = torch.zeros(1, 9, H, D, dtype=torch.bool)
    nan[0, 4, 1] = True
    assert torch.equal(ko.isnan().cpu(), nan) and torch.equal(vo.isnan().cpu(), nan)


def test_tokens_outside_their_table_or_pool_are_skipped():
    D, H, B = 64, 2, 4
    k, v = (torch.from_numpy(x.reshape(B, 6, H, D)) for x in rows(np.random.default_rng(3), B * 6 * H, D))
    c = _Store(B, H, D, 2)
    lens = [253, -1, 2 ** 31 - 3, 0]
    want = c.expect(k.numpy(), v.numpy(), lens, [6] * 4)
    c.write(k.to(DEV), v.to(DEV), lens)
    assert kvarn.device_error() == kvarn.DEVERR_WINDOW
    _same_bytes(c.records(), want)
    ko, vo = (torch.full((B, 6, H, D), 7.0, device=DEV) for _ in "kv")
    c.read(ko, vo, lens)
    assert kvarn.device_error() == kvarn.DEVERR_WINDOW
    assert bool((ko[0, 3:] == 7).all()) and bool((ko[1:3] == 7).all()) and not bool((ko[0, :3] == 7).any())
    before = c.tiles.clone()
    for off in (-16, 8, c.tiles.numel() - c.lay.record_bytes + 16, 1 << 62):
        old = c.table.clone()
        c.table[3, 1, 0] = off
        c.write(k.to(DEV) * 2, v.to(DEV), [300, 300, 300, 0], [0, 0, -5, 6])
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
        ko, vo = (torch.full((B, 6, H, D), 7.0, device=DEV) for _ in "kv")
        c.read(ko, vo, [0, 0, 0, 0], [0, 0, 0, 6])
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
        for x in (ko, vo):
            assert bool(x[3, :, 1].isnan().all()) and bool(x[3, :, 0].isfinite().all()) and bool((x[:3] == 7).all())
        c.table.copy_(old)
    changed = (c.tiles != before).view(-1, c.lay.record_bytes).any(1).cpu().numpy()
    assert changed.nonzero()[0].tolist() == [int(c.place[3, 0, 0])]


def test_rows_of_nothing():
    c = _Store(2, 2, 64, 1)
    before = c.tiles.clone()
    x = torch.zeros(2, 3, 2, 64, device=DEV)
    c.write(x, x.clone(), [0, 0], [0, 0])
    c.write(x[:, :0], x[:, :0], [0, 0])
    c.write(x, x.clone(), [0, 0], [-1, -(2 ** 31)])
    c.read(x, x.clone(), [0, 0], [0, 0])
    assert torch.equal(c.tiles, before)
    e = torch.zeros(2, 2, 0, dtype=torch.int64, device=DEV)
    kvarn.write_rows4(x, x.clone(), torch.zeros(0, dtype=torch.uint8, device=DEV), e, _dev([0, 0], torch.int32), c.lay,
                      counts=_dev([0, 0], torch.int32))


# ---------------------------------------------------------------- decode

def _check_decode(c, q, out, scale=None, mass=None, mass_in=None, bound_extra=0.0):
    B, Hq, D = q.shape
    G = Hq // c.Hkv
    qn = q.double().cpu().numpy()
    scale = D ** -0.5 if scale is None else scale
    for b in range(B):
        n = c.k[b].shape[1]
        for h in range(c.Hkv):
            o = out[b, h * G:(h + 1) * G]
            if n == 0:
                assert bool((o == 0).all())
                w = np.zeros(c.max_tiles)
            else:
                want, p, bound = attend(qn[b, h * G:(h + 1) * G], c.k[b][h], c.v[b][h], scale, [n] * G, np.ones(n), 2.0 ** -39)
                check(o, want, bound, q.dtype)
                w = np.zeros(c.max_tiles * T)
                w[:n] = p.sum(0)
                w = w.reshape(-1, T).sum(1)
            if mass is not None:
                base = 0.0 if mass_in is None else mass_in[b, h].double().cpu().numpy()
                # a weight is within 2^-17 of itself and of the scores' bound (standard normal queries: below 2^-12)
                got = mass[b, h].double().cpu().numpy()
                assert (np.abs(got - base - w) <= 2.0 ** -12 * w + 2.0 ** -23 * (np.abs(base) + w) + 1e-30).all()


@pytest.fixture(params=[0, 40])
def tables(request, monkeypatch):
    """Short tables, which a block reads by itself, and long ones, whose tiles are shared out."""
    monkeypatch.setattr(Cache4, "beyond", request.param)


@pytest.mark.usefixtures("tables")
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_matches_the_formula(D, io):
    c = Cache4(D, [300, 129, 5], 2, D)
    q = _query(1, (3, 8, D), io)
    _check_decode(c, q, c.decode(q))


@pytest.mark.usefixtures("tables")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8])
def test_decode_head_groups(G, D):
    c = Cache4(10 * G, [140, 77], 2, D)
    q = _query(G, (2, 2 * G, D), "f32")
    _check_decode(c, q, c.decode(q))


@pytest.mark.usefixtures("tables")
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_lengths(D):
    """Around every end of a run and a tile; tokens behind the last hold every byte 0xFF, or 0x7C: NaN and infinite
    scales, in a table with tiles to spare."""
    for fill in (0xFF, 0x7C):
        c = Cache4(7, [0, 1, 2, 31, 32, 33, 64, 65, 96, 127, 128, 129, 160, 255, 257, 384], 1, D, max_tiles=5, fill=fill)
        for io in ("f32", "bf16"):
            q = _query(3, (16, 3, D), io)
            _check_decode(c, q, c.decode(q))


def test_decode_of_long_sequences():
    """Several items per head, many runs per warp, entries of the table read in several lots."""
    c = Cache4(8, [6001], 1, 64)
    q = _query(3, (1, 5, 64), "f32")
    _check_decode(c, q, c.decode(q))
    # a plan for a batch of long sequences, few of which are: items of many tiles
    B, tiles = 32, 400
    n = 128 * 37 + 5
    c = Cache4(9, [n], 1, 64)
    table = torch.full((B, 8, tiles), -1, dtype=torch.int64, device=DEV)
    table[3, 2, :38] = c.table[0, 0]
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    lens[3] = n
    q = _query(5, (B, 8, 64), "f32")
    table[3] = table[3, 2]
    out = kvarn.decode_attention4(q, c.tiles, table, lens, c.lay)
    for h in range(8):
        want, _, bound = attend(q[3, h:h + 1].double().cpu().numpy(), c.k[0][0], c.v[0][0], 64 ** -0.5, [n], np.ones(n), 2.0 ** -39)
        check(out[3, h:h + 1], want, bound, q.dtype)
    assert bool((out[:3] == 0).all()) and bool((out[4:] == 0).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_of_one_long_sequence_among_empty_ones(D):
    """A warp per row is planned for the pieces, of which the one sequence has more than a warp takes."""
    c, table, ln, rows_of = _shared(D, D, 3, [0] * 17 + [6000] + [0] * 22)
    q = _query(D, (40, 9, D), "f32")
    m = torch.zeros(table.shape, device=DEV)
    out = kvarn.decode_attention4(q, c.tiles, table, ln, c.lay, mass_out=m)
    for h in range(3):
        k, v = rows_of(17, h, 6000)
        want, p, bound = attend(q[17, 3 * h:3 * h + 3].double().cpu().numpy(), k, v, D ** -0.5, [6000] * 3, np.ones(6000),
                                2.0 ** -39)
        check(out[17, 3 * h:3 * h + 3], want, bound, q.dtype)
        w = np.append(p.sum(0), np.zeros(47 * T - 6000)).reshape(-1, T).sum(1)
        assert (np.abs(m[17, h].double().cpu().numpy() - w) <= 2.0 ** -12 * w).all()
    keep = torch.arange(40, device=DEV) != 17
    assert bool((out[keep] == 0).all()) and bool((m[keep] == 0).all())


def _shared(seed, D, H, lens, distinct=5):
    """Ragged sequences whose tables name the same few tiles in any order: (pool's cache, table, lens, K and V rows by
    (b, h))."""
    c = Cache4(seed, [T * distinct], 1, D)
    rng = np.random.default_rng(seed + 1)
    tiles = max(-(-max(lens) // T), 1)
    pick = rng.integers(0, distinct, (len(lens), H, tiles))
    table = c.table[0, 0][torch.from_numpy(pick).to(DEV)].contiguous()

    def rows_of(b, h, n):
        return (x[0].reshape(distinct, T, D)[pick[b, h]].reshape(-1, D)[:n] for x in (c.k[0], c.v[0]))
    return c, table, _dev(lens, torch.int32), rows_of


@pytest.mark.parametrize("longest", [6000, 1000])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 2), (64, 7), (128, 4), (128, 8), (256, 3), (256, 5)])
def test_decode_of_ragged_batches(D, G, io, longest):
    """More tiles than CTAs: shares that begin and end inside sequences, that span several, and sequences of no
    tokens between them (or a table short enough for a block per sequence and KV head); weights of all tiles."""
    H = 3
    rng = np.random.default_rng(D + G)
    lens = [int(n) for n in rng.integers(0, 900, 60)]
    lens[0] = lens[7] = lens[8] = lens[31] = lens[-1] = 0
    lens[5], lens[20] = longest, 128
    c, table, ln, rows_of = _shared(D, D, H, lens)
    q = _query(G, (len(lens), H * G, D), io)
    m = torch.zeros(table.shape, device=DEV)
    out = kvarn.decode_attention4(q, c.tiles, table, ln, c.lay, mass_out=m)
    qn, mn = q.double().cpu().numpy(), m.double().cpu().numpy()
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 0).all()) and not mn[b].any()
            continue
        for h in range(H):
            k, v = rows_of(b, h, n)
            want, p, bound = attend(qn[b, h * G:(h + 1) * G], k, v, D ** -0.5, [n] * G, np.ones(n), 2.0 ** -39)
            check(out[b, h * G:(h + 1) * G], want, bound, q.dtype)
            w = np.zeros(table.shape[2] * T)
            w[:n] = p.sum(0)
            w = w.reshape(-1, T).sum(1)
            assert (np.abs(mn[b, h] - w) <= 2.0 ** -12 * w + 1e-30).all()
    assert torch.equal(out, kvarn.decode_attention4(q, c.tiles, table, ln, c.lay, flags=kvarn.LAUNCH_PDL))
    # a batch of more sequences than threads: the same ones, apart by sequences of no tokens
    far = torch.zeros(60 * 7, dtype=torch.int32, device=DEV)
    far[::7] = ln
    q7 = q.repeat_interleave(7, 0)
    out7 = kvarn.decode_attention4(q7, c.tiles, table.repeat_interleave(7, 0), far, c.lay)
    # (shares are cut elsewhere: the same but for the order of sums)
    assert torch.allclose(out7[::7].float(), out.float(), rtol=2.0 ** -6 if io == "bf16" else 2.0 ** -14, atol=2.0 ** -9)
    assert bool((out7.view(60, 7, -1)[:, 1:] == 0).all())


@pytest.mark.parametrize("G", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,H,n", [(400, 3, 0), (400, 3, 1), (100, 3, 4), (1, 200, 5), (80, 2, 3), (300, 4, 2)])
def test_decode_of_many_short_tables(B, H, n, D, G):
    """Segments in one round of CTAs, two and more; with no tile at all, and lengths from none to full tables."""
    lens = [(37 * b + 633) % (T * n + 1) for b in range(B)]
    c, table, dlens, rows_of = _shared(D + G, D, H, lens)
    table = table[:, :, :n].contiguous()
    if n and table.shape[2] < n:
        table = torch.nn.functional.pad(table, (0, n - table.shape[2]))
    q = _query(B, (B, H * G, D), "bf16")
    mass = torch.empty(B, H, n, device=DEV)
    out = kvarn.decode_attention4(q, c.tiles, table, dlens, c.lay, mass_out=mass)
    assert torch.equal(out, kvarn.decode_attention4(q, c.tiles, table, dlens, c.lay))
    assert bool((mass.sum(-1) - G * (dlens > 0).float()[:, None]).abs().max() < 1e-4 * G)
    assert bool((out[dlens == 0] == 0).all())
    for b in (0, 1, 2, B // 3, B // 2, B - 1):
        if b >= B or lens[b] == 0:
            continue
        for h in (0, H - 1):
            k, v = rows_of(b, h, lens[b])
            want, p, bound = attend(q[b, h * G:(h + 1) * G].double().cpu().numpy(), k, v, D ** -0.5, [lens[b]] * G,
                                    np.ones(lens[b]), 2.0 ** -39)
            check(out[b, h * G:(h + 1) * G], want, bound, q.dtype)


@pytest.mark.parametrize("n", [600, 2200])  # a block for each row group and head, and tiles shared out
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_of_few_rows_over_many_segments(D, n):
    """A chunk on the decode kernels with more tiles than CTAs: shares that span row groups and heads."""
    H, G, C = 8, 4, 31
    c, table, _, rows_of = _shared(D + 5, D, H, [n])
    for io in ("f32", "bf16"):
        q = _query(D, (C, H * G, D), io)
        out = kvarn.prefill_attention4(q, n - C, c.tiles, table[0], c.lay)
        for h in range(H):
            k, v = rows_of(0, h, n)
            qn = q[:, h * G:(h + 1) * G].double().cpu().numpy().reshape(C * G, D)
            want, p, bound = attend(qn, k, v, D ** -0.5, np.repeat(n - C + 1 + np.arange(C), G), np.ones(n), 2.0 ** -33)
            check(out[:, h * G:(h + 1) * G].reshape(C * G, D), want, bound, q.dtype, 0.0 if io == "f32" else 2.0 ** -11,
                  p @ np.abs(v))


@pytest.mark.usefixtures("tables")
@pytest.mark.parametrize("D,G", [(64, 3), (64, 8), (128, 4), (128, 8), (256, 4)])
def test_decode_weights_accumulate(D, G):
    c = Cache4(20 + D, [450, 0, 128, 33], 2, D, max_tiles=6)
    q = _query(5, (4, 2 * G, D), "f32")
    m = torch.full((4, 2, c.max_tiles), float("nan"), device=DEV)
    _check_decode(c, q, c.decode(q, mass_out=m), mass=m)
    base = torch.rand(4, 2, c.max_tiles, device=DEV) * 3
    m2 = base.clone()
    out = c.decode(q, mass_in=m2, mass_out=m2)
    _check_decode(c, q, out, mass=m2, mass_in=base)
    m3 = torch.empty_like(base)
    c.decode(q, mass_in=base, mass_out=m3)
    assert torch.equal(m2, m3) and torch.equal(out, c.decode(q))
    assert torch.equal(m2[1], base[1])


@pytest.mark.parametrize("n", [300, 3000])
def test_decode_without_weights_needs_no_room_for_them(n):
    c = Cache4(27, [n, 7], 2, 64)
    q = _query(28, (2, 8, 64), "bf16")
    need = kvarn.decode4_workspace_bytes(2, 8, 2, 64, c.max_tiles, weights=False)
    room = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    out = c.decode(q, ws=room[:need])
    assert torch.equal(out, c.decode(q)) and torch.equal(out, c.decode(q, mass_out=torch.zeros(2, 2, c.max_tiles, device=DEV)))
    assert bool((room[need:] == 0xA5).all())
    _check_decode(c, q, out)
    with pytest.raises(kvarn.KvarnError):
        c.decode(q, ws=room[:need], mass_out=torch.zeros(2, 2, c.max_tiles, device=DEV))


@pytest.mark.parametrize("tokens", [256, 2560])
def test_decode_counts_past_their_table_are_clamped(tokens):
    c = Cache4(30, [tokens, 40], 2, 128)
    q = _query(5, (2, 4, 128), "f32")
    want = c.decode(q)
    c.lens = _dev([2 ** 31 - 1, 40], torch.int32)
    assert torch.equal(c.decode(q), want)
    c.lens = _dev([-(2 ** 31), 40], torch.int32)
    out = c.decode(q)
    assert bool((out[0] == 0).all()) and torch.equal(out[1], want[1])


@pytest.mark.usefixtures("tables")
def test_decode_scales_of_either_sign_and_zero():
    c = Cache4(31, [200], 1, 64)
    q = _query(5, (1, 4, 64), "f32")
    for scale in (-0.2, 0.0, 1e-30, 2.0):
        _check_decode(c, q, c.decode(q, softmax_scale=scale), scale)


@pytest.mark.usefixtures("tables")
def test_decode_with_far_apart_values():
    """Value rows from the smallest scale to the largest magnitude, under keys that favour the small ones."""
    def change(b, h, k, v):
        v[::3] *= np.float32(1e-6)
        v[1::3] = np.sign(v[1::3]) * np.float32(MAX4)
        k[:] *= np.float32(0.3)
    for D in (64, 256):
        c = Cache4(32, [190], 2, D, change=change)
        q = _query(6, (1, 4, D), "f32")
        _check_decode(c, q, c.decode(q))


@pytest.mark.usefixtures("tables")
def test_decode_poison_and_bad_queries():
    def change(b, h, k, v):
        if (b, h) == (1, 0):
            v[150, 7] = np.inf
    c = Cache4(33, [160, 160], 2, 128, change=change)
    d = Cache4(33, [160, 160], 2, 128)
    q = _query(7, (2, 8, 128), "f32")
    want, out = d.decode(q), c.decode(q)
    assert bool(out[1, :4].isnan().all()) and torch.equal(out[0], want[0]) and torch.equal(out[1, 4:], want[1, 4:])
    for io in ("f32", "f16", "bf16"):
        q = _query(7, (2, 8, 128), io)
        want = d.decode(q)
        q[0, 1, 5], q[0, 6, 99], q[1, 3, 0] = float("inf"), float("nan"), float("-inf")
        out = d.decode(q)
        bad = torch.zeros(2, 8, dtype=torch.bool, device=DEV)
        bad[0, 1] = bad[0, 6] = bad[1, 3] = True
        assert bool(out[bad].isnan().all()) and torch.equal(out[~bad], want[~bad])


@pytest.mark.usefixtures("tables")
@pytest.mark.parametrize("D,G", [(64, 8), (128, 2), (256, 2)])
def test_decode_bad_offsets_poison_their_head_only(D, G):
    many = 1 if Cache4.beyond else 40  # (sequences enough that a block reads eight tiles by itself)
    c = Cache4(34, [900, 300] + [1] * many, 2, D)
    q = _query(8, (2 + many, 2 * G, D), "bf16")
    m = torch.zeros(2 + many, 2, c.max_tiles, device=DEV)
    want = c.decode(q, mass_out=m)
    for off in (-16, 8, c.tiles.numel() - c.lay.record_bytes + 16, 1 << 62):
        t = c.table.clone()
        t[0, 1, 5] = off
        t[1, 0, 3] = off  # behind the sequence's last tile: not read
        m2 = torch.zeros_like(m)
        out = kvarn.decode_attention4(q, c.tiles, t, c.lens, c.lay, mass_out=m2)
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
        assert bool(out[0, G:].isnan().all()) and torch.equal(out[0, :G], want[0, :G]) and torch.equal(out[1:], want[1:])
        assert bool(m2[0, 1, :8].isnan().all()) and torch.equal(m2[0, 0], m[0, 0]) and torch.equal(m2[1:], m[1:])


@pytest.mark.usefixtures("tables")
def test_decode_launch_modes_and_graphs_are_bit_identical():
    """Two graphs of different sizes that share a workspace, replayed in turn after a step has moved the cache on."""
    c = Cache4(35, [400, 90, 1], 2, 128, max_tiles=4)
    q = _query(9, (3, 8, 128), "bf16")
    want = c.decode(q)
    assert torch.equal(c.decode(q, flags=kvarn.LAUNCH_PDL), want)
    ws = torch.empty(kvarn.decode4_workspace_bytes(3, 8, 2, 128, c.max_tiles), dtype=torch.uint8, device=DEV)
    out, few = torch.empty_like(q), torch.empty_like(q[:1])
    row = _query(10, (3, 1, 2, 128), "bf16")
    torch.cuda.synchronize()
    graphs = []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for k in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                if k == 0:
                    kvarn.write_rows4(row, row, c.tiles, c.table, c.lens, c.lay, flags=kvarn.LAUNCH_PDL)
                    c.lens.add_(1)
                    c.decode(q, ws=ws, out=out, flags=kvarn.LAUNCH_PDL)
                else:
                    kvarn.decode_attention4(q[:1], c.tiles, c.table[:1], c.lens[:1], c.lay, ws=ws, out=few,
                                            flags=kvarn.LAUNCH_PDL)
            graphs.append(g)
    assert c.lens.tolist() == [400, 90, 1]
    for step in range(3):
        graphs[0].replay()
        a = out.clone()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert c.lens.tolist() == [401 + step, 91 + step, 2 + step]
        assert torch.equal(a, c.decode(q)) and torch.equal(few[0], a[0])


def test_calls_run_on_the_stream_that_they_are_given():
    c = Cache4(36, [300], 2, 64)
    q = _query(11, (1, 4, 64), "f32")
    want, want_pre = c.decode(q), c.prefill(q, 299)
    side, late = torch.cuda.Stream(), torch.zeros_like(q)
    row = _query(12, (1, 5, 2, 64), "f32")
    back = torch.zeros(2, 1, 5, 2, 64, device=DEV)
    for first in (True, False):  # (the first time kernels are loaded, which waits for the device)
        torch.cuda.synchronize()
        if not first:
            with torch.cuda.stream(side):
                torch.cuda._sleep(100_000_000)
                late.copy_(q)
        out = c.decode(late, stream=side)
        pre = c.prefill(late, 299, stream=side)
        kvarn.write_rows4(row, row, c.tiles, c.table, c.lens, c.lay, stream=side)
        kvarn.read_rows4(c.tiles, c.table, c.lens, back[0], back[1], c.lay, stream=side)
        turned, _ = kvarn.norm_rotate(late, None, None, None, hadamard=True, stream=side)
        assert bool((late == 0).all())
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(pre, want_pre)
    assert torch.equal(back[0], back[1]) and bool((back != 0).any())
    assert torch.equal(turned, kvarn.norm_rotate(q, None, None, None, hadamard=True)[0])


def test_decode_on_two_streams_at_once():
    c, d = Cache4(37, [3000], 2, 64), Cache4(38, [2000], 2, 64)
    q = _query(13, (1, 8, 64), "f32")
    want = c.decode(q), d.decode(q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [x.decode(q, stream=s) for x, s in zip((c, d), streams)]
        for s in streams:
            s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_host_tensors_and_wrong_shapes_are_refused():
    c = Cache4(39, [130], 2, 64)
    q, row = _query(14, (1, 4, 64), "f32"), _query(15, (1, 1, 2, 64), "f32")
    ok = [row, row, c.tiles, c.table, c.lens]
    for i in range(5):
        a = list(ok)
        a[i] = a[i].cpu()
        with pytest.raises((TypeError, ValueError)):
            kvarn.write_rows4(*a, c.lay)
    for a in ([row[:, :, :1], row[:, :, :1], *ok[2:]], [row, row.half(), *ok[2:]], [*ok[:4], c.lens.long()],
              [*ok[:3], c.table[0], c.lens]):
        with pytest.raises((TypeError, ValueError)):
            kvarn.write_rows4(*a, c.lay)
    for lay in (kvarn.layout4(128),):
        with pytest.raises(ValueError, match="head_dim"):
            kvarn.write_rows4(*ok, lay)
        with pytest.raises(ValueError, match="head_dim"):
            kvarn.decode_attention4(q, c.tiles, c.table, c.lens, lay)
    with pytest.raises(ValueError, match="counts"):
        kvarn.write_rows4(*ok, c.lay, counts=_dev([1, 2], torch.int32))
    for i in range(4):
        a = [q, c.tiles, c.table, c.lens]
        a[i] = a[i].cpu()
        with pytest.raises((TypeError, ValueError)):
            kvarn.decode_attention4(*a, c.lay)
    with pytest.raises(kvarn.KvarnError):
        c.decode(q, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(kvarn.KvarnError):
        c.prefill(q, 256)  # past the table
    with pytest.raises(ValueError):
        c.decode(q, out=torch.empty(2, 4, 64, device=DEV))


# ---------------------------------------------------------------- prefill

def _check_prefill(c, q, pos0, out, scale=None, b=0):
    C, Hq, D = q.shape
    G = Hq // c.Hkv
    extra = 0.0 if q.dtype == torch.float32 else 2.0 ** -11
    for h in range(c.Hkv):
        n = pos0 + C
        qn = q[:, h * G:(h + 1) * G].double().cpu().numpy().reshape(C * G, D)
        want, p, bound = attend(qn, c.k[b][h][:n], c.v[b][h][:n], D ** -0.5 if scale is None else scale,
                                np.repeat(pos0 + 1 + np.arange(C), G), np.ones(n), 2.0 ** -33)
        check(out[:, h * G:(h + 1) * G].reshape(C * G, D), want, bound, q.dtype, extra, p @ np.abs(c.v[b][h][:n]))


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_matches_the_formula(D, io):
    c = Cache4(40 + D, [530], 2, D)
    for C, pos0 in ((230, 300), (3, 527), (129, 0)):
        q = _query(C, (C, 8, D), io)
        _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8])
def test_prefill_head_groups(G):
    for D in (64, 128):
        c = Cache4(50 + G, [300], 2, D)
        for C, pos0 in ((140, 160), (2, 200)):
            q = _query(G, (C, 2 * G, D), "f32")
            _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("C", [1, 2, 31, 100])
def test_prefill_lengths_and_positions(C, D):
    """Chunks at the start, over and next to ends of tiles and runs, before and behind the cache's last token."""
    for fill in (0xFF, 0x7C):
        c = Cache4(60, [300], 1, D, max_tiles=4, fill=fill)
        for pos0 in (0, 31, 32, 127, 128, 129, 200):
            for io in ("f32", "bf16"):
                q = _query(C + pos0, (C, 4, D), io)
                _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hkv,C,n", [(8, 320, 2800), (2, 200, 4300), (1, 130, 1100)])
def test_prefill_of_many_blocks(Hkv, C, n, io):
    for D in (64, 128, 256):
        if n * Hkv * D > 3_000_000:
            continue
        c = Cache4(61, [n], Hkv, D)
        q = _query(C, (C, 2 * Hkv, D), io)
        _check_prefill(c, q, n - C, c.prefill(q, n - C))


@pytest.mark.parametrize("D,io", [(64, "f32"), (128, "bf16"), (256, "f32")])
def test_prefill_of_more_blocks_than_one_round(D, io):
    """More blocks of rows than SMs over a long context: keys in shares that take several rounds. Rows of the first and
    the last blocks."""
    H, G, C, n = 8, 8, 330, 11000
    c, table, _, rows_of = _shared(D + 9, D, H, [n])
    q = _query(D, (C, H * G, D), io)
    out = kvarn.prefill_attention4(q, n - C, c.tiles, table[0], c.lay)
    at = [0, 1, 15, 16, 200, 319, 320, 329]
    for h in (0, 3, 7):
        k, v = rows_of(0, h, n)
        qn = q[at, h * G:(h + 1) * G].double().cpu().numpy().reshape(-1, D)
        want, p, bound = attend(qn, k, v, D ** -0.5, np.repeat(n - C + 1 + np.array(at), G), np.ones(n), 2.0 ** -33)
        check(out[at, h * G:(h + 1) * G].reshape(-1, D), want, bound, q.dtype, 0.0 if io == "f32" else 2.0 ** -11,
              p @ np.abs(v))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_of_long_fp32_contexts(D):
    """O is emptied into rounded sums every so many blocks: several times, under growing scores."""
    def change(b, h, k, v):
        k *= np.linspace(0.1, 2, k.shape[0], dtype=np.float32)[:, None]
    n, C = 36 * 64 * 3 + 100, 70
    c = Cache4(62, [n], 1, D, change=change)
    q = _query(C, (C, 8, D), "f32")
    q = q.repeat(1, 1, 1)
    _check_prefill(c, q, n - C, c.prefill(q, n - C))


def test_prefill_scales_of_either_sign_and_zero():
    c = Cache4(63, [400], 1, 64)
    for C in (3, 200):
        q = _query(5, (C, 4, 64), "f32")
        for scale in (-0.2, 0.0, 1e-30, 2.0):
            _check_prefill(c, q, 400 - C, c.prefill(q, 400 - C, softmax_scale=scale), scale)


@pytest.mark.parametrize("C", [9, 100])  # on the decode kernels, and on the images
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_poison_reaches_only_the_rows_that_see_it(D, C):
    def change(b, h, k, v):
        if h == 1:
            v[260, 5] = np.nan
            k[261, 9] = np.inf
    c, d = Cache4(64, [290], 2, D, change=change), Cache4(64, [290], 2, D)
    pos0 = 264 - C
    for io in ("f32", "bf16"):
        q = _query(8, (C, 4, D), io)
        want, out = d.prefill(q, pos0), c.prefill(q, pos0)
        first = 260 - pos0
        assert torch.equal(out[:first], want[:first]) and torch.equal(out[:, :2], want[:, :2])
        assert bool(out[first:, 2:].isnan().all())


@pytest.mark.parametrize("C", [9, 100])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_prefill_bad_queries_are_nan(io, C):
    c = Cache4(65, [276], 2, 128)
    for pos0 in (0, 276 - C):
        q = _query(8, (C, 4, 128), io)
        want = c.prefill(q, pos0)
        q[1, 2, 5], q[2, 2, 5], q[3, 3, 7], q[5, 0, 0] = -np.inf, np.inf, np.nan, -np.inf
        out = c.prefill(q, pos0)
        bad = torch.zeros(C, 4, dtype=torch.bool, device=DEV)
        bad[1, 2] = bad[2, 2] = bad[3, 3] = bad[5, 0] = True
        assert bool(out[bad].isnan().all()) and torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("C", [8, 200])
def test_prefill_bad_offsets_poison_what_sees_them(C):
    c = Cache4(66, [620], 2, 128)
    q = _query(3, (C, 8, 128), "bf16")
    pos0 = 3 * T - 4 if C == 8 else 4 * T - C
    want = c.prefill(q, pos0)
    for off in (-16, 8, c.tiles.numel() - c.lay.record_bytes + 16, 1 << 62):
        t = c.table[0].clone()
        t[1, 3] = off
        t[:, 4] = off  # behind the chunk's last position: not read
        out = kvarn.prefill_attention4(q, pos0, c.tiles, t, c.lay)
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
        first = 3 * T - pos0
        assert torch.equal(out[:, :4], want[:, :4]) and bool(out[first:, 4:].isnan().all())
        assert torch.equal(out[:first, 4:], want[:first, 4:])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C,G", [(5, 8), (6, 8), (11, 4), (64, 1), (13, 5), (16, 4), (40, 2)])
def test_prefill_around_the_change_of_kernels(C, G, io):
    for Hkv, n in ((1, 700), (2, 1500)):
        c = Cache4(67, [n], Hkv, 64)
        q = _query(C, (C, G * Hkv, 64), io)
        _check_prefill(c, q, n - C, c.prefill(q, n - C))


def test_prefill_of_one_position_agrees_with_decode_and_replays():
    c = Cache4(68, [777], 2, 128)
    for Hq in (8, 12):  # (the same products, but for the order of the parts up to four heads to a group)
        q = _query(9, (1, Hq, 128), "f32")
        pre, dec = c.prefill(q, 776), c.decode(q)
        _check_prefill(c, q, 776, pre)
        assert torch.equal(pre, dec) if Hq == 12 else torch.allclose(pre, dec, rtol=0, atol=2.0 ** -15 * float(dec.abs().max()))
    for C in (4, 300):  # a workspace for more serves both
        q = _query(10, (C, 8, 128), "bf16")
        want = c.prefill(q, 777 - C)
        ws = torch.empty(kvarn.prefill4_workspace_bytes(300, 7, 8, 2, 128), dtype=torch.uint8, device=DEV)
        out, g = torch.empty_like(q), torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            c.prefill(q, 777 - C, ws=ws, out=out)
        for _ in range(3):
            ws.fill_(255)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,H,C,n", [(64, 2, 48, 16000), (128, 1, 96, 20001), (256, 4, 40, 24700)])
def test_prefill_of_few_rows_over_long_tables(D, H, C, n, io):
    """On the images from some length on, in as many key shares as there can be."""
    G = 4
    c, table, _, rows_of = _shared(D + 11, D, H, [n])
    q = _query(D, (C, H * G, D), io)
    out = kvarn.prefill_attention4(q, n - C, c.tiles, table[0], c.lay)
    at = [0, 1, C // 2, C - 1]
    for h in range(H):
        k, v = rows_of(0, h, n)
        qn = q[at, h * G:(h + 1) * G].double().cpu().numpy().reshape(-1, D)
        want, p, bound = attend(qn, k, v, D ** -0.5, np.repeat(n - C + 1 + np.array(at), G), np.ones(n), 2.0 ** -33)
        check(out[at, h * G:(h + 1) * G].reshape(-1, D), want, bound, q.dtype, 0.0 if io == "f32" else 2.0 ** -11, p @ np.abs(v))


@pytest.mark.parametrize("C", [9, 70, 200])  # on the decode kernels, on the images in key shares, and without
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_of_equal_values_gives_them(D, C):
    """Weights add up to one as the products see them: with the same V row at every token each output is that row. All
    else is below (n / 16 + 2) 2^-23 + 2^-20 of it (the products' sums, which are cut off, and the sum of weights), 7e-6 here, and
    half a step of an fp16 number is 2^-12 of it at least: the very row comes out."""
    n, H, G = 700, 2, 4
    s = _Store(1, H, D, 6)
    k = torch.randn(1, n, H, D, generator=torch.Generator().manual_seed(D)).to(DEV)
    v = _query(D + 1, (1, 1, H, D), "f32").expand(1, n, H, D).contiguous()
    s.write(k, v, [0])
    k, v = torch.zeros_like(k), torch.zeros_like(v)
    s.read(k, v, [0])
    for scale in (D ** -0.5, 0.3, 1.0):  # many weights to a row, or a few large ones
        q = _query(C, (C, H * G, D), "f16")
        out = kvarn.prefill_attention4(q, n - C, s.tiles, s.table[0], s.lay, softmax_scale=scale)
        assert torch.equal(out.float(), v[0, 0].repeat_interleave(G, 0).expand(C, H * G, D))


# ---------------------------------------------------------------- sizes

@pytest.mark.parametrize("D", [64, 256])
def test_records_past_32_bit_offsets(D):
    """A pool of more than 2^32 bytes: rows written, read and attended to at its end."""
    lay = kvarn.layout4(D)
    n = (1 << 32) // lay.record_bytes + 3
    tiles = torch.zeros(n * lay.record_bytes, dtype=torch.uint8, device=DEV)
    small = torch.zeros(2 * lay.record_bytes, dtype=torch.uint8, device=DEV)
    last = _dev([[[n - 2, n - 1]]]) * lay.record_bytes
    low = _dev([[[0, 1]]]) * lay.record_bytes
    k, v = (torch.from_numpy(x.reshape(1, 200, 1, D)).to(DEV) for x in rows(np.random.default_rng(1), 200, D))
    lens, q = _dev([0], torch.int32), _query(2, (150, 4, D), "bf16")
    res = []
    for pool, table in ((tiles, last), (small, low)):
        kvarn.write_rows4(k, v, pool, table, lens, lay)
        back = torch.zeros(2, 1, 200, 1, D, device=DEV)
        kvarn.read_rows4(pool, table, lens, back[0], back[1], lay)
        res.append([back, kvarn.decode_attention4(q[:1], pool, table, lens + 200, lay),
                    kvarn.prefill_attention4(q, 50, pool, table[0], lay), kvarn.prefill_attention4(q[:2], 50, pool, table[0], lay)])
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert torch.equal(tiles[last[0, 0, 0]:], small)


# ---------------------------------------------------------------- a run of them together

@pytest.mark.parametrize("D,io", [(128, "f32"), (64, "bf16"), (256, "f16")])
def test_a_cache_lives_prompt_drafts_decode_evict(D, io):
    """Packed products of a layer, two sequences: a prompt in chunks, drafted tokens, decode steps with weights, tiles
    evicted by them, and more decode steps: at each step the outputs are those of softmax attention over the rows
    as read back, the queries as norm_rotate gives them."""
    H, G, n_tiles = 2, 3, 4
    dt = IO[io]
    lay = kvarn.layout4(D)
    place = torch.randperm(2 * H * n_tiles, generator=torch.Generator().manual_seed(1))
    table = (place * lay.record_bytes).view(2, H, n_tiles).to(DEV)
    tiles = torch.full((2 * H * n_tiles * lay.record_bytes,), 0xFF, dtype=torch.uint8, device=DEV)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    spare = torch.zeros(2, dtype=torch.int32, device=DEV)
    plan = kvarn.rotary(D // 2, theta=500000.0)
    weight = (1 + 0.1 * _query(1, (D,), "f32")).to(dt)
    mass = torch.zeros(2, H, n_tiles, device=DEV)
    seed = [100]

    def product(n):
        seed[0] += 1
        return _query(seed[0], (2, n, (G + 2) * H, D), io)

    def ready(x, pos):
        """One product's rows made ready in place, and written."""
        n = x.shape[1]
        rows_ = x.view(2 * n, -1, D)
        kvarn.norm_rotate(rows_[:, :G * H], rows_[:, G * H:(G + 1) * H], pos.reshape(-1), plan, q_weight=weight, k_weight=weight,
                          eps=1e-5, hadamard=True, q_out=rows_[:, :G * H], k_out=rows_[:, G * H:(G + 1) * H])
        kvarn.write_rows4(x[:, :, G * H:(G + 1) * H], x[:, :, (G + 1) * H:], tiles, table, lens, lay)
        kvarn.window_advance(spare, lens, None, n, 0, T * n_tiles)
        return x[:, :, :G * H].contiguous()

    def held(b):
        n = int(lens[b])
        k, v = (torch.zeros(1, n, H, D, device=DEV) for _ in "kv")
        kvarn.read_rows4(tiles, table[b:b + 1], torch.zeros(1, dtype=torch.int32, device=DEV), k, v, lay)
        return (x[0].transpose(0, 1).double().cpu().numpy() for x in (k, v))

    def verify(q, out, b, extra, floor):
        n = q.shape[0]
        k, v = held(b)
        for h in range(H):
            qn = q[:, h * G:(h + 1) * G].double().cpu().numpy().reshape(n * G, D)
            total = k.shape[1]
            want, p, bound = attend(qn, k[h], v[h], D ** -0.5, np.repeat(total - n + 1 + np.arange(n), G), np.ones(total), floor)
            check(out[:, h * G:(h + 1) * G].reshape(n * G, D), want, bound, dt, extra, p @ np.abs(v[h]))

    at = 0
    for n in (150, 101, 4, 2):  # a prompt of two chunks, drafts
        q = ready(product(n), (at + torch.arange(n, device=DEV)).repeat(2, 1))
        for b in range(2):
            out = kvarn.prefill_attention4(q[b], at, tiles, table[b], lay)
            verify(q[b], out, b, 0.0 if io == "f32" else 2.0 ** -11, 2.0 ** -33)
        at += n
    for step in range(150):
        q = ready(product(1), torch.full((2, 1), at, device=DEV))
        out = kvarn.decode_attention4(q[:, 0], tiles, table, lens, lay, mass_in=mass, mass_out=mass)
        at += 1
        if step % 49 == 0:
            for b in range(2):
                verify(q[b], out[b:b + 1], b, 0.0, 2.0 ** -39)
    total = (H * G) * 150 / H
    assert bool(((mass.sum(-1) - total).abs() < 1e-3 * total).all())
    n = (lens + T - 1) // T
    gone = torch.empty_like(table)
    kvarn.evict_tiles(table, mass, n, keep=3, sinks=1, recent=1, evicted=gone)
    assert n.tolist() == [3, 3] and bool((gone[..., 0] >= 0).all())
    lens -= T
    table[:, :, 3] = gone[:, :, 0]  # the record that left is the next one to be filled
    for step in range(3):
        q = ready(product(1), torch.full((2, 1), at, device=DEV))
        out = kvarn.decode_attention4(q[:, 0], tiles, table, lens, lay)
        at += 1
        for b in range(2):
            verify(q[b], out[b:b + 1], b, 0.0, 2.0 ** -39)
