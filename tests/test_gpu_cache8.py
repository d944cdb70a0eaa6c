"""The 8-bit cache on the GPU against plain 64-bit statements of its operators."""
import numpy as np
import pytest
import torch

from kv_cache_quantization_token_gb300 import kvarn
from tests.cache8_helpers import DEV, T, Cache8, attend, check, pack, quantise, rows

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


# ---------------------------------------------------------------- compress and expand

def _compress(k, v, src, dst, n_rec, lay):
    tiles = torch.full((n_rec * lay.record_bytes,), 0xA5, dtype=torch.uint8, device=DEV)
    kvarn.compress_tile8(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV),
                         torch.tensor(src, device=DEV), tiles,
                         torch.tensor(dst, device=DEV) * lay.record_bytes, lay)
    return tiles


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_records_are_bit_exact(code, D, block):
    rng = np.random.default_rng(D + block)
    n, stride = 3, D + 12
    k, v = np.zeros((n * T + 9, stride), np.float32), np.zeros((n * T + 9, stride), np.float32)
    k[:, :D], v[:, :D] = rows(rng, n * T + 9, D)
    v[5 + T:5 + T + block, :D] = 0                      # a block of zeros
    k[5:5 + block] *= np.float32(1e-33)                 # under the scale floor
    k[5 + T:5 + T + block] *= np.float32(1e30)
    v[5 + 2 * T:5 + 2 * T + 16, :D] = -0.0
    src, dst = [5, 5 + T, 5 + 2 * T], [2, 0, 3]
    lay = kvarn.layout8(D, code, block)
    tiles = _compress(k, v, src, dst, 4, lay).cpu().numpy().reshape(4, -1)
    for s, d in zip(src, dst):
        kb, _, ks = quantise(k[s:s + T, :D], code, block)
        vb, _, vs = quantise(v[s:s + T, :D], code, block)
        assert np.array_equal(tiles[d], pack(kb, ks, vb, vs))
    assert (tiles[1] == 0xA5).all()  # the record of no unit


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_quotients_next_to_the_middle_of_two_codes(code):
    """Values on, and one fp32 step to either side of, every middle of two codes: the
    quotient's side is decided exactly, ties go to the even code."""
    D, block = 128, 128
    lay = kvarn.layout8(D, code, block)
    if code == "i8":
        mids = np.arange(0.5, 127)
    else:
        from tests.cache8_helpers import e4m3_values
        x = e4m3_values()
        mids = (x[1:] + x[:-1]) / 2
    rng = np.random.default_rng(3)
    k = np.zeros((4 * T, D), np.float32)
    for u in range(4):
        top = np.float32([1.0, 448.0, 0.3, 7.77e5][u])
        s = np.float64(np.float32(top / np.float32({"i8": 127, "e4m3": 448}[code])))
        m = (rng.choice(mids, (T, D)) * s).astype(np.float32)
        step = rng.integers(-2, 3, (T, D))
        m = np.where(step < 0, np.nextafter(m, np.float32(0)), np.where(step > 0, np.nextafter(m, top * 2), m))
        k[u * T:u * T + T] = np.minimum(m, top) * rng.choice([-1, 1], (T, D))
        k[u * T, 0] = top
    tiles = _compress(k, k, [0, T, 2 * T, 3 * T], [0, 1, 2, 3], 4, lay).cpu().numpy().reshape(4, -1)
    for u in range(4):
        b, _, s = quantise(k[u * T:u * T + T], code, block)
        assert np.array_equal(tiles[u], pack(b, s, b, s))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_expand_writes_code_times_scale_and_nothing_else(code, D):
    rng = np.random.default_rng(D)
    k, v = rows(rng, 2 * T, D)
    lay = kvarn.layout8(D, code, 32)
    tiles = _compress(k, v, [0, T], [1, 0], 2, lay)
    stride = D + 4
    ko, vo = (torch.full((3 * T, stride), 7.0, device=DEV) for _ in range(2))
    kvarn.expand_tile8(tiles, torch.tensor([lay.record_bytes, 0], device=DEV), ko, vo,
                       torch.tensor([T + 3, 1], device=DEV), lay)
    for raw, out in ((k, ko.cpu().numpy()), (v, vo.cpu().numpy())):
        want = np.full((3 * T, stride), 7.0, np.float32)
        for u, row in enumerate((T + 3, 1)):
            _, val, s = quantise(raw[u * T:u * T + T], code, 32)
            want[row:row + T, :D] = (val * s.astype(np.float64).repeat(16)[:, None]).astype(np.float32)
        assert np.array_equal(out, want)


@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_block_with_a_non_finite_value_has_scale_nan_and_zero_codes(code, bad):
    k, v = rows(np.random.default_rng(1), T, 64)
    k[40, 3], v[127, 63] = bad, bad
    lay = kvarn.layout8(64, code, 32)
    rec = _compress(k, v, [0], [0], 1, lay).cpu().numpy()
    scales = rec[lay.off_k_scale:lay.off_k_scale + 64].view(np.float32)
    assert np.isnan(scales).tolist() == [False] * 2 + [True] * 2 + [False] * 4 + [False] * 6 + [True] * 2
    kb, _, ks = quantise(k, code, 32)
    vb, _, vs = quantise(v, code, 32)
    if code == "i8":
        assert np.array_equal(rec[:2 * T * 64], pack(kb, ks, vb, vs)[:2 * T * 64])


def test_units_outside_their_arrays_are_skipped():
    lay = kvarn.layout8(128)
    k, v = rows(np.random.default_rng(2), 2 * T, 128)
    rb = lay.record_bytes
    tiles = torch.zeros(2 * rb, dtype=torch.uint8, device=DEV)
    kd, vd = torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV)
    big = 1 << 62
    for src, dst in ((-1, 0), (T + 1, 0), (0, -rb), (0, rb + 16), (0, 8), (big, 0), (-big, 0), (0, big)):
        kvarn.compress_tile8(kd, vd, torch.tensor([src], device=DEV), tiles, torch.tensor([dst], device=DEV), lay)
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
    assert int(tiles.count_nonzero()) == 0
    out_k, out_v = torch.zeros(2 * T, 128, device=DEV), torch.zeros(2 * T, 128, device=DEV)
    for rec, row in ((0, -1), (0, T + 1), (0, big)):
        kvarn.expand_tile8(tiles, torch.tensor([rec], device=DEV), out_k, out_v, torch.tensor([row], device=DEV), lay)
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
    assert int(out_k.count_nonzero()) == 0 and int(out_v.count_nonzero()) == 0
    for rec in (-16, 8, rb + 16, big):
        kvarn.expand_tile8(tiles, torch.tensor([rec], device=DEV), out_k, out_v, torch.tensor([0], device=DEV), lay)
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
        assert bool(out_k[:T].isnan().all()) and bool(out_v[:T].isnan().all())
        assert int(out_k[T:].count_nonzero()) == 0


# ---------------------------------------------------------------- decode

def _check_decode(c, q, out, scale=None, mass=None, mass_in=None):
    scale = c.D ** -0.5 if scale is None else scale
    G = q.shape[1] // c.Hkv
    qn = q.double().cpu().numpy()
    for b in range(c.B):
        n = c.k[b].shape[1]
        for h in range(c.Hkv):
            sl = slice(h * G, h * G + G)
            if n == 0:
                assert int(out[b, sl].count_nonzero()) == 0
                continue
            want, p, bound = attend(qn[b, sl], c.k[b][h], c.v[b][h], scale, [n] * G, c.vs[b][h], 2.0 ** -39)
            check(out[b, sl], want, bound, q.dtype)
            if mass is not None:
                nt = c.tiles_of[b]
                w = p[:, :T * nt].sum(0).reshape(nt, T).sum(1)
                got = mass[b, h].double().cpu().numpy()
                base = mass_in[b, h].double().cpu().numpy()
                size = (np.abs(qn[b, sl]) @ np.abs(c.k[b][h]).T).max() * abs(scale)
                # the weights' own error, and one fp32 addition each to the sums and to mass_in
                tol = (2.0 ** -17 * size + 2.0 ** -19 + n / 16 * 2.0 ** -23) * w + 2.0 ** -23 * (base[:nt] + w) + 1e-30
                assert (np.abs(got[:nt] - base[:nt] - w) <= tol).all()
                assert np.array_equal(got[nt:], base[nt:])


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_matches_the_formula(D, code, io):
    c = Cache8(D, [5, 1, 0], [17, 128, 1], 2, D, code, 32)
    q = _query(D, (3, 8, D), io)
    _check_decode(c, q, c.decode(q))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8])
def test_decode_head_groups(G):
    c = Cache8(G, [3, 2], [0, 65], 3, 128, "i8", 16)
    q = _query(G, (2, 3 * G, 128), "f32")
    _check_decode(c, q, c.decode(q))


@pytest.mark.parametrize("tiles,windows,cap,starts", [
    ([0, 0], [0, 5], 128, [0, 126]),           # a sequence without any token, a window across the ring's end
    ([0], [1], 1, [0]), ([1], [0], 128, [3]), ([40], [300], 384, [380]), ([2, 9], [200, 1], 200, [199, 100]),
    ([700], [3], 128, [0])])
def test_decode_lengths_and_rings(tiles, windows, cap, starts):
    c = Cache8(11, tiles, windows, 1, 64, "e4m3", 128, cap=cap, starts=starts)
    q = _query(5, (len(tiles), 4, 64), "f32")
    mass_in = torch.rand(c.table.shape, device=DEV)
    mass = torch.empty_like(mass_in)
    _check_decode(c, q, c.decode(q, mass_in=mass_in, mass_out=mass), mass=mass, mass_in=mass_in)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_weights_accumulate(D):
    c = Cache8(21, [6, 3], [40, 10], 2, D, "i8", 64, max_tiles=9)
    q = _query(1, (2, 6, D), "bf16")
    zero = torch.zeros(c.table.shape, device=DEV)
    mass = torch.full_like(zero, 9.0)
    out = c.decode(q, mass_out=mass)                       # no mass_in: zeros
    _check_decode(c, q, out, mass=mass, mass_in=zero)
    first = mass.clone()
    c.decode(q, mass_in=mass, mass_out=mass)               # in place
    _check_decode(c, q, out, mass=mass, mass_in=first)
    assert torch.equal(c.decode(q), out)                   # the weights do not change the output


def test_decode_without_tiles_or_window():
    lay = kvarn.layout8(64)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    q = _query(1, (2, 4, 64), "f16")
    n = torch.zeros(2, dtype=torch.int32, device=DEV)
    table = torch.empty(2, 2, 0, dtype=torch.int64, device=DEV)
    win = torch.empty(2, 2, 0, 64, device=DEV)
    out = torch.full_like(q, 7.0)
    kvarn.decode_attention8(q, none, table, n, win, win, n, n, lay, out=out)
    assert int(out.count_nonzero()) == 0
    c = Cache8(5, [0, 0], [30, 128], 2, 64)
    args = list(c.args())
    args[0], args[1] = none, table
    _check_decode(c, q, kvarn.decode_attention8(q, *args))
    c = Cache8(6, [2, 1], [0, 0], 2, 64)
    args = list(c.args())
    args[3] = args[4] = win
    _check_decode(c, q, kvarn.decode_attention8(q, *args))


def test_calls_run_on_the_stream_that_they_are_given():
    c = Cache8(97, [12], [77], 2, 128)
    q = _query(3, (1, 8, 128), "f32")
    qc = _query(4, (60, 8, 128), "f32")
    want, want_c = c.decode(q), c.prefill(qc, 12 * T + 17)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    busy = torch.cuda.Event()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        busy.record()
    outs = [torch.zeros_like(q), torch.zeros_like(qc)]
    c.decode(q, out=outs[0], stream=st)
    c.prefill(qc, 12 * T + 17, out=outs[1], stream=st)
    assert not busy.query()  # nothing waited
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want_c)


def test_workspaces_allocated_for_a_stream_stay_its_own(monkeypatch):
    """A workspace that a call allocates is not handed to another stream while the call may run."""
    c = Cache8(97, [12], [77], 2, 128)
    calls, real = [], kvarn._call
    monkeypatch.setattr(kvarn, "_call", lambda *a: (calls.append(a), real(*a))[1])
    st = torch.cuda.Stream()
    for q, run in ((_query(3, (1, 8, 128), "f32"), lambda q: c.decode(q, stream=st)),
                   (_query(4, (60, 8, 128), "f32"), lambda q: c.prefill(q, 12 * T + 17, stream=st))):
        want = run(q)
        st.synchronize()
        calls.clear()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        out = run(q)
        sizes = [x for x in calls[0] if isinstance(x, int)]
        mine = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes if 256 <= n < 1 << 28 for _ in range(3)]
        assert not {t.data_ptr() for t in mine} & set(sizes)
        st.synchronize()
        assert torch.equal(out, want)


def test_decode_on_two_streams_at_once():
    cs = [Cache8(98 + i, [60, 20], [30, 99], 4, 128) for i in range(2)]
    qs = [_query(i, (2, 16, 128), "bf16") for i in range(2)]
    want = [c.decode(q) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [torch.empty(kvarn.decode8_workspace_bytes(2, 16, 4, 128, c.max_tiles, c.cap), dtype=torch.uint8, device=DEV)
          for c in cs]
    outs = [torch.empty_like(q) for q in qs]
    for _ in range(20):
        for c, q, s, w, o in zip(cs, qs, streams, ws, outs):
            c.decode(q, ws=w, out=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_decode_scales_of_either_sign_and_zero():
    c = Cache8(31, [3], [20], 2, 128)
    q = _query(2, (1, 8, 128), "f32")
    for s in (0.0, -0.05, 0.2):
        _check_decode(c, q, c.decode(q, softmax_scale=s), scale=s)


def test_decode_with_far_apart_value_scales():
    """A block of values 10^6 times the others that gets no weight must not cost the others their bits."""
    c = Cache8(41, [4], [0], 1, 128, "i8", 16)
    k, v = (x.copy() for x in rows(np.random.default_rng(4), 4 * T, 128))
    v[32:48] *= 1e6
    v[200:216] *= 1e-6
    q = np.random.default_rng(5).standard_normal((1, 2, 128)).astype(np.float32)
    k[32:48] = -3 * q[0, 0]
    kvarn.compress_tile8(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV),
                         torch.arange(4, device=DEV) * T, c.tiles, c.table[0, 0].contiguous(), c.lay)
    for x, dst in ((k, c.k), (v, c.v)):
        for i in range(4):
            _, val, s = quantise(x[T * i:T * i + T], "i8", 16)
            dst[0][0, T * i:T * i + T] = val * s.astype(np.float64).repeat(16)[:, None]
            c.vs[0][0, T * i:T * i + T] = s.repeat(16)
    qd = torch.from_numpy(q[:, :1]).to(DEV)
    _check_decode(c, qd, c.decode(qd))
    _check_decode(c, torch.from_numpy(q[:, 1:]).contiguous().to(DEV), c.decode(torch.from_numpy(q[:, 1:]).contiguous().to(DEV)))


def test_decode_bad_offsets_poison_their_head_only():
    c = Cache8(51, [4, 4], [9, 9], 2, 128)
    q = _query(3, (2, 8, 128), "f32")
    want = c.decode(q)
    for off in (-16, 8, c.tiles.numel() - c.lay.record_bytes + 16, 1 << 62, -(1 << 62)):
        t = c.table.clone()
        t[1, 0, 2] = off
        mass = torch.zeros(t.shape, device=DEV)
        out = kvarn.decode_attention8(q, c.tiles, t, *c.args()[2:], mass_out=mass)
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
        assert bool(out[1, :4].isnan().all()) and bool(mass[1, 0].isnan().all())
        assert torch.equal(out[0], want[0]) and torch.equal(out[1, 4:], want[1, 4:])
        assert bool(mass[0].isfinite().all()) and bool(mass[1, 1].isfinite().all())


def test_decode_non_finite_rows_and_queries():
    c = Cache8(61, [3, 3], [30, 30], 2, 64)
    q = _query(4, (2, 4, 64), "f32")
    want = c.decode(q)
    c.win_v[0, 1, (c.starts[0] + 7) % c.cap, 5] = float("inf")
    c.win_k[1, 0, (c.starts[1] + 29) % c.cap, 5] = float("nan")
    q2 = q.clone()
    q2[0, 0, 0] = float("nan")
    out = c.decode(q2)
    assert bool(out[0, 0].isnan().all()) and torch.equal(out[0, 1], want[0, 1])
    assert bool(out[0, 2:, 5].isnan().all())
    assert bool(out[1, :2].isnan().all()) and torch.equal(out[1, 2:], want[1, 2:])


# bit patterns: what GPU arithmetic gives for a NaN, its negative, the last and the first of the NaNs, inf, -inf
NON_FINITE = [0x7FFFFFFF, -1, 0x7F800001, 0x7FC00000, 0x7F800000, -0x800000]


@pytest.mark.parametrize("bits", NON_FINITE)
@pytest.mark.parametrize("tiles", [0, 2])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_non_finite_window_keys_poison_the_rows_that_see_them(D, tiles, bits):
    """In decode and in prefill of few rows, whatever the signs of the products with the rest of the pair."""
    c = Cache8(65, [tiles, tiles], [70, 6], 2, D)
    q, qc = _query(4, (2, 8, D), "f32"), _query(5, (4, 8, D), "f32")
    pos0 = T * tiles + 2
    want, want_c = c.decode(q), c.prefill(qc, pos0, b=1)
    for b, at in ((0, 69), (1, 4)):
        for ch in (0, D // 2 + 5, D - 1):
            word = c.win_k.view(torch.int32)[b, 1, (c.starts[b] + at) % c.cap]
            old = int(word[ch])
            word[ch] = bits
            out = c.decode(q)
            assert bool(out[b, 4:].isnan().all())
            assert torch.equal(out[b, :4], want[b, :4]) and torch.equal(out[1 - b], want[1 - b])
            if b == 1:  # the chunk's rows 2 and 3 see it
                out = c.prefill(qc, pos0, b=1)
                assert bool(out[2:, 4:].isnan().all())
                assert torch.equal(out[:2], want_c[:2]) and torch.equal(out[:, :4], want_c[:, :4])
            word[ch] = old


@pytest.mark.parametrize("bits", NON_FINITE)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_non_finite_queries_over_a_window_alone_are_nan(D, bits):
    c = Cache8(66, [0, 0], [70, 1], 2, D)
    for seed in range(4):
        q, qc = _query(seed, (2, 8, D), "f32"), _query(seed + 9, (4, 8, D), "f32")
        want, want_c = c.decode(q), c.prefill(qc, 0)  # the chunk's first row sees one key
        bad, bad_c = torch.zeros(2, 8, dtype=torch.bool, device=DEV), torch.zeros(4, 8, dtype=torch.bool, device=DEV)
        for b, h, ch in ((0, 1, 0), (1, 2, D - 1), (1, 7, D // 2 + 5)):
            q.view(torch.int32)[b, h, ch] = bits
            bad[b, h] = True
            for i in (0, 2):
                qc.view(torch.int32)[i, h, ch] = bits
                bad_c[i, h] = True
        for out, ok, nan in ((c.decode(q), want, bad), (c.prefill(qc, 0), want_c, bad_c)):
            assert bool(out[nan].isnan().all()) and torch.equal(out[~nan], ok[~nan])


def test_decode_counts_past_their_arrays_are_clamped():
    c = Cache8(71, [3], [128], 2, 64)
    q = _query(6, (1, 4, 64), "f32")
    want = c.decode(q)
    c.n_tiles.fill_(100)
    c.win_len.fill_(1000)
    c.win_start.add_(-5 * c.cap)
    assert torch.equal(c.decode(q), want)
    c.n_tiles.fill_(-3)
    c.win_len.fill_(-1)
    assert int(c.decode(q).count_nonzero()) == 0


# ---------------------------------------------------------------- prefill

def _check_prefill(c, q, pos0, out, b=0, scale=None):
    scale = c.D ** -0.5 if scale is None else scale
    C, Hq, _ = q.shape
    G = Hq // c.Hkv
    qn = q.double().cpu().numpy()
    extra = 0.0 if q.dtype == torch.float32 else 2.0 ** -11
    for h in range(c.Hkv):
        for g in range(G):
            vis = pos0 + 1 + np.arange(C)
            want, p, bound = attend(qn[:, h * G + g], c.k[b][h], c.v[b][h], scale, vis, c.vs[b][h],
                                     2.0 ** -33)
            check(out[:, h * G + g], want, bound, q.dtype, extra, p @ np.abs(c.v[b][h]))


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("code", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_matches_the_formula(D, code, io):
    c = Cache8(D + 1, [4], [77], 2, D, code, 32)
    C = 150
    q = _query(D, (C, 8, D), io)
    pos0 = 4 * T + 77 - C
    _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 6, 7, 8])
def test_prefill_head_groups(G):
    c = Cache8(G + 100, [2], [33], 2, 64, "i8", 16)
    q = _query(G, (70, 2 * G, 64), "f32")
    _check_prefill(c, q, 2 * T + 33 - 70, c.prefill(q, 2 * T + 33 - 70))


@pytest.mark.parametrize("tiles,window,C,pos0", [
    (0, 1, 1, 0), (0, 130, 130, 0), (1, 0, 128, 0), (1, 0, 1, 127), (3, 5, 20, 0), (3, 300, 64, 100),
    (3, 300, 64, 3 * T - 10), (0, 500, 90, 410), (1, 500, 3, 625), (30, 0, 3, 30 * T - 3), (30, 64, 1, 30 * T + 63), (61, 17, 2, 900),
    (5, 129, 500, 5 * T + 129 - 500)])
@pytest.mark.parametrize("D", [128, 256])
def test_prefill_lengths_and_positions(tiles, window, C, pos0, D):
    c = Cache8(7, [tiles], [window], 1, D, "e4m3", 128)
    q = _query(C, (C, 4, D), "f32")
    _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hkv,C,tiles,window", [(8, 320, 21, 70), (2, 200, 33, 0), (1, 130, 5, 500)])
def test_prefill_of_many_blocks(Hkv, C, tiles, window, D, io):
    """Enough keys that every ring of the kernel wraps, with all keys in one CTA and in several shares."""
    c = Cache8(D + C, [tiles], [window], Hkv, D, "e4m3", 64)
    q = _query(C, (C, 4 * Hkv, D), io)
    pos0 = T * tiles + window - C
    _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("case", ["rising", "uneven", "falling"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_of_long_fp32_contexts(D, case, monkeypatch):
    """More than three times the blocks after which an fp32 accumulator is emptied, in one CTA. The row's largest
    weighted score rises by about 2^9 before the second, the third and the last part ("rising"); value scales do so,
    by 300 twice ("uneven"); or the largest comes first ("falling")."""
    u = np.random.default_rng(D).choice([-1.0, 1.0], D)

    def cache_rows(rng, n, D):
        k, v = 0.3 * rng.standard_normal((n, D)), rng.standard_normal((n, D))
        if case == "uneven":
            v[2500:] *= 300
            v[5000:] *= 300
        for i, at in enumerate((1000, 3500, 5800, 7300)):  # scores 6 apart: emptyings are at 2304, 4608 and 6912 keys
            k[at] += (6.0 * (i if case == "rising" else 4 - i if case == "falling" else 1) / D ** 0.5) * u
        return k.astype(np.float32), v.astype(np.float32)

    monkeypatch.setattr("tests.cache8_helpers.rows", cache_rows)
    tiles, window, C, Hkv, G = 60, 40, 320, 8, 4  # 80 row blocks: no key shares
    c = Cache8(D, [tiles], [window], Hkv, D, "i8", 16)
    q = torch.from_numpy((np.random.default_rng(1).standard_normal((C, G * Hkv, D)) + u).astype(np.float32)).to(DEV)
    pos0 = T * tiles + window - C
    out = c.prefill(q, pos0)
    qn = q.double().cpu().numpy()
    for h in (0, 13, 31):
        want, _, bound = attend(qn[:, h], c.k[0][h // G], c.v[0][h // G], D ** -0.5, pos0 + 1 + np.arange(C),
                                c.vs[0][h // G], 2.0 ** -33)
        check(out[:, h], want, bound, torch.float32)


def test_prefill_scales_of_either_sign_and_zero():
    c = Cache8(32, [3], [20], 2, 128)
    q = _query(2, (40, 4, 128), "f32")
    for s in (0.0, -0.05, 0.2):
        _check_prefill(c, q, 200, c.prefill(q, 200, softmax_scale=s), scale=s)


@pytest.mark.parametrize("C", [9, 100])  # on the decode kernels, and on the images
@pytest.mark.parametrize("D", [64, 256])
def test_prefill_non_finite_rows_reach_only_the_rows_that_see_them(D, C):
    c = Cache8(62, [2], [60], 2, D, "i8", 16)
    pos0 = 2 * T + 34 - C                    # the chunk ends four positions past the bad row
    q = _query(8, (C, 4, D), "f32")
    want = c.prefill(q, pos0)
    for arr, bad in ((c.win_v, float("inf")), (c.win_k, float("nan")), (c.win_v, float("nan"))):
        old = arr.clone()
        arr[0, 1, (c.starts[0] + 30) % c.cap, 5] = bad
        out = c.prefill(q, pos0)
        first = 2 * T + 30 - pos0
        assert torch.equal(out[:first], want[:first])
        assert torch.equal(out[:, :2], want[:, :2])
        assert bool(out[first:, 2:].isnan().all())
        arr.copy_(old)
    # the same for a tile's group of 16 tokens: its scale says so
    k, v = rows(np.random.default_rng(9), T, D)
    k[100] = np.nan
    kvarn.compress_tile8(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), torch.zeros(1, dtype=torch.int64, device=DEV),
                         c.tiles, c.table[0, 1, 1:2].contiguous(), c.lay)
    pos0 = min(T + 93, 2 * T + 60 - C)
    seen = T + 96 - pos0                     # the chunk's row at the group's first token
    out = c.prefill(q, pos0)
    assert bool(out[seen:, 2:].isnan().all()) and bool(out[:seen].isfinite().all())
    assert bool(out[:, :2].isfinite().all())


@pytest.mark.parametrize("C", [9, 100])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_prefill_non_finite_queries_are_nan(io, C):
    """Also where every product of an infinite query with a key has the same sign."""
    c = Cache8(63, [2], [20], 2, 128, "i8", 32)
    k, v = rows(np.random.default_rng(3), T, 128)
    k[:, 5] = 1
    for i in range(2):
        kvarn.compress_tile8(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV),
                             torch.zeros(1, dtype=torch.int64, device=DEV), c.tiles, c.table[0, 1, i:i + 1].contiguous(),
                             c.lay)
    for pos0 in (T, 2 * T + 20 - C):
        q = _query(8, (C, 4, 128), io)
        want = c.prefill(q, pos0)
        q[1, 2, 5], q[2, 2, 5], q[3, 3, 7], q[5, 0, 0] = -np.inf, np.inf, np.nan, -np.inf
        out = c.prefill(q, pos0)
        bad = torch.zeros(C, 4, dtype=torch.bool, device=DEV)
        bad[1, 2] = bad[2, 2] = bad[3, 3] = bad[5, 0] = True
        assert bool(out[bad].isnan().all()) and torch.equal(out[~bad], want[~bad])


@pytest.mark.parametrize("C", [8, 200])
def test_prefill_bad_offsets_poison_what_sees_them(C):
    c = Cache8(52, [4], [9], 2, 128)
    q = _query(3, (C, 8, 128), "bf16")
    pos0 = 3 * T - 4 if C == 8 else 4 * T + 9 - C
    want = c.prefill(q, pos0)
    for off in (-16, 8, c.tiles.numel() - c.lay.record_bytes + 16, 1 << 62):
        t = c.table[0].clone()
        t[1, 3] = off
        out = kvarn.prefill_attention8(q, pos0, c.tiles, t, 4, c.win_k[0], c.win_v[0], c.starts[0], 9, c.lay)
        assert kvarn.device_error() == kvarn.DEVERR_RECORD
        first = 3 * T - pos0
        assert torch.equal(out[:, :4], want[:, :4]) and bool(out[first:, 4:].isnan().all())
        assert bool(out[:first, 4:].isfinite().all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("C", [1, 6, 100])
def test_prefill_reads_no_tile_behind_the_chunk(C, D):
    """Few rows and many: an offset that no position sees is not an error, and the result is that of the visible part."""
    c = Cache8(53, [40], [150], 2, D, "i8", 64)
    q = _query(3, (C, 8, D), "f32")
    for pos0 in (0, 3 * T - C, 3 * T + 1 - C, 20 * T + 5, 40 * T - C, 40 * T + 20 - C):
        if pos0 < 0:
            continue
        t = c.table[0].clone()
        t[:, (pos0 + C - 1) // T + 1:] = torch.tensor([[-16], [8]], device=DEV)
        out = kvarn.prefill_attention8(q, pos0, c.tiles, t, 40, c.win_k[0], c.win_v[0], c.starts[0], 150, c.lay)
        assert kvarn.device_error() == 0
        _check_prefill(c, q, pos0, out)


@pytest.mark.parametrize("C", [4, 100])
def test_a_pool_smaller_than_a_record_is_not_read(C):
    lay = kvarn.layout8(128)
    pool = torch.zeros(4096, dtype=torch.uint8, device=DEV)
    win = torch.randn(1, 128, 128, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int64, device=DEV)
    out = kvarn.prefill_attention8(_query(1, (C, 1, 128), "f32"), 128, pool, table, 1, win, win, 0, 128, lay)
    assert kvarn.device_error() == kvarn.DEVERR_RECORD and bool(out.isnan().all())
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    out = kvarn.decode_attention8(_query(1, (1, 1, 128), "f32"), pool, table[None], one, win[None], win[None], one, one, lay)
    assert kvarn.device_error() == kvarn.DEVERR_RECORD and bool(out.isnan().all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("C,G", [(5, 8), (6, 8), (11, 4), (64, 1), (13, 5), (16, 4)])
def test_prefill_around_the_change_of_kernels(C, G, io):
    """Chunks just below and above the row count from which the images pay; also at 0 tiles."""
    for tiles, window in ((70, 90), (0, 130)):
        c = Cache8(C + G, [tiles], [window], 3, 64, "i8", 32)
        q = _query(C, (C, 3 * G, 64), io)
        pos0 = T * tiles + window - C
        _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("io", ["f32", "f16"])
@pytest.mark.parametrize("Hkv,tiles,window", [(2, 0, 1500), (8, 0, 300), (1, 3, 900), (8, 9, 20)])
def test_prefill_around_the_change_of_kernels_with_windows(Hkv, tiles, window, io):
    """Chunks from a few rows to 64 groups of eight, over windows that decide which kernels serve them."""
    c = Cache8(window, [tiles], [window], Hkv, 64, "i8", 32)
    for C in (2, 8, 11, 20, 40, 64):
        q = _query(C, (C, 4 * Hkv, 64), io)
        pos0 = T * tiles + window - C
        _check_prefill(c, q, pos0, c.prefill(q, pos0))


def test_prefill_of_one_position_agrees_with_decode():
    c = Cache8(81, [33], [50], 4, 128, "e4m3", 64)
    q = _query(9, (1, 16, 128), "f32")
    pos0 = 33 * T + 49
    _check_prefill(c, q, pos0, c.prefill(q, pos0))
    _check_decode(c, q, c.decode(q))


# ---------------------------------------------------------------- eviction

def _evict_plain(table, mass, n, keep, sinks, recent):
    out_t, out_m, gone = [], [], []
    for b in range(len(n)):
        for h in range(table.shape[1]):
            m, t = mass[b, h], table[b, h]
            if n[b] <= keep:
                stay = list(range(n[b]))
            else:
                key = np.where(np.isnan(m), np.inf, m + 0.0)
                mid = list(range(sinks, n[b] - recent))
                best = sorted(mid, key=lambda i: (-key[i], i))[:keep - sinks - recent]
                stay = sorted(list(range(sinks)) + best + list(range(n[b] - recent, n[b])))
            left = [i for i in range(n[b]) if i not in set(stay)]
            pad = table.shape[2]
            out_t.append([t[i] for i in stay] + [-1] * (pad - len(stay)))
            out_m.append([m[i] for i in stay] + [0.0] * (pad - len(stay)))
            gone.append([t[i] for i in left] + [-1] * (pad - len(left)))
    f = lambda x, d: np.array(x, d).reshape(table.shape)
    return f(out_t, np.int64), f(out_m, np.float32), np.minimum(n, keep), f(gone, np.int64)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,H,n_max,keep,sinks,recent", [
    (1, 8, 160, 128, 1, 8), (3, 1, 1500, 700, 4, 64), (2, 2, 33, 1, 0, 0), (2, 3, 40, 40, 0, 0), (2, 5, 300, 20, 20, 0),
    (2, 16, 100, 30, 0, 30), (1, 17, 130, 64, 3, 5), (4, 4, 1, 1, 0, 0), (2, 9, 777, 776, 0, 1), (1, 20, 64, 3, 1, 1)])
def test_evict_matches_the_rule(B, H, n_max, keep, sinks, recent, in_place):
    rng = np.random.default_rng(n_max)
    mass = np.round(np.exp(rng.standard_normal((B, H, n_max))) * 8) / 8  # ties
    mass = mass.astype(np.float32)
    flat = mass.reshape(-1)
    for x in (np.nan, np.inf, -np.inf, -0.0, 0.0, -1.5):
        flat[rng.integers(0, flat.size, 1 + flat.size // 40)] = x
    table = rng.permutation(B * H * n_max).reshape(B, H, n_max) * 32896
    n = rng.integers(n_max // 2, n_max + 1, B).astype(np.int32)
    n[0] = n_max
    want = _evict_plain(table, mass, n, keep, sinks, recent)
    t, m, nt = (torch.from_numpy(x).to(DEV) for x in (table, mass.copy(), n.copy()))
    ev = torch.zeros_like(t)
    kw = {} if in_place else dict(table_out=torch.empty_like(t), mass_out=torch.empty_like(m), n_tiles_out=torch.empty_like(nt))
    got = kvarn.evict_tiles(t, m, nt, keep, sinks, recent, evicted=ev, **kw)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w, equal_nan=g.dtype == torch.float32)
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(nt.cpu().numpy(), n)


def test_evict_clamps_counts():
    t = torch.arange(12, device=DEV).view(2, 2, 3)
    m = torch.ones(2, 2, 3, device=DEV)
    n = torch.tensor([9, -4], dtype=torch.int32, device=DEV)
    table, mass, n_out, _ = kvarn.evict_tiles(t.clone(), m, n, 2)
    assert n_out.tolist() == [2, 0]
    assert table.tolist() == [[[0, 1, -1], [3, 4, -1]], [[-1] * 3] * 2]


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("D,io", [(128, "f32"), (64, "bf16")])
def test_a_cache_lives_prefill_decode_promote_evict(D, io):
    """A prompt's tiles and window, decode steps that append, promote and weigh, an eviction, and decode and
    prefill over what is left, each against the formula on the rows the cache then holds."""
    Hkv, G = 2, 3
    c = Cache8(91, [6], [120], Hkv, D, "i8", 32, cap=256, max_tiles=9)
    rng = np.random.default_rng(10)
    rb = c.lay.record_bytes
    pool = torch.zeros(c.tiles.numel() + 2 * Hkv * rb, dtype=torch.uint8, device=DEV)
    pool[:c.tiles.numel()] = c.tiles
    free = [c.tiles.numel() + i * rb for i in range(2 * Hkv)]
    c.tiles = pool
    c.starts[0] = 0                                      # a ring that starts on a tile
    wk, wv = torch.zeros(1, Hkv, 256, D, device=DEV), torch.zeros(1, Hkv, 256, D, device=DEV)
    wk[0, :, :120] = torch.from_numpy(c.k[0][:, 6 * T:]).float()
    wv[0, :, :120] = torch.from_numpy(c.v[0][:, 6 * T:]).float()
    c.win_k, c.win_v = wk, wv
    c.win_start.zero_()
    q = _query(11, (40, Hkv * G, D), io)
    _check_prefill(c, q, 6 * T + 80, c.prefill(q, 6 * T + 80))
    mass = torch.zeros(c.table.shape, device=DEV)
    for step in range(12):
        k, v = rows(rng, Hkv, D)
        kvarn.append_window(torch.from_numpy(k).to(DEV).view(1, 1, Hkv, D), torch.from_numpy(v).to(DEV).view(1, 1, Hkv, D),
                            c.win_k, c.win_v, c.win_start, c.win_len)
        c.k[0] = np.concatenate([c.k[0], k[:, None].astype(np.float64)], 1)
        c.v[0] = np.concatenate([c.v[0], v[:, None].astype(np.float64)], 1)
        c.vs[0] = np.concatenate([c.vs[0], np.abs(v).max(1, keepdims=True) / 256.0], 1)
        promote = c.windows[0] + 1 >= T
        if promote:
            src = torch.arange(Hkv, device=DEV) * 256 + c.starts[0]
            dst = torch.tensor([free.pop() for _ in range(Hkv)], device=DEV)
            kvarn.compress_tile8(c.win_k.view(-1, D), c.win_v.view(-1, D), src, c.tiles, dst, c.lay)
            c.table[0, :, c.tiles_of[0]] = dst
            at = T * c.tiles_of[0]
            for x in (c.k[0], c.v[0]):
                for h in range(Hkv):
                    _, val, s = quantise(x[h, at:at + T].astype(np.float32), "i8", 32)
                    x[h, at:at + T] = val * s.astype(np.float64).repeat(16)[:, None]
                    c.vs[0][h, at:at + T] = s.repeat(16)  # V's, the second of the two
            c.tiles_of[0] += 1
            c.starts[0] = (c.starts[0] + T) % 256
        kvarn.window_advance(c.win_start, c.win_len, c.n_tiles, 1, int(promote), 256)
        c.windows[0] += 1 - T * promote
        q1 = _query(20 + step, (1, Hkv * G, D), io)
        before = mass.clone()
        out = c.decode(q1, mass_in=mass, mass_out=mass)
        _check_decode(c, q1, out, mass=mass, mass_in=before)
    assert c.tiles_of[0] == 7 and int(c.n_tiles[0]) == 7 and int(c.win_len[0]) == c.windows[0]
    want = _evict_plain(c.table.cpu().numpy(), mass.cpu().numpy(), [7], 4, 1, 1)
    old = c.table[0].cpu().numpy().copy()
    gone = torch.empty_like(c.table)
    kvarn.evict_tiles(c.table, mass, c.n_tiles, 4, sinks=1, recent=1, evicted=gone)
    assert np.array_equal(c.table.cpu().numpy(), want[0]) and np.array_equal(gone.cpu().numpy(), want[3])
    ks, vs, ss = [], [], []
    for h in range(Hkv):
        left = [int(np.flatnonzero(old[h] == t)[0]) for t in want[0][0, h, :4]]
        at = np.concatenate([np.arange(T * i, T * i + T) for i in left] + [np.arange(7 * T, c.k[0].shape[1])])
        ks.append(c.k[0][h, at])
        vs.append(c.v[0][h, at])
        ss.append(c.vs[0][h, at])
    c.k[0], c.v[0], c.vs[0] = np.stack(ks), np.stack(vs), np.stack(ss)
    c.tiles_of[0] = 4
    q1 = _query(50, (1, Hkv * G, D), io)
    _check_decode(c, q1, c.decode(q1))
    q = _query(51, (3, Hkv * G, D), io)
    pos0 = 4 * T + c.windows[0] - 3
    _check_prefill(c, q, pos0, c.prefill(q, pos0))


@pytest.mark.parametrize("D", [64, 256])
def test_records_and_rows_past_32_bit_offsets(D):
    """A pool longer than 2^32 bytes and raw rows past 2^31 elements give what small ones give."""
    c = Cache8(94, [9], [30], 2, D, "e4m3", 32)
    rb, n = c.lay.record_bytes, 18
    k, v = (torch.from_numpy(x).to(DEV) for x in rows(np.random.default_rng(5), n * T, D))
    src, near = torch.arange(n, device=DEV) * T, c.table.view(-1)
    kvarn.compress_tile8(k, v, src, c.tiles, near, c.lay)
    out_k, out_v = torch.empty_like(k), torch.empty_like(v)
    kvarn.expand_tile8(c.tiles, near, out_k, out_v, src, c.lay)

    shift = (1 << 32) + 16 - (n // 2) * rb  # records on both sides of 2^32 and one across it
    big = torch.empty(shift + n * rb, dtype=torch.uint8, device=DEV)
    row0 = (1 << 31) // D + 3
    raw_k, raw_v = (torch.empty(row0 + n * T, D, device=DEV) for _ in range(2))
    raw_k[row0:], raw_v[row0:] = k, v
    kvarn.compress_tile8(raw_k, raw_v, src + row0, big, near + shift, c.lay)
    assert torch.equal(big[shift:], c.tiles)
    raw_k[row0:], raw_v[row0:] = 0, 0
    kvarn.expand_tile8(big, near + shift, raw_k, raw_v, src + row0, c.lay)
    assert torch.equal(raw_k[row0:], out_k) and torch.equal(raw_v[row0:], out_v)
    del raw_k, raw_v

    table = c.table + shift
    q = _query(1, (1, 8, D), "f32")
    assert torch.equal(kvarn.decode_attention8(q, big, table, *c.args()[2:]), c.decode(q))
    for C in (3, 200):
        q = _query(2, (C, 8, D), "bf16")
        pos0 = 9 * T + 30 - C
        out = kvarn.prefill_attention8(q, pos0, big, table[0], 9, c.win_k[0], c.win_v[0], c.starts[0], 30, c.lay)
        assert torch.equal(out, c.prefill(q, pos0))


# ---------------------------------------------------------------- launches

def test_decode_launch_modes_and_graphs_are_bit_identical():
    c = Cache8(95, [20, 7], [100, 3], 4, 128, "i8", 64)
    q = _query(12, (2, 16, 128), "bf16")
    mass = torch.zeros(c.table.shape, device=DEV)
    ref = c.decode(q, mass_out=mass)
    both = kvarn.LAUNCH_PDL | kvarn.LAUNCH_PREFETCH
    need = kvarn.decode8_workspace_bytes(2, 16, 4, 128, c.max_tiles, c.cap)
    for flags in (0, kvarn.LAUNCH_PDL, both):
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        out, m = torch.empty_like(q), torch.empty_like(mass)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            c.decode(q, mass_out=m, ws=ws, out=out, flags=flags)
        st.synchronize()
        assert torch.equal(out, ref) and torch.equal(m, mass)
        out.zero_()
        m.zero_()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                c.decode(q, mass_in=m, mass_out=m, ws=ws, out=out, flags=flags)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        assert torch.allclose(m, 3 * mass, rtol=2.0 ** -21)


def test_prefill_compress_and_evict_replay_from_a_graph():
    c = Cache8(96, [9], [100], 2, 128, "e4m3", 64)
    q = _query(13, (30, 8, 128), "f32")
    pos0 = 9 * T + 70
    ref = c.prefill(q, pos0)
    ws = torch.empty(kvarn.prefill8_workspace_bytes(30, 9, 100, 8, 2, 128), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    mass = torch.rand(c.table.shape, device=DEV)
    to = (torch.empty_like(c.table), torch.empty_like(mass), torch.empty_like(c.n_tiles), torch.empty_like(c.table))
    want = [x.clone() for x in kvarn.evict_tiles(c.table, mass, c.n_tiles, 5, 1, 1, *to)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        c.prefill(q, pos0, ws=ws, out=out)
        kvarn.evict_tiles(c.table, mass, c.n_tiles, 5, 1, 1, *to)
    for x in to:
        x.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    assert all(torch.equal(a, b) for a, b in zip(to, want))
