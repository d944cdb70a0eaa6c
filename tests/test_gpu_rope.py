"""norm_rotate on the GPU against its formula in 64 bits, angles reduced in exact arithmetic."""
import numpy as np
import pytest
import torch

from kv_cache_quantization_token_gb300 import kvarn
from tests.cache4_helpers import DEV, HALF_STEP, check, norm_rotate  # noqa: F401

pytestmark = pytest.mark.gpu
IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _rows(seed, shape, io):
    x = np.random.default_rng(seed).standard_normal(shape) * np.exp(np.random.default_rng(seed + 1).standard_normal(shape[-1]))
    return torch.from_numpy(x.astype(np.float32)).to(IO[io]).to(DEV)


def _host(x):
    return None if x is None else x.double().cpu().numpy()


def _check(q, k, got, qw, kw, eps, pos, freq, axis, adjacent, hadamard):
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        if x is not None:
            want, bound = norm_rotate(_host(x), _host(w), eps, pos, freq, axis, adjacent, hadamard)
            check(y, want, bound, x.dtype)


@pytest.mark.parametrize("hadamard", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_matches_the_formula(D, io, adjacent, hadamard):
    q, k = _rows(D, (7, 9, D), io), _rows(D + 1, (7, 3, D), io)
    qw, kw = _rows(2, (D,), io), _rows(3, (D,), io)
    pos = np.array([0, 1, 5, 1000, 16384, 131071, 999983])
    for R in (D, D // 2, 3 * D // 4, 16):
        freq = [10000.0 ** (-2 * i / R) for i in range(R // 2)]
        plan = kvarn.rotary(R, pairing="adjacent" if adjacent else "halves")
        got = kvarn.norm_rotate(q, k, torch.from_numpy(pos).to(DEV), plan, q_weight=qw, k_weight=kw, eps=1e-6,
                                hadamard=hadamard)
        _check(q, k, got, qw, kw, 1e-6, pos[None], freq, [0] * (R // 2), adjacent, hadamard)


@pytest.mark.parametrize("adjacent", [False, True])
def test_positions_of_several_axes(adjacent):
    D, n = 128, 24
    q, k = _rows(5, (11, 4, D), "f32"), _rows(6, (11, 2, D), "f32")
    rng = np.random.default_rng(1)
    for axes in (2, 3, 4):
        axis = list(rng.integers(0, axes, n))
        axis[3] = axes - 1
        freq = list(rng.uniform(-1, 1, n))
        pos = rng.integers(-5000, 5000, (axes, 11))
        plan = kvarn.rotary(2 * n, inv_freq=freq, pair_axis=axis, pairing="adjacent" if adjacent else "halves")
        got = kvarn.norm_rotate(q, k, torch.from_numpy(pos).to(DEV), plan)
        _check(q, k, got, None, None, None, pos, freq, axis, adjacent, False)
    pos = rng.integers(0, 70, (3, 11))
    plan = kvarn.rotary(128, theta=1e6, sections=(16, 24, 24))
    got = kvarn.norm_rotate(q, k, torch.from_numpy(pos).to(DEV), plan, eps=1e-5)
    _check(q, k, got, None, None, 1e-5, pos, [1e6 ** (-i / 64) for i in range(64)], [0] * 16 + [1] * 24 + [2] * 24, False, False)


def test_far_and_negative_positions():
    D = 64
    pos = np.array([2 ** 31, 2 ** 31 - 1, -1, -(2 ** 31), 2 ** 20 + 1, 123456789, -987654321])
    q = _rows(7, (7, 3, D), "f32")
    freq = [500000.0 ** (-i / 32) for i in range(32)]
    plan = kvarn.rotary(64, theta=500000.0)
    got = kvarn.norm_rotate(q, None, torch.from_numpy(pos).to(DEV), plan)
    assert got[1] is None
    _check(q, None, got, None, None, None, pos[None], freq, [0] * 32, False, False)


@pytest.mark.parametrize("T", [1, 2, 33, 1000, 4866, 4867])
def test_numbers_of_tokens(T):
    """One CTA per row block of a token, and several tokens to a CTA; rows of a packed product, in place and out
    of place, bit for bit the same; what lies between the rows stays."""
    for D, Hq, Hkv in ((128, 5, 3), (64, 1, 1), (256, 2, 0), (128, 33, 8)):
        if T * D * (Hq + Hkv) > 4_000_000:
            continue
        x = _rows(T, (T, Hq + 2 * Hkv + 1, D), "bf16")
        q, k = x[:, :Hq], x[:, Hq:Hq + Hkv] if Hkv else None
        w = _rows(2, (D,), "bf16")
        pos = torch.arange(T, device=DEV) * 37
        plan = kvarn.rotary(D)
        a = kvarn.norm_rotate(q, k, pos, plan, q_weight=w, eps=1e-6, hadamard=True)
        y = x.clone()
        kq, kk = y[:, :Hq], y[:, Hq:Hq + Hkv] if Hkv else None
        kvarn.norm_rotate(kq, kk, pos, plan, q_weight=w, eps=1e-6, hadamard=True, q_out=kq, k_out=kk, flags=kvarn.LAUNCH_PDL)
        assert torch.equal(kq, a[0]) and (kk is None or torch.equal(kk, a[1]))
        assert torch.equal(y[:, Hq + Hkv:], x[:, Hq + Hkv:])
        some = np.unique(np.linspace(0, T - 1, 12).astype(int))
        freq = [10000.0 ** (-2 * i / D) for i in range(D // 2)]
        _check(q[some], None if k is None else k[some], (a[0][some], None if k is None else a[1][some]), w, None, 1e-6,
               37 * some[None], freq, [0] * (D // 2), False, True)


@pytest.mark.parametrize("Hq,Hkv", [(1, 0), (5, 3), (17, 1)])
@pytest.mark.parametrize("D", [64, 256])
def test_warps_that_take_many_tokens(D, Hq, Hkv):
    """Shares that begin in the middle of a token, end in another and span whole ones: each token as if alone."""
    T = 12345
    q, k = _rows(9, (T, Hq, D), "bf16"), _rows(10, (T, Hkv, D), "bf16") if Hkv else None
    qw, kw = _rows(2, (D,), "bf16"), _rows(3, (D,), "bf16") if Hkv else None
    pos = torch.arange(T, device=DEV) * 3
    plan = kvarn.rotary(D // 2)
    call = lambda i: kvarn.norm_rotate(q[i], None if k is None else k[i], pos[i], plan, q_weight=qw, k_weight=kw, eps=1e-6)
    got = call(slice(None))
    for lo in range(0, T, 1000):
        part = call(slice(lo, min(lo + 1000, T)))
        for x, y in zip(got, part):
            assert y is None or torch.equal(x[lo:lo + 1000], y)


def test_parts_alone():
    """A norm without weights or rotation, a transform alone (rotate_query's, to rounding), nothing at all."""
    q, k = _rows(9, (6, 3, 128), "f32"), _rows(10, (6, 2, 128), "f32")
    got = kvarn.norm_rotate(q, k, None, None, eps=0.0)
    _check(q, k, got, None, None, 0.0, None, None, None, False, False)
    got = kvarn.norm_rotate(q, k, None, None, hadamard=True)
    _check(q, k, got, None, None, None, None, None, None, False, True)
    ref = kvarn.rotate_query(q)
    assert bool(((got[0] - ref).abs() <= 22 * 2.0 ** -24 * q.abs().sum(-1, keepdim=True) / 128 ** 0.5).all())
    got = kvarn.norm_rotate(q, k, None, None)
    assert torch.equal(got[0], q) and torch.equal(got[1], k)
    e = torch.empty(0, 3, 128, device=DEV)
    assert kvarn.norm_rotate(e, None, None, None, eps=1e-6)[0].shape == (0, 3, 128)


def test_scores_are_kept():
    """Rotated queries and keys meet by the difference of their positions, transformed or not."""
    D = 128
    q, k = _rows(11, (1, 1, D), "f32").expand(50, 1, D).contiguous(), _rows(12, (1, 1, D), "f32").expand(50, 1, D).contiguous()
    pos = torch.arange(50, device=DEV) * 1000
    plan = kvarn.rotary(D)
    size = float((q[0].abs() * k[0].abs()).sum()) * 2
    for hadamard in (False, True):
        a, b = kvarn.norm_rotate(q, k, pos, plan, hadamard=hadamard)
        c, _ = kvarn.norm_rotate(q, k, pos + 12345, plan, hadamard=hadamard)
        _, d = kvarn.norm_rotate(q, k, pos + 12345, plan, hadamard=hadamard)
        one, two = (a * b).double().sum(-1), (c * d).double().sum(-1)
        # each element is within 2^-19 of its pair; the transform spreads that over the row
        lim = 2.0 ** -17 * (size if not hadamard else float(q[0].abs().sum() * k[0].abs().sum()))
        assert float((one - two).abs().max()) <= lim


def test_non_finite_values_stay_in_their_rows():
    q = _rows(13, (4, 3, 64), "f32")
    plan = kvarn.rotary(32)
    pos = torch.arange(4, device=DEV)
    want, _ = kvarn.norm_rotate(q, None, pos, plan, eps=1e-6, hadamard=True)
    x = q.clone()
    x[1, 2, 5], x[3, 0, 60] = float("nan"), float("inf")
    out, _ = kvarn.norm_rotate(x, None, pos, plan, eps=1e-6, hadamard=True)
    bad = torch.zeros(4, 3, dtype=torch.bool, device=DEV)
    bad[1, 2] = bad[3, 0] = True
    assert bool(out[bad].isnan().any(-1).all()) and torch.equal(out[~bad], want[~bad])
    # without a norm an infinity behind the turned channels stays one, and its neighbours stay themselves
    out, _ = kvarn.norm_rotate(x, None, pos, plan)
    assert bool(out[3, 0, 60].isinf()) and bool(out[3, 0, :60].isfinite().all())


def test_captured_calls_replay():
    q, k = _rows(14, (3, 8, 128), "bf16"), _rows(15, (3, 2, 128), "bf16")
    pos = torch.tensor([5, 6, 7], device=DEV)
    plan = kvarn.rotary(128)
    qo, ko, g = torch.empty_like(q), torch.empty_like(k), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        kvarn.norm_rotate(q, k, pos, plan, eps=1e-6, q_out=qo, k_out=ko, flags=kvarn.LAUNCH_PDL)
    for step in range(3):
        pos += 1000
        g.replay()
        torch.cuda.synchronize()
        a, b = kvarn.norm_rotate(q, k, pos, plan, eps=1e-6)
        assert torch.equal(qo, a) and torch.equal(ko, b)


def test_refusals():
    q, k = _rows(16, (3, 4, 64), "f32"), _rows(17, (3, 2, 64), "f32")
    plan, pos = kvarn.rotary(64), torch.arange(3, device=DEV)
    for kw in (dict(positions=pos[:2]), dict(positions=pos.int()), dict(positions=pos.cpu()), dict(positions=pos.view(3, 1)),
               dict(rot=kvarn.rotary(64, sections=(16, 16))), dict(q_weight=q[0, 0]), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=1e-6, q_weight=q[0, 0, :32]), dict(eps=1e-6, q_weight=q[0, 0].half()), dict(k=k[:2]), dict(k=k.half()),
               dict(q_out=k), dict(k=None, k_out=k), dict(q=q.cpu()), dict(q=q.double()), dict(q=q.transpose(0, 1)),
               dict(q_out=k.new_empty(3, 4, 64).transpose(0, 1).contiguous().transpose(0, 1))):
        a = dict(q=q, k=k, positions=pos, rot=plan)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            kvarn.norm_rotate(**a)
    for kw in (dict(rot=kvarn.rotary(128)), dict(q_out=q.view(-1)[:3 * 4 * 64].view(3, 4, 64), k_out=q[:, :2])):
        a = dict(q=q, k=k, positions=pos, rot=plan)
        a.update(kw)
        with pytest.raises(kvarn.KvarnError):
            kvarn.norm_rotate(**a)
