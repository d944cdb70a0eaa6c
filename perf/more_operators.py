"""The operators of a cache held in 4 bits that takes rows as they come: what each computes, in plain torch operations,
and the calls that reach the library's kernels.

  rope      queries and keys of new tokens: RMS norm of each head, rotation by position (one to three axes), and on
            request an orthonormal Walsh-Hadamard transform of each head, in one pass
  store     new K and V rows quantised into the cache behind the tokens it holds, and those rows read back
  decode    attention of one query token per sequence over the cache, with or without the attention weight that
            each tile received
  prefill   causal attention of a chunk of query positions of one sequence over the cache

A record holds one 128-token tile of one KV head as four runs of 32 tokens. A run: K units [D/128 or 1][32][D/4, 32 at
most], V units [D/32][32][8], K scales [32][D/32], V scales [D/32][32]; a unit is 16 bits with four consecutive channels
of a token, a scale an fp16 number for 32 channels of a token.
"""
import math

import torch

own = False

TILE = 128
RUN = 32             # tokens of a run, and channels of a group
MOST = 14336.0       # largest magnitude that 4 bits hold
IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6


def _rope(name, io, D, G, Hkv, tokens, rot, adjacent, axes, norm, hadamard, packed, far):
    return {"name": name, "op": "rope", "io": io, "D": D, "G": G, "Hkv": Hkv, "tokens": tokens, "rot": rot,
            "adjacent": adjacent, "axes": axes, "norm": norm, "hadamard": hadamard, "packed": packed, "far": far}


def _store(name, io, D, Hkv, B, T, held, ragged, packed):
    return {"name": name, "op": "store", "io": io, "D": D, "Hkv": Hkv, "B": B, "T": T, "held": held, "ragged": ragged,
            "packed": packed}


def _decode(name, io, D, B, G, Hkv, length, ragged, mass):
    return {"name": name, "op": "decode", "io": io, "D": D, "B": B, "G": G, "Hkv": Hkv, "len": length, "ragged": ragged,
            "mass": mass}


def _prefill(name, io, D, G, Hkv, held, C):
    return {"name": name, "op": "prefill", "io": io, "D": D, "G": G, "Hkv": Hkv, "held": held, "C": C}


def listed():
    return [
        # one layer of an 8B-like model's decode step: the heads of one new token
        _rope("rope_step", "bf16", 128, 4, 8, 1, 128, False, 1, True, False, True, 16384),
        # image and video tokens among text: three axes, odd sizes, heads transformed for the 4-bit cache
        _rope("rope_media", "f16", 128, 5, 3, 1337, 128, False, 3, True, True, False, 400000),
        # a whole 8,192-token prompt, straight from the product that makes queries, keys and values
        _rope("rope_prompt", "bf16", 128, 4, 8, 8192, 128, False, 1, True, False, True, 0),
        # one layer of a batched decode step: a new token of each of 32 sequences
        _store("store_step", "bf16", 128, 8, 32, 1, 1000, True, True),
        # the prompts of four sequences of different lengths, up to 2,048 tokens
        _store("store_prompt", "bf16", 128, 8, 4, 2048, 77, True, True),
        # one layer of a decode step soon after a short prompt, at full precision
        _decode("decode_short", "f32", 128, 1, 2, 8, 401, False, False),
        # one layer of an 8B-like decode step at 16k context
        _decode("decode_16k", "bf16", 128, 1, 4, 8, 16461, False, False),
        # a few sequences of a small-head model whose tiles are weighed for eviction
        _decode("decode_weighed", "f16", 64, 5, 7, 3, 32001, True, True),
        # batched serving with large heads: 32 ragged sequences of up to 32k tokens
        _decode("decode_batch_d256", "bf16", 256, 32, 4, 4, 32768, True, False),
        # a few drafted tokens checked at once, at full precision
        _prefill("prefill_draft", "f32", 128, 4, 8, 1960, 5),
        # an odd last chunk of a prompt, five query heads per KV head
        _prefill("prefill_odd", "f16", 64, 5, 3, 4636, 301),
        # the last 512-token chunk of a 15,500-token prompt of an 8B-like model
        _prefill("prefill_15k", "bf16", 128, 4, 8, 14988, 512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "store", "decode", "decode", "prefill", "prefill"])
    io, D = rng.choice(["f32", "f16", "bf16"]), rng.choice([64, 128, 256])
    size = 4 if io == "f32" else 2
    G, Hkv = rng.randint(1, 8), _log(rng, 1, 8)
    if op == "rope":
        tokens = _log(rng, 1, 8192 * 40 * 256 // ((G + 1) * Hkv * D * size))
        rot = rng.choice([D, D, D // 2, 3 * D // 4])
        case = _rope("", io, D, G, Hkv, tokens, rot, rng.random() < 0.3, rng.choice([1, 1, 2, 3]), rng.random() < 0.7,
                     rng.random() < 0.4, rng.random() < 0.5, rng.choice([0, 5000, 1000000]))
    elif op == "store":
        B = _log(rng, 1, 32)
        T = _log(rng, 1, max(2, 4 * 2048 * 8 * 128 * 2 // (B * Hkv * D * size)))
        case = _store("", io, D, Hkv, B, T, rng.randint(0, 1500), rng.random() < 0.6, rng.random() < 0.5)
    elif op == "decode":
        B = _log(rng, 1, 32)
        length = _log(rng, 1, max(2, min(120000, 128 * 32768 * 256 // (B * Hkv * D))))
        case = _decode("", io, D, B, G, Hkv, length, rng.random() < 0.5, rng.random() < 0.4)
    else:
        C = _log(rng, 1, 700)
        held = _log(rng, 1, max(2, min(60000, 15000 * 512 * 32 * 128 // (C * G * Hkv * D)))) - 1
        case = _prefill("", io, D, G, Hkv, held, C)
    del case["name"]
    return case


# ---------------------------------------------------------------------------------------------------------------
# inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(g, lead, tokens, D):
    """K with a spread of channel scales and a few outlier channels, V with heavy-tailed token scales: [lead, tokens, D]."""
    ch = torch.randn(lead, 1, D, generator=g, device=DEV).exp()
    ch = torch.where(torch.rand(lead, 1, D, generator=g, device=DEV) < 0.02, ch * 20, ch)
    k = torch.randn(lead, tokens, D, generator=g, device=DEV) * ch
    t4 = torch.randn(lead, tokens, 1, generator=g, device=DEV) / (
        torch.randn(lead, tokens, 4, generator=g, device=DEV).square().mean(-1, keepdim=True) + 1e-3).sqrt()
    v = torch.randn(lead, tokens, D, generator=g, device=DEV) * t4.abs()
    return k, v


def _quantise(x):
    """x [..., D] -> codes -7..7 [..., D] and a scale for each group of 32 channels [..., D/32], both in 64 bits: the
    quotients next to the border of two codes, or of two scales."""
    y = x.double().unflatten(-1, (-1, RUN))
    least = y.abs().amax(-1) / 7
    step = torch.exp2((torch.frexp(least).exponent - 8).clamp_min(-24).double())
    s = ((least / step).ceil() * step).clamp_min(2.0 ** -24)
    return (y / s.unsqueeze(-1)).round().flatten(-2), s


def _units(codes):
    """Codes [..., D] -> units [..., D/4] as integers: code + 8 of the four channels at bits 6, 10 and 2 and, the
    fourth, its low half at bit 14 and its high half at bit 0."""
    u = (codes + 8).to(torch.int32).unflatten(-1, (-1, 4))
    return u[..., 0] << 6 | u[..., 1] << 10 | u[..., 2] << 2 | (u[..., 3] & 3) << 14 | u[..., 3] >> 2


def _scale_place():
    """Place of token t's V scale in its run."""
    t = torch.arange(RUN, device=DEV)
    return 8 * (t % 8 // 2) + 2 * (t // 8) + t % 2


def _records(k, v):
    """Rows [n, 128, D] of n tiles -> records [n, 144 D]."""
    n, _, D = k.shape
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    wide = min(D, 128) // 4
    ku = _units(kc).view(n, 4, RUN, -1, wide).transpose(2, 3)
    vu = _units(vc).view(n, 4, RUN, D // 32, 8).transpose(2, 3)
    ks = ks.view(n, 4, RUN, D // 32)
    vs = torch.empty(n, 4, D // 32, RUN, dtype=torch.float64, device=DEV).index_copy_(
        3, _scale_place(), vs.view(n, 4, RUN, D // 32).transpose(2, 3).contiguous())
    parts = [x.reshape(n, 4, -1).to(torch.int16) for x in (ku, vu)]
    parts += [x.reshape(n, 4, -1).half().view(torch.int16) for x in (ks, vs)]
    return torch.cat(parts, 2).view(torch.uint8).view(n, -1)


def _paged(g, heads, n, D):
    """n tiles of each head, scattered over a pool, and the byte offset of each."""
    rb = 144 * D
    place = torch.randperm(heads * n, generator=g, device=DEV)
    pool = torch.empty(heads * n, rb, dtype=torch.uint8, device=DEV)
    for h in range(heads):
        k, v = _rows(g, 1, TILE * n, D)
        pool[place[h * n:(h + 1) * n]] = _records(k.view(n, TILE, D), v.view(n, TILE, D))
    return pool.view(-1), (place * rb).view(heads, n)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op, D, H, io = case["op"], case["D"], case["Hkv"], IO[case["io"]]
    if op == "rope":
        T, Hq = case["tokens"], case["G"] * H
        x = torch.randn(T, Hq + 2 * H, D, generator=g, device=DEV)
        x = (x * torch.randn(1, Hq + 2 * H, D, generator=g, device=DEV).exp()).to(io)
        st["q"], st["k"] = x[:, :Hq], x[:, Hq:Hq + H]  # the rows of a product that makes q, k and v at once
        if not case["packed"]:
            st["q"], st["k"] = st["q"].contiguous(), st["k"].contiguous()
        n = case["rot"] // 2
        st["inv_freq"] = [10000.0 ** (-i / n) for i in range(n)]
        cut = [n // 4, n // 4 + (n - n // 4) // 2, n] if case["axes"] == 3 else [n // 2, n]
        st["pair_axis"] = [0 if case["axes"] == 1 else sum(i >= c for c in cut) for i in range(n)]
        pos = torch.arange(T, device=DEV).view(1, T) + case["far"]
        if case["axes"] > 1:  # time, height and width of a grid of patches
            pos = torch.cat([pos // 64, pos % 64 // 8, pos % 8])[:case["axes"]]
        st["positions"] = pos.contiguous()
        if case["norm"]:
            st["qw"], st["kw"] = ((1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(io) for _ in "qk")
    elif op == "store":
        B, T = case["B"], case["T"]
        k, v = _rows(g, B * H, T, D)
        k, v = (x.view(B, H, T, D).transpose(1, 2).to(io) for x in (k, v))
        if case["packed"]:  # behind queries of four heads each, as the product makes them
            x = torch.cat([torch.zeros(B, T, 4 * H, D, dtype=io, device=DEV), k, v], 2)
            st["k"], st["v"] = x[:, :, 4 * H:5 * H], x[:, :, 5 * H:]
        else:
            st["k"], st["v"] = k.contiguous(), v.contiguous()
        low = case["held"] // 2 if case["ragged"] else case["held"]
        st["lens"] = torch.randint(low, case["held"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        low = (T + 1) // 2 if case["ragged"] else T
        st["counts"] = torch.randint(low, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        n = -(-(case["held"] + T) // TILE)
        st["table"] = (torch.randperm(B * H * n, generator=g, device=DEV) * (144 * D)).view(B, H, n)
        st["pool"] = torch.zeros(B * H * n * 144 * D, dtype=torch.uint8, device=DEV)
        st["k_out"], st["v_out"] = (torch.zeros(B, T, H, D, dtype=io, device=DEV) for _ in "kv")
    else:
        B = case.get("B", 1)
        most = case["len"] if op == "decode" else case["held"] + case["C"]
        n = -(-most // TILE)
        st["pool"], table = _paged(g, B * H, n, D)
        st["table"], st["n"] = table.view(B, H, n), n
        rows = (B, H * case["G"], D) if op == "decode" else (case["C"], H * case["G"], D)
        st["q"] = torch.randn(*rows, generator=g, device=DEV).to(io)
        if op == "decode":
            low = max(1, most // 4) if case["ragged"] else most
            st["lens"] = torch.randint(low, most + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
            if case["mass"]:
                st["mass"] = torch.rand(B, H, n, generator=g, device=DEV) * 10
    return st


# ---------------------------------------------------------------------------------------------------------------
# the operators in plain form

def _plain_rope(st):
    D, R, half = st["D"], st["rot"], st["rot"] // 2
    pos = st["positions"][torch.tensor(st["pair_axis"], device=DEV)].double()  # [pairs, tokens]
    angle = pos.transpose(0, 1) * torch.tensor(st["inv_freq"], dtype=torch.float64, device=DEV)
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)

    def one(x, w):
        y = x.float()
        if st["norm"]:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        r = y[..., :R]
        a, b = (r[..., 0::2], r[..., 1::2]) if st["adjacent"] else (r[..., :half], r[..., half:])
        c, d = a * cos - b * sin, a * sin + b * cos
        r = torch.stack([c, d], -1).flatten(-2) if st["adjacent"] else torch.cat([c, d], -1)
        y = torch.cat([r, y[..., R:]], -1)
        if st["hadamard"]:
            h = 1
            while h < D:
                z = y.unflatten(-1, (-1, 2, h))
                y = torch.stack([z[..., 0, :] + z[..., 1, :], z[..., 0, :] - z[..., 1, :]], -2).flatten(-3)
                h *= 2
            y = y / math.sqrt(D)
        return y.to(x.dtype)

    return {"q": one(st["q"], st.get("qw")), "k": one(st["k"], st.get("kw"))}


def _plain_store(st):
    B, T, n = st["B"], st["T"], st["table"].shape[2]
    t = torch.arange(T, device=DEV)
    there = t < st["counts"].view(B, 1)
    b = torch.arange(B, device=DEV).view(B, 1).expand(B, T)[there]
    at = (st["lens"].view(B, 1) + t)[there]
    for name, out in (("k", st["k_out"]), ("v", st["v_out"])):
        codes, s = _quantise(st[name])
        cache = torch.zeros(B, n * TILE, *codes.shape[2:], dtype=torch.int8, device=DEV)
        scales = torch.zeros(B, n * TILE, *s.shape[2:], dtype=torch.float16, device=DEV)
        cache[b, at], scales[b, at] = codes.to(torch.int8)[there], s.half()[there]
        x = cache[b, at].float() * scales[b, at].float().repeat_interleave(RUN, -1)
        out[there] = x.to(out.dtype)
    return {"k": st["k_out"], "v": st["v_out"]}


def _values(records, D):
    """Records [..., 144 D] -> K and V rows [..., 128, D] in 32 bits."""
    lead = records.shape[:-1]
    x = records.view(torch.int16).view(*lead, 4, 18 * D)
    wide = min(D, 128) // 4
    ku = x[..., :8 * D].unflatten(-1, (-1, RUN, wide)).transpose(-3, -2).reshape(*lead, TILE, D // 4)
    vu = x[..., 8 * D:16 * D].unflatten(-1, (D // 32, RUN, 8)).transpose(-3, -2).reshape(*lead, TILE, D // 4)
    ks = x[..., 16 * D:17 * D].contiguous().view(torch.float16).reshape(*lead, TILE, D // 32)
    vs = x[..., 17 * D:].contiguous().view(torch.float16).unflatten(-1, (D // 32, RUN))[..., _scale_place()]
    vs = vs.transpose(-2, -1).reshape(*lead, TILE, D // 32)

    def rows(u, s):
        u = u.int()
        c = torch.stack([u >> 6, u >> 10, u >> 2, (u >> 14 & 3) | (u & 3) << 2], -1) & 15
        return (c - 8).float().flatten(-2) * s.float().repeat_interleave(RUN, -1)

    return rows(ku, ks), rows(vu, vs)


def _plain_decode(st):
    D, H, G, n, B = st["D"], st["Hkv"], st["G"], st["n"], st["B"]
    k, v = _values(st["pool"].view(-1, 144 * D)[st["table"] // (144 * D)], D)
    k, v = k.view(B, H, n * TILE, D), v.view(B, H, n * TILE, D)
    seen = torch.arange(n * TILE, device=DEV) < st["lens"].view(B, 1)
    s = st["q"].float().view(B, H, G, D) @ k.transpose(-1, -2) * D ** -0.5
    s = s.masked_fill(~seen.view(B, 1, 1, -1), -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = {"out": (p @ v).view(B, H * G, D).to(st["q"].dtype)}
    if st["mass"] is not False:
        out["mass"] = st["mass"] + p.sum(2).view(B, H, n, TILE).sum(-1)
    return out


def _plain_prefill(st):
    D, H, G, n, C = st["D"], st["Hkv"], st["G"], st["n"], st["C"]
    k, v = _values(st["pool"].view(-1, 144 * D)[st["table"][0] // (144 * D)], D)
    total = st["held"] + C
    k, v = k.view(H, n * TILE, D)[:, :total], v.view(H, n * TILE, D)[:, :total]
    s = st["q"].float().view(C, H, G, D).permute(1, 2, 0, 3).reshape(H, G * C, D) @ k.transpose(-1, -2) * D ** -0.5
    late = torch.arange(total, device=DEV) > st["held"] + torch.arange(C, device=DEV).view(C, 1)
    s = s.view(H, G, C, total).masked_fill(late, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p.view(H, G * C, total) @ v).view(H, G, C, D) / p.sum(-1, keepdim=True)
    return {"out": o.permute(2, 0, 1, 3).reshape(C, H * G, D).to(st["q"].dtype)}


# ---------------------------------------------------------------------------------------------------------------
# the library's calls

def _library(st):
    if "kvarn" not in st:
        from kv_cache_quantization_token_gb300 import kvarn
        st["kvarn"] = kvarn
        if st["op"] != "rope":
            st["lay"] = kvarn.layout4(st["D"])
    return st["kvarn"]


def _own_rope(st):
    kvarn = _library(st)
    if "plan" not in st:
        st["plan"] = kvarn.rotary(st["rot"], inv_freq=st["inv_freq"], pair_axis=st["pair_axis"],
                                  pairing="adjacent" if st["adjacent"] else "halves")
        st["to"] = [torch.empty(x.shape, dtype=x.dtype, device=DEV) for x in (st["q"], st["k"])]
    q, k = kvarn.norm_rotate(st["q"], st["k"], st["positions"], st["plan"], q_weight=st.get("qw"),
                             k_weight=st.get("kw"), eps=EPS if st["norm"] else None, hadamard=st["hadamard"],
                             q_out=st["to"][0], k_out=st["to"][1])
    return {"q": q, "k": k}


def _own_store(st):
    kvarn = _library(st)
    kvarn.write_rows4(st["k"], st["v"], st["pool"], st["table"], st["lens"], st["lay"], counts=st["counts"])
    kvarn.read_rows4(st["pool"], st["table"], st["lens"], st["k_out"], st["v_out"], st["lay"], counts=st["counts"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_decode(st):
    kvarn = _library(st)
    if "ws" not in st:
        need = kvarn.decode4_workspace_bytes(st["B"], st["Hkv"] * st["G"], st["Hkv"], st["D"], st["n"])
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
        st["out"] = torch.empty_like(st["q"])
        st["mass_out"] = torch.empty_like(st["mass"]) if st["mass"] is not False else None
    weighed = st["mass"] is not False
    kvarn.decode_attention4(st["q"], st["pool"], st["table"], st["lens"], st["lay"],
                            mass_in=st["mass"] if weighed else None, mass_out=st["mass_out"], ws=st["ws"], out=st["out"])
    return {"out": st["out"], "mass": st["mass_out"]} if weighed else {"out": st["out"]}


def _own_prefill(st):
    kvarn = _library(st)
    if "ws" not in st:
        need = kvarn.prefill4_workspace_bytes(st["C"], st["n"], st["Hkv"] * st["G"], st["Hkv"], st["D"])
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
        st["out"] = torch.empty_like(st["q"])
    kvarn.prefill_attention4(st["q"], st["held"], st["pool"], st["table"][0], st["lay"], ws=st["ws"], out=st["out"])
    return {"out": st["out"]}


def run(state):
    op = state["op"]
    if own:
        return {"rope": _own_rope, "store": _own_store, "decode": _own_decode, "prefill": _own_prefill}[op](state)
    return {"rope": _plain_rope, "store": _plain_store, "decode": _plain_decode, "prefill": _plain_prefill}[op](state)


def work(case):
    op, D, H = case["op"], case["D"], case["Hkv"]
    size = torch.empty(0, dtype=IO[case["io"]]).element_size()
    if op == "rope":  # queries and keys in and out; a norm and a rotation, and log2 D sums of a transform
        elements = case["tokens"] * (case["G"] + 1) * H * D
        return {"bytes": 2 * elements * size + 8 * case["axes"] * case["tokens"],
                "flops": elements * (8 + (D.bit_length() if case["hadamard"] else 0))}
    if op == "store":  # rows in, codes and scales out; codes and scales in, rows out
        rows = case["B"] * case["T"] * (0.75 if case["ragged"] else 1.0) * H
        return {"bytes": int(rows * 2 * (2 * D * size + 1.125 * D)), "flops": int(rows * 2 * D * 6)}
    G = case["G"]
    if op == "decode":
        tokens = case["B"] * case["len"] * (5 / 8 if case["ragged"] else 1.0)  # a quarter of the most up to the most
        return {"bytes": int(tokens * H * 1.125 * D + 2 * case["B"] * H * G * D * size +
                             (8 * case["B"] * H * -(-case["len"] // TILE) if case["mass"] else 0)),
                "flops": int(4 * tokens * H * G * D)}
    C, held = case["C"], case["held"]
    return {"bytes": int(H * (held + C) * 1.125 * D) + 2 * C * H * G * D * size,
            "flops": 4 * (C * held + C * (C + 1) // 2) * H * G * D}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(pool, offset, D):
    """K and V of the records at `offset` [...], each value its code times its scale: [..., 128, D] in 64 bits."""
    t, c = torch.arange(TILE, device=DEV).view(TILE, 1), torch.arange(D, device=DEV)
    run, r = 18 * D * (t // 32), t % 32  # in 16-bit words
    wide = min(D, 128)
    at_k = run + (c // wide) * (RUN * wide // 4) + r * (wide // 4) + c % wide // 4
    at_v = run + 8 * D + (c // 32) * 256 + r * 8 + c % 32 // 4
    at_ks = run + 16 * D + r * (D // 32) + c // 32
    at_vs = run + 17 * D + (c // 32) * 32 + 8 * ((r % 8) // 2) + 2 * (r // 8) + r % 2
    words, halves = pool.view(torch.int16), pool.view(torch.float16)
    first = offset[..., None, None] // 2
    both = []
    for at, at_s in ((at_k, at_ks), (at_v, at_vs)):
        u = words[first + at].long() & 0xFFFF
        swapped = (u >> 8 | u << 8) & 0xFFFF
        place = torch.tensor([6, 10, 2, 6], device=DEV)[c % 4]
        code = (torch.where(c % 4 == 3, swapped, u) >> place) % 16 - 8
        both.append(code.double() * halves[first + at_s].double())
    return both


def _softmax_sum(q, k, v, hidden):
    s = torch.einsum("...qd,...kd->...qk", q, k) / math.sqrt(q.shape[-1])
    w = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
    return torch.einsum("...qk,...kd->...qd", w, v), w


def _exact_quantised(x):
    """The value that each element of x [..., D] becomes, by search: of all scales of eight significant bits the least
    that reaches a seventh of the group's largest magnitude, of all codes the nearest, of two the even one."""
    scales = torch.cat([torch.arange(256, dtype=torch.float64, device=DEV) * 2.0 ** -24] +
                       [torch.arange(128, 256, dtype=torch.float64, device=DEV) * 2.0 ** e for e in range(-23, 4)] +
                       [torch.tensor([2048.0], dtype=torch.float64, device=DEV)])
    y = x.double().unflatten(-1, (-1, RUN))
    s = scales[torch.searchsorted(7 * scales, y.abs().amax(-1)).clamp_min(1)].unsqueeze(-1)
    below = (y.abs() / s).floor()
    rest = y.abs() - (below + 0.5) * s
    code = below + ((rest > 0) | ((rest == 0) & (below % 2 == 1)))
    return (code * s).copysign(y).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    op, D, H = case["op"], case["D"], case["Hkv"]
    if op == "rope":
        R = case["rot"]
        i = torch.arange(R // 2, device=DEV)
        first, second = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + R // 2)
        f = torch.tensor(st["inv_freq"], dtype=torch.float64, device=DEV)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           st["positions"].double()[st["pair_axis"]].T * f)
        hada = torch.ones(1, 1, dtype=torch.float64, device=DEV)
        while hada.shape[0] < D:
            hada = torch.cat([torch.cat([hada, hada], 1), torch.cat([hada, -hada], 1)])
        out = {}
        for name in ("q", "k"):
            x = st[name].double()
            if case["norm"]:
                x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * st[name + "w"].double()
            z = torch.complex(x[..., first], x[..., second]) * turn.unsqueeze(1)
            x = x.clone()
            x[..., first], x[..., second] = z.real, z.imag
            out[name] = x @ hada / math.sqrt(D) if case["hadamard"] else x
        return out
    if op == "store":
        out = {}
        there = torch.arange(case["T"], device=DEV) < st["counts"].view(-1, 1)
        for name in ("k", "v"):
            out[name] = torch.where(there[..., None, None], _exact_quantised(st[name]), 0.0)
        return out
    G = case["G"]
    if op == "prefill":
        C, total = case["C"], case["held"] + case["C"]
        out = torch.empty(C, H * G, D, dtype=torch.float64, device=DEV)
        hidden = torch.arange(total, device=DEV) > (case["held"] + torch.arange(C, device=DEV)).view(C, 1)
        for h in range(H):
            k, v = (x.reshape(-1, D)[:total] for x in _exact_rows(st["pool"], st["table"][0, h], D))
            q = st["q"][:, h * G:(h + 1) * G].double().transpose(0, 1)
            out[:, h * G:(h + 1) * G] = _softmax_sum(q, k, v, hidden)[0].transpose(0, 1)
        return {"out": out}
    B = case["B"]
    out = torch.empty(B, H * G, D, dtype=torch.float64, device=DEV)
    mass = st["mass"].double().clone() if case["mass"] else None
    none = torch.zeros((), dtype=torch.bool, device=DEV)
    for b, length in enumerate(st["lens"].tolist()):
        n = -(-length // TILE)
        for h in range(H):
            k, v = (x.reshape(-1, D)[:length] for x in _exact_rows(st["pool"], st["table"][b, h, :n], D))
            o, p = _softmax_sum(st["q"][b, h * G:(h + 1) * G].double(), k, v, none)
            out[b, h * G:(h + 1) * G] = o
            if mass is not None:
                p = torch.nn.functional.pad(p.sum(0), (0, n * TILE - length))
                mass[b, h, :n] += p.view(n, TILE).sum(-1)
    return {"out": out, "mass": mass} if mass is not None else {"out": out}
