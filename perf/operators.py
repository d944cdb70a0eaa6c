"""The operators on a cache held in 8 bits: what each computes, in plain torch operations, and the calls that reach
the library's kernels.

  tile      raw K and V rows compressed to 8-bit tile records, and the records expanded to rows again
  decode    attention of one query token per sequence over records and the FP32 window, with or without the
            attention weight that each tile received
  prefill   causal attention of a chunk of query positions of one sequence over records and the FP32 window
  evict     the tiles of each KV head with the least accumulated weight leave the tile table

A record holds one 128-token tile of one KV head: K codes [16][D/64][8][64] (tokens in groups of 8, channels in
groups of 64), V codes [D/8][2][8][64] (channels in groups of 8, tokens in groups of 64), then the fp32 scales of the
eight 16-token groups of K and of V, then 64 zero bytes. `block` tokens (16 to 128) of a head share a scale.
"""
import math

import torch

own = False

TILE = 128
GROUPS = 8          # 16-token groups of a tile
FLOOR = 2.0 ** -100  # smallest scale
QMAX = {"i8": 127.0, "e4m3": 448.0}
IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


def _tile(name, code, D, block, units, stride=0):
    return {"name": name, "op": "tile", "code": code, "D": D, "block": block, "units": units, "stride": stride or D}


def _decode(name, code, io, D, block, B, G, Hkv, tiles, ragged, window, mass):
    return {"name": name, "op": "decode", "code": code, "io": io, "D": D, "block": block, "B": B, "G": G, "Hkv": Hkv,
            "tiles": tiles, "ragged": ragged, "window": window, "mass": mass}


def _prefill(name, code, io, D, block, G, Hkv, tiles, window, C):
    return {"name": name, "op": "prefill", "code": code, "io": io, "D": D, "block": block, "G": G, "Hkv": Hkv,
            "tiles": tiles, "window": window, "C": C}


def _evict(name, B, Hkv, max_tiles, keep, sinks, recent, ragged):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "max_tiles": max_tiles, "keep": keep, "sinks": sinks,
            "recent": recent, "ragged": ragged}


def listed():
    return [
        # one layer's promotion while decoding: the full tile of each of 8 KV heads
        _tile("tile_promote", "i8", 128, 64, 8),
        # the 32k-token caches of one layer of an 8B-like model, compressed in one launch
        _tile("tile_bulk", "e4m3", 128, 128, 2048),
        # one layer of a decode step soon after a short prompt, at full precision
        _decode("decode_short", "e4m3", "f32", 128, 16, 1, 2, 8, 3, False, 17, False),
        # one layer of an 8B-like decode step at 16k context
        _decode("decode_16k", "i8", "bf16", 128, 64, 1, 4, 8, 128, False, 77, False),
        # a few sequences of a small-head model whose tiles are weighed for eviction
        _decode("decode_weighed", "e4m3", "f32", 64, 32, 5, 3, 4, 250, True, 101, True),
        # batched serving with large heads: 32 ragged sequences of up to 32k tokens
        _decode("decode_batch_d256", "i8", "f16", 256, 128, 32, 4, 4, 256, True, 128, False),
        # a few drafted tokens checked at once
        _prefill("prefill_draft", "i8", "f32", 128, 64, 4, 8, 15, 40, 5),
        # an odd last chunk of a prompt, five query heads per KV head
        _prefill("prefill_odd", "e4m3", "f16", 64, 32, 5, 3, 37, 201, 301),
        # the last 512-token chunk of a 15,500-token prompt of an 8B-like model
        _prefill("prefill_15k", "e4m3", "bf16", 128, 128, 4, 8, 120, 140, 512),
        # the last 512-token chunk of an 8,192-token prompt with large heads, at full precision
        _prefill("prefill_d256", "i8", "f32", 256, 64, 4, 4, 63, 128, 512),
        # one sequence past its budget of tiles
        _evict("evict_one", 1, 8, 160, 128, 1, 8, False),
        # a batch of long ragged sequences cut back to half
        _evict("evict_batch", 48, 8, 2048, 1024, 4, 64, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tile", "decode", "decode", "prefill", "prefill", "evict"])
    code, D, block = rng.choice(["i8", "e4m3"]), rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    io = rng.choice(["f32", "f16", "bf16"])
    if op == "tile":
        stride = D if rng.random() < 0.6 else D + 4 * rng.randint(1, 20)
        case = _tile("", code, D, block, _log(rng, 1, 1900 * 128 // stride), stride)
    elif op == "decode":
        B, G, Hkv = _log(rng, 1, 32), rng.randint(1, 8), _log(rng, 1, 8)
        tiles = _log(rng, 1, max(2, min(900, 128 * 256 * 256 // (B * Hkv * D))))
        case = _decode("", code, io, D, block, B, G, Hkv, tiles, rng.random() < 0.5, rng.randint(0, 255),
                       rng.random() < 0.5)
    elif op == "prefill":
        G, Hkv, C = rng.randint(1, 8), _log(rng, 1, 8), _log(rng, 1, 700)
        tiles = _log(rng, 1, max(2, min(500, 120 * 512 * 32 * 128 // (C * G * Hkv * D))))
        case = _prefill("", code, io, D, block, G, Hkv, tiles, rng.randint(0, 383), C)
        case["C"] = min(C, TILE * case["tiles"] + case["window"])
    else:
        max_tiles = _log(rng, 2, 4000)
        keep = rng.randint(1, max_tiles)
        sinks = rng.randint(0, min(4, keep))
        case = _evict("", _log(rng, 1, 24), _log(rng, 1, 8), max_tiles, keep, sinks, rng.randint(0, keep - sinks),
                      rng.random() < 0.5)
    del case["name"]
    return case


# ---------------------------------------------------------------------------------------------------------------
# inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(g, heads, tokens, D):
    """K with a spread of channel scales and a few outlier channels, V with heavy-tailed token scales: [heads, tokens, D]."""
    ch = torch.randn(heads, 1, D, generator=g, device=DEV).exp()
    ch = torch.where(torch.rand(heads, 1, D, generator=g, device=DEV) < 0.02, ch * 20, ch)
    k = torch.randn(heads, tokens, D, generator=g, device=DEV) * ch
    t4 = torch.randn(heads, tokens, 1, generator=g, device=DEV) / (
        torch.randn(heads, tokens, 4, generator=g, device=DEV).square().mean(-1, keepdim=True) + 1e-3).sqrt()
    v = torch.randn(heads, tokens, D, generator=g, device=DEV) * t4.abs()
    return k, v


def _quantise(x, code, block):
    """x [..., 128, D] -> code bytes [..., 128, D] and a scale for each 16-token group [..., 8]."""
    amax = x.abs().unflatten(-2, (TILE // block, block)).amax((-1, -2))
    s = (amax.double() / QMAX[code]).float().clamp_min(FLOOR)
    s = s.repeat_interleave(block // 16, -1)
    # in 64 bits: the quotients next to the middle of two codes
    y = x.double() / s.double().repeat_interleave(16, -1).unsqueeze(-1)
    if code == "i8":
        return (y.round() + 128).to(torch.uint8), s
    step = (torch.frexp(y.abs().clamp_min(2.0 ** -6)).exponent.long() + 1019 << 52).view(torch.float64)  # 2^(e - 4)
    return ((y / step).round() * step).float().to(torch.float8_e4m3fn).view(torch.uint8), s


def _pack(kc, ks, vc, vs):
    """Code bytes [n, 128, D] and group scales [n, 8] of K and V -> records [n, 256 D + 128]."""
    n, _, D = kc.shape
    k = kc.view(n, 16, 8, D // 64, 64).transpose(2, 3).reshape(n, -1)
    v = vc.transpose(1, 2).reshape(n, D // 8, 8, 2, 64).transpose(2, 3).reshape(n, -1)
    scales = torch.cat([ks, vs, torch.zeros_like(ks), torch.zeros_like(ks)], 1)
    return torch.cat([k, v, scales.contiguous().view(torch.uint8)], 1)


def _records(g, code, block, D, heads, n):
    """Records [heads, n, bytes] of n consecutive tiles of each head."""
    k, v = _rows(g, heads, TILE * n, D)
    kc, ks = _quantise(k.view(heads * n, TILE, D), code, block)
    vc, vs = _quantise(v.view(heads * n, TILE, D), code, block)
    return _pack(kc, ks, vc, vs).view(heads, n, -1)


def _paged(g, records):
    """The records scattered over a pool, and the byte offset of each."""
    heads, n, rb = records.shape
    place = torch.randperm(heads * n, generator=g, device=DEV)
    pool = torch.empty(heads * n, rb, dtype=torch.uint8, device=DEV)
    pool[place] = records.view(heads * n, rb)
    return pool, (place * rb).view(heads, n)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "tile":
        D, n, stride = case["D"], case["units"], case["stride"]
        k, v = _rows(g, 1, TILE * n + 3, stride)  # the tiles start three rows in
        st["k"], st["v"] = k[0], v[0]
        st["src"] = torch.arange(n, device=DEV) * TILE + 3
        st["rb"] = 256 * D + 128
        st["dst"] = torch.randperm(n, generator=g, device=DEV) * st["rb"]
        st["pool"] = torch.zeros(n * st["rb"], dtype=torch.uint8, device=DEV)
        st["k_out"], st["v_out"] = torch.zeros_like(k[0]), torch.zeros_like(k[0])
    elif op == "evict":
        B, H, n = case["B"], case["Hkv"], case["max_tiles"]
        # weights with ties: a sum over a few steps, on a coarse grid for the seldom used tiles
        m = torch.randn(B, H, n, generator=g, device=DEV).exp()
        st["mass"] = torch.where(m < 1, (m * 16).round() / 16, m)
        st["table"] = (torch.randperm(B * H * n, generator=g, device=DEV) * 32896).view(B, H, n)
        low = max(1, n // 4) if case["ragged"] else n
        st["n_tiles"] = torch.randint(low, n + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    else:
        D, H, G, n = case["D"], case["Hkv"], case["G"], case["tiles"]
        B = case.get("B", 1)
        pool, table = _paged(g, _records(g, case["code"], case["block"], D, B * H, n))
        st["pool"], st["table"] = pool.view(-1), table.view(B, H, n)
        cap = max(TILE, -(-case["window"] // TILE) * TILE)
        wk, wv = _rows(g, B * H, cap, D)
        st["win_k"], st["win_v"] = wk.view(B, H, cap, D), wv.view(B, H, cap, D)
        if op == "decode":
            st["q"] = torch.randn(B, H * G, D, generator=g, device=DEV).to(IO[case["io"]])
            low = max(1, n // 4) if case["ragged"] else n
            st["n_tiles"] = torch.randint(low, n + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
            low = case["window"] // 2 if case["ragged"] else case["window"]
            st["win_len"] = torch.randint(low, case["window"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
            st["win_start"] = torch.randint(0, cap, (B,), generator=g, device=DEV, dtype=torch.int32)
            if case["mass"]:
                st["mass"] = torch.rand(B, H, n, generator=g, device=DEV) * 10
        else:
            st["q"] = torch.randn(case["C"], H * G, D, generator=g, device=DEV).to(IO[case["io"]])
            st["win_start"] = (seed * 37) % cap
    return st


# ---------------------------------------------------------------------------------------------------------------
# the operators in plain form

def _values(records, D, code):
    """Records [..., bytes] -> K and V rows [..., 128, D] in 32 bits."""
    lead = records.shape[:-1]
    k = records[..., :128 * D].view(*lead, 16, D // 64, 8, 64).transpose(-3, -2).reshape(*lead, TILE, D)
    v = records[..., 128 * D:256 * D].view(*lead, D // 8, 2, 8, 64).transpose(-3, -2).reshape(*lead, D, TILE)
    v = v.transpose(-1, -2)
    s = records[..., 256 * D:256 * D + 64].contiguous().view(torch.float32).view(*lead, 2, GROUPS)
    s = s.repeat_interleave(16, -1).unsqueeze(-1)
    if code == "i8":
        k, v = k.float() - 128, v.float() - 128
    else:
        k, v = (x.contiguous().view(torch.float8_e4m3fn).float() for x in (k, v))
    return k * s[..., 0, :, :], v * s[..., 1, :, :]


def _plain_tile(st):
    D, n = st["D"], st["units"]
    rows = st["src"].view(n, 1) + torch.arange(TILE, device=DEV)
    rb = st["rb"]
    pool = st["pool"].view(n, rb)
    kc, ks = _quantise(st["k"][rows, :D], st["code"], st["block"])
    vc, vs = _quantise(st["v"][rows, :D], st["code"], st["block"])
    pool[st["dst"] // rb] = _pack(kc, ks, vc, vs)
    k, v = _values(pool[st["dst"] // rb], D, st["code"])
    st["k_out"][rows, :D], st["v_out"][rows, :D] = k, v
    return {"k": st["k_out"], "v": st["v_out"]}


def _window(st, B):
    """Window rows in order of position, [B, H, cap, D]."""
    H, cap, D = st["win_k"].shape[1:]
    start = st["win_start"] if torch.is_tensor(st["win_start"]) else torch.full((B,), st["win_start"], device=DEV)
    slot = ((start.view(B, 1) + torch.arange(cap, device=DEV)) % cap).view(B, 1, cap, 1).expand(B, H, cap, D)
    return st["win_k"].gather(2, slot), st["win_v"].gather(2, slot)


def _plain_decode(st):
    D, H, G, n, B = st["D"], st["Hkv"], st["G"], st["tiles"], st["B"]
    rb = 256 * D + 128
    k, v = _values(st["pool"].view(-1, rb)[st["table"] // rb], D, st["code"])
    wk, wv = _window(st, B)
    cap = wk.shape[2]
    k = torch.cat([k.reshape(B, H, n * TILE, D), wk], 2)
    v = torch.cat([v.reshape(B, H, n * TILE, D), wv], 2)
    j = torch.arange(n * TILE + cap, device=DEV)
    seen = torch.where(j < n * TILE, j < TILE * st["n_tiles"].view(B, 1), j - n * TILE < st["win_len"].view(B, 1))
    s = st["q"].float().view(B, H, G, D) @ k.transpose(-1, -2) * D ** -0.5
    s = s.masked_fill(~seen.view(B, 1, 1, -1), -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = {"out": (p @ v).view(B, H * G, D).to(st["q"].dtype)}
    if st["mass"] is not False:
        out["mass"] = st["mass"] + p[..., :n * TILE].sum(2).view(B, H, n, TILE).sum(-1)
    return out


def _plain_prefill(st):
    D, H, G, n, C, w = st["D"], st["Hkv"], st["G"], st["tiles"], st["C"], st["window"]
    rb = 256 * D + 128
    k, v = _values(st["pool"].view(-1, rb)[st["table"][0] // rb], D, st["code"])
    wk, wv = _window(st, 1)
    k = torch.cat([k.reshape(H, n * TILE, D), wk[0, :, :w]], 1)
    v = torch.cat([v.reshape(H, n * TILE, D), wv[0, :, :w]], 1)
    total = n * TILE + w
    s = st["q"].float().view(C, H, G, D).permute(1, 2, 0, 3).reshape(H, G * C, D) @ k.transpose(-1, -2) * D ** -0.5
    late = torch.arange(total, device=DEV) > total - C + torch.arange(C, device=DEV).view(C, 1)
    s = s.view(H, G, C, total).masked_fill(late, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p.view(H, G * C, total) @ v).view(H, G, C, D) / p.sum(-1, keepdim=True)
    return {"out": o.permute(2, 0, 1, 3).reshape(C, H * G, D).to(st["q"].dtype)}


def _plain_evict(st):
    n_max = st["max_tiles"]
    i = torch.arange(n_max, device=DEV)
    n = st["n_tiles"].view(-1, 1, 1)
    middle = (i >= st["sinks"]) & (i < n - st["recent"])
    key = torch.where(st["mass"].isnan(), math.inf, st["mass"])
    order = torch.argsort(key, dim=-1, descending=True, stable=True)
    order = order.gather(-1, torch.argsort(middle.expand_as(key).gather(-1, order).byte(), dim=-1, descending=True,
                                               stable=True))
    rank = torch.empty_like(order).scatter_(-1, order, i.expand_as(order).contiguous())
    live = (i < n) & (n > st["keep"])
    gone = live & middle & (rank >= st["keep"] - st["sinks"] - st["recent"])
    stay = (i < n) & ~gone

    def front(flag, x, empty):  # the flagged entries in order, then `empty`
        o = torch.argsort((~flag).byte(), dim=-1, stable=True)
        return torch.where(i < flag.sum(-1, keepdim=True), x.gather(-1, o), empty)

    return {"table": front(stay, st["table"], -1), "mass": front(stay, st["mass"], 0.0),
            "n_tiles": st["n_tiles"].clamp_max(st["keep"]), "evicted": front(gone, st["table"], -1)}


# ---------------------------------------------------------------------------------------------------------------
# the library's calls

def _layout(st):
    if "lay" not in st:
        from kv_cache_quantization_token_gb300 import kvarn
        st["kvarn"], st["lay"] = kvarn, kvarn.layout8(st["D"], st["code"], st["block"])
    return st["kvarn"], st["lay"]


def _own_tile(st):
    kvarn, lay = _layout(st)
    kvarn.compress_tile8(st["k"], st["v"], st["src"], st["pool"], st["dst"], lay)
    kvarn.expand_tile8(st["pool"], st["dst"], st["k_out"], st["v_out"], st["src"], lay)
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_decode(st):
    kvarn, lay = _layout(st)
    if "ws" not in st:
        need = kvarn.decode8_workspace_bytes(st["B"], st["Hkv"] * st["G"], st["Hkv"], st["D"], st["tiles"],
                                             st["win_k"].shape[2])
        st["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        st["out"] = torch.empty_like(st["q"])
        st["mass_out"] = torch.empty_like(st["mass"]) if st["mass"] is not False else None
    weighed = st["mass"] is not False
    kvarn.decode_attention8(st["q"], st["pool"], st["table"], st["n_tiles"], st["win_k"], st["win_v"],
                            st["win_start"], st["win_len"], lay, mass_in=st["mass"] if weighed else None,
                            mass_out=st["mass_out"], ws=st["ws"], out=st["out"])
    return {"out": st["out"], "mass": st["mass_out"]} if weighed else {"out": st["out"]}


def _own_prefill(st):
    kvarn, lay = _layout(st)
    n, w, C = st["tiles"], st["window"], st["C"]
    if "ws" not in st:
        need = kvarn.prefill8_workspace_bytes(C, n, w, st["Hkv"] * st["G"], st["Hkv"], st["D"])
        st["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)
        st["out"] = torch.empty_like(st["q"])
    kvarn.prefill_attention8(st["q"], TILE * n + w - C, st["pool"], st["table"][0], n, st["win_k"][0],
                             st["win_v"][0], st["win_start"], w, lay, ws=st["ws"], out=st["out"])
    return {"out": st["out"]}


def _own_evict(st):
    from kv_cache_quantization_token_gb300 import kvarn
    if "to" not in st:
        st["to"] = (torch.empty_like(st["table"]), torch.empty_like(st["mass"]), torch.empty_like(st["n_tiles"]),
                    torch.empty_like(st["table"]))
    table, mass, n, evicted = st["to"]
    kvarn.evict_tiles(st["table"], st["mass"], st["n_tiles"], st["keep"], sinks=st["sinks"], recent=st["recent"],
                      table_out=table, mass_out=mass, n_tiles_out=n, evicted=evicted)
    return {"table": table, "mass": mass, "n_tiles": n, "evicted": evicted}


def run(state):
    op = state["op"]
    if own:
        return {"tile": _own_tile, "decode": _own_decode, "prefill": _own_prefill, "evict": _own_evict}[op](state)
    return {"tile": _plain_tile, "decode": _plain_decode, "prefill": _plain_prefill, "evict": _plain_evict}[op](state)


def work(case):
    op = case["op"]
    if op == "evict":  # weights and offsets in; weights, offsets and the evicted offsets out
        return {"bytes": case["B"] * case["Hkv"] * case["max_tiles"] * 32, "flops": 0}
    D = case["D"]
    rec = 256 * D + 64
    if op == "tile":  # rows in, records out; records in, rows out
        return {"bytes": case["units"] * 2 * (2 * TILE * D * 4 + rec), "flops": case["units"] * 2 * TILE * D * 4}
    H, G, n, w = case["Hkv"], case["G"], case["tiles"], case["window"]
    size = torch.empty(0, dtype=IO[case["io"]]).element_size()
    if op == "decode":
        mean = 5 / 8 if case["ragged"] else 1.0  # tiles are drawn from a quarter of the most up to the most
        tiles, win = case["B"] * H * n * mean, case["B"] * H * w * (3 / 4 if case["ragged"] else 1.0)
        return {"bytes": int(tiles * rec + win * 2 * D * 4 + 2 * case["B"] * H * G * D * size +
                             (8 * case["B"] * H * n if case["mass"] else 0)),
                "flops": int(4 * (tiles * TILE + win) * G * D)}
    C = case["C"]
    seen = C * (TILE * n + w) - C * (C - 1) // 2
    return {"bytes": H * (n * rec + w * 2 * D * 4) + 2 * C * H * G * D * size, "flops": 4 * seen * H * G * D}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rows(pool, offset, D, code):
    """K and V of the records at `offset` [...], each value its code times its scale: [..., 128, D] in 64 bits."""
    t, c = torch.arange(TILE, device=DEV).view(TILE, 1), torch.arange(D, device=DEV)
    at_k = (t // 8) * (8 * D) + (c // 64) * 512 + (t % 8) * 64 + c % 64
    at_v = 128 * D + (c // 8) * 1024 + (t // 64) * 512 + (c % 8) * 64 + t % 64
    words = pool.view(torch.float32)
    both = []
    for at, field in ((at_k, 0), (at_v, 8)):
        byte = pool[offset[..., None, None] + at]
        value = byte.double() - 128 if code == "i8" else byte.view(torch.float8_e4m3fn).double()
        both.append(value * words[offset[..., None, None] // 4 + 64 * D + field + t // 16].double())
    return both


def _softmax_sum(q, k, v, hidden):
    s = torch.einsum("...qd,...kd->...qk", q, k) / math.sqrt(q.shape[-1])
    w = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
    return torch.einsum("...qk,...kd->...qd", w, v), w


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        return None
    D, code = case["D"], case["code"]
    if op == "tile":
        out = {}
        for name in ("k", "v"):
            full = torch.zeros_like(st[name], dtype=torch.float64)
            x = st[name][3:, :D].double().view(-1, case["block"], D)
            s = (x.abs().amax((1, 2), keepdim=True) / torch.tensor(QMAX[code], device=DEV).double()).clamp_min(FLOOR)
            s = s.float().double()  # the scale is stored in 32 bits
            y = x / s
            if code == "i8":
                y = y.round()
            else:  # the nearest of the format's values, of two the one with the even code
                values = torch.arange(127, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
                middles = (values[1:] + values[:-1]) / 2
                at = torch.bucketize(y.abs(), middles)
                tie = y.abs() == middles[at.clamp_max(125)]
                y = values[at + (tie & (at % 2 == 1))].copysign(y)
            full[3:, :D] = (y * s).view(-1, D)
            out[name] = full
        return out
    H, G, n, w = case["Hkv"], case["G"], case["tiles"], case["window"]
    B, cap = case.get("B", 1), st["win_k"].shape[2]
    if op == "prefill":
        C, start = case["C"], st["win_start"]
        out = torch.empty(C, H * G, D, dtype=torch.float64, device=DEV)
        slots = (start + torch.arange(w, device=DEV)) % cap
        pos = torch.arange(TILE * n + w, device=DEV)
        hidden = pos > (TILE * n + w - C + torch.arange(C, device=DEV)).view(C, 1)
        for h in range(H):
            k, v = _exact_rows(st["pool"], st["table"][0, h], D, code)
            k = torch.cat([k.reshape(-1, D), st["win_k"][0, h, slots].double()])
            v = torch.cat([v.reshape(-1, D), st["win_v"][0, h, slots].double()])
            q = st["q"][:, h * G:(h + 1) * G].double().transpose(0, 1)
            out[:, h * G:(h + 1) * G] = _softmax_sum(q, k, v, hidden)[0].transpose(0, 1)
        return {"out": out}
    out = torch.empty(B, H * G, D, dtype=torch.float64, device=DEV)
    mass = st["mass"].double().clone() if case["mass"] else None
    tiles, wins, starts = st["n_tiles"].tolist(), st["win_len"].tolist(), st["win_start"].tolist()
    for b in range(B):
        slots = (starts[b] + torch.arange(wins[b], device=DEV)) % cap
        k, v = _exact_rows(st["pool"], st["table"][b, :, :tiles[b]], D, code)
        k = torch.cat([k.reshape(H, -1, D), st["win_k"][b][:, slots].double()], 1)
        v = torch.cat([v.reshape(H, -1, D), st["win_v"][b][:, slots].double()], 1)
        o, p = _softmax_sum(st["q"][b].double().view(H, G, D), k, v, torch.zeros((), dtype=torch.bool, device=DEV))
        out[b] = o.reshape(H * G, D)
        if mass is not None:
            mass[b, :, :tiles[b]] += p[..., :TILE * tiles[b]].sum(1).view(H, tiles[b], TILE).sum(-1)
    return {"out": out, "mass": mass} if mass is not None else {"out": out}
