"""Measured cases of attention over an 8-bit cache and of what stands between
it and the shared linear layers:

  rope       norms of each query and key head with the position rotation
  append     new keys and values quantized into a paged 8-bit cache that has
             one scale for each page and head
  read       keys and values of sequences read back out of it
  attention  the new tokens' queries over their sequences' cached tokens

run() computes them with elementary torch operations in 32 bits (own =
False), or through the library's entry points (own = True).  exact() gives
the same from the definitions in 64 bits.

Sizes: the heads of the dense layers of hidden size 2048, 4096 and 5120 that
the workloads name (16, 32 and 64 query heads, 8 key heads, 128 wide), and
heads of 64 and 256, which the same code has to serve.

A page holds 16, 32, 64 or 128 tokens of one sequence.  Its codes are stored
in tiles of 16 tokens, in the order in which a matrix core takes them:

  keys    [pages][heads][page / 16][D / 64][4: g][16: t][16: i]
          token 16 tile + t, channel 64 j + 16 g + i
  values  [pages][heads][page / 16][D / 64][4: g][16: c][4: b][4: t]
          token 16 tile + 4 g + t, channel 64 j + 16 b + c
"""
import math
import random

import torch

own = False

FP8, INT8 = 0, 1
QMAX = {FP8: 448.0, INT8: 127.0}


def _rope(name, T, Hq, Hk, D, rotary, interleaved=False, dtype="bf16", out="bf16", positions=8192, norm=True):
    c = {"op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rotary": rotary, "interleaved": interleaved, "dtype": dtype,
         "out": out, "positions": positions, "norm": norm}
    return dict(c, name=name) if name else c


def _cached(op, name, fmt, B, new, ragged, shortest, longest, Hk, D, page, dtype, **more):
    """B sequences of shortest to longest tokens, the last `new` of each (0 to
    `new` where ragged) being the call's own."""
    c = {"op": op, "fmt": fmt, "B": B, "new": new, "ragged": ragged, "shortest": shortest, "longest": longest, "Hk": Hk,
         "D": D, "page": page, "dtype": dtype, **more}
    return dict(c, name=name) if name else c


def _attention(name, fmt, B, new, ragged, shortest, longest, Hq, Hk, D, page, dtype="bf16", window=0, causal=True):
    return _cached("attention", name, fmt, B, new, ragged, shortest, longest, Hk, D, page, dtype, Hq=Hq, window=window,
                   causal=causal)


def listed():
    return [
        # one token of one request: latency of the call
        _rope("rope_1_token", 1, 16, 8, 128, 128),
        # a decode batch of a narrower model, fp32 projections, half of each head rotated, in neighbouring pairs
        _rope("rope_61_tokens_interleaved", 61, 32, 4, 64, 32, interleaved=True, dtype="f32"),
        # a prompt of the widest layer, far positions
        _rope("rope_8192_tokens", 8192, 64, 8, 128, 128, positions=131072),
        # a decode batch: one token each into the open page of its sequence
        _cached("append", "append_32_tokens", FP8, 32, 1, False, 1, 4096, 8, 128, 64, "bf16"),
        # drafts of up to 5 tokens that verification keeps, small pages, fp32 projections
        _cached("append", "append_drafts_237_int8", INT8, 237, 5, True, 5, 900, 4, 64, 16, "f32"),
        # prompts of several requests
        _cached("append", "append_prompts", FP8, 5, 4001, True, 500, 9000, 8, 128, 128, "bf16"),
        # one request's cache read back in 32 bits, and those of a batch on their way to another worker
        _cached("read", "read_1_sequence_int8", INT8, 1, 1000, False, 1000, 1000, 8, 128, 16, "f32"),
        _cached("read", "read_16_sequences", FP8, 16, 5000, True, 100, 6000, 8, 128, 64, "bf16"),
        # one token of one short request: latency of the call
        _attention("attention_1_token", FP8, 1, 1, False, 61, 61, 16, 8, 128, 16),
        # a decode batch of ragged contexts on the widest layer: what serving does most
        _attention("attention_64_tokens", FP8, 64, 1, False, 300, 16384, 64, 8, 128, 64),
        # one request with a very long context, the sum kept in 32 bits
        _attention("attention_131072_context_int8", INT8, 1, 1, False, 131071, 131071, 32, 8, 128, 128, dtype="f32"),
        # prompts' pieces over what is cached of them already
        _attention("attention_prompts", FP8, 3, 1500, True, 1500, 8192, 32, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attention", "attention", "attention"])
    D = rng.choice([64, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        return _rope(None, _log(rng, 1, 8192 * 64 * 128 // ((4 + 4 * Hk) * D * 4)), Hk * rng.randint(1, 8), Hk, D,
                     rng.choice([D, D, D // 16 * 8]), rng.random() < 0.4, rng.choice(["bf16", "f32"]),
                     rng.choice(["bf16", "bf16", "f32"]), _log(rng, 100, 131072), rng.random() < 0.8)
    fmt, page = rng.choice([FP8, INT8]), rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("append", "read"):
        new = rng.choice([1, _log(rng, 1, 64), _log(rng, 64, 4000)])
        B = _log(rng, 1, max(1, min(256, 8000 * 128 // (new * D))))
        longest = new + _log(rng, 1, 4000)
        return _cached(op, None, fmt, B, new, rng.random() < 0.5, min(longest, new + rng.randint(0, 100)), longest, Hk, D, page,
                       dtype)
    group = rng.choice([1, 2, 4, 5, 8, 16])
    if rng.random() < 0.65:      # decode, and drafts to verify
        B, new = _log(rng, 1, 128), rng.choice([1, 1, 1, rng.randint(2, 8)])
        longest = _log(rng, 16, max(32, min(131072, 16384 * 64 * 8 * 128 // (2 * B * Hk * D))))
        shortest = max(1, longest // rng.choice([1, 4, 100]))
    else:                        # pieces of prompts
        B, new = rng.randint(1, 4), _log(rng, 30, 700)
        longest = new + _log(rng, 1, 3000)
        shortest = new
        group = min(group, 8)
    return _attention(None, fmt, B, new, new > 1 and rng.random() < 0.5, shortest, max(longest, shortest, new), Hk * group, Hk,
                      D, page, dtype, rng.choice([0, 0, 0, _log(rng, 16, 4096)]), rng.random() < 0.9)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _torch(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _lengths(case):
    """(new tokens, length with them) of each sequence: the same for every seed."""
    rng = random.Random(case["B"] * 1000003 + case["longest"] * 101 + case["new"])
    new = [case["new"] if i == 0 or not case["ragged"] else rng.randint(0, case["new"]) for i in range(case["B"])]
    longs = [case["longest"] if i == 0 else _log(rng, case["shortest"], case["longest"]) for i in range(case["B"])]
    return new, [max(n, l) for n, l in zip(new, longs)]


def _code_dtype(fmt):
    return torch.int8 if fmt == INT8 else torch.float8_e4m3fn


def _outliers(g, D):
    """Some channels of keys are much larger than the others."""
    f = torch.ones(D, device="cuda")
    f[torch.randint(0, D, (max(1, D // 40),), generator=g, device="cuda")] = 6.0
    return f


def _fill(g, s, factor):
    """A pool of pages of random tokens, each page quantized with its scale: (codes in tiles, scales)."""
    P, H, D, page, fmt = s["pages"], s["Hk"], s["D"], s["page"], s["fmt"]
    x = torch.randn(P, H, page, D, generator=g, device="cuda") * factor
    scale = x.abs().amax((2, 3)) / torch.full((), QMAX[fmt], device="cuda")
    x = x / scale[:, :, None, None]
    return (x.round() if fmt == INT8 else x).to(_code_dtype(fmt)), scale


def _key_tiles(x):
    P, H, page, D = x.shape
    return x.view(P, H, page // 16, 16, D // 64, 4, 16).permute(0, 1, 2, 4, 5, 3, 6).contiguous()


def _value_tiles(x):
    P, H, page, D = x.shape
    return x.view(P, H, page // 16, 4, 4, D // 64, 4, 16).permute(0, 1, 2, 5, 3, 7, 6, 4).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dev = {"device": "cuda"}
    i32 = {"dtype": torch.int32, "device": "cuda"}
    if case["op"] == "rope":
        T, Hq, Hk, D, R = case["T"], case["Hq"], case["Hk"], case["D"], case["rotary"]
        qkv = _normal(g, T, (Hq + 2 * Hk) * D, dtype=_torch(case["dtype"]))     # as the shared projection writes it
        s["qkv"], s["q"], s["k"] = qkv, qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hk) * D]
        s["q_norm"], s["k_norm"] = (1 + _normal(g, D, std=0.2) if case["norm"] else None for _ in range(2))
        turn = 1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
        angle = torch.arange(case["positions"], dtype=torch.float64)[:, None] * turn
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        s["at"] = torch.randint(0, case["positions"], (T,), generator=g, device="cuda").to(torch.int32)
        s["q_out"] = torch.empty(T, Hq * D, dtype=_torch(case["out"]), **dev)
        s["k_out"] = torch.empty(T, Hk * D, dtype=_torch(case["out"]), **dev)
        return s
    new, lengths = _lengths(case)
    B, T, D, H, page = case["B"], sum(new), case["D"], case["Hk"], case["page"]
    s["T"] = T
    held = [-(-n // page) for n in lengths]
    s["width"] = max(held) + 1
    s["pages"] = sum(held) + 3
    table = torch.full((B, s["width"]), -1, dtype=torch.int64)
    used = torch.randperm(s["pages"], generator=torch.Generator().manual_seed(int(seed)))[:sum(held)]
    table[torch.arange(s["width"])[None, :] < torch.tensor(held)[:, None]] = used
    s["table"] = table.to(**i32)
    s["offsets"] = torch.tensor([sum(new[:i]) for i in range(B + 1)], **i32)
    s["lengths"] = torch.tensor(lengths, **i32)
    s["most"], s["most_new"] = max(lengths), max(new)
    s["factor"] = _outliers(g, D)
    codes, s["ks"] = _fill(g, s, s["factor"])
    s["kc"] = _key_tiles(codes)
    codes, s["vs"] = _fill(g, s, 0.5)
    s["vc"] = _value_tiles(codes)
    del codes
    dtype = _torch(case["dtype"])
    if case["op"] == "append":
        qkv = torch.randn(T, 4, H, D, generator=g, **dev)                       # queries (twice as many), keys, values
        qkv[:, 2] *= s["factor"]
        qkv[:, 3] *= 0.5
        # a token in eight is larger than what its page holds so far
        qkv *= torch.where(torch.rand(T, 1, 1, 1, generator=g, **dev) < 0.125, 1.7, 1.0)
        s["qkv"] = qkv.to(dtype).view(T, 4 * H * D)
        s["k"], s["v"] = s["qkv"][:, 2 * H * D:3 * H * D], s["qkv"][:, 3 * H * D:]
    elif case["op"] == "read":
        s["k"], s["v"] = (torch.empty(T, H * D, dtype=dtype, **dev) for _ in range(2))
    else:
        s["scale"] = D ** -0.5
        s["q"] = (_normal(g, T, case["Hq"], D) / s["factor"].sqrt()).to(torch.bfloat16).view(T, case["Hq"] * D)
        s["y"] = torch.empty(T, case["Hq"] * D, dtype=dtype, **dev)
    return s


# -------------------------------------------------------------- plain forms

def _plain_rope(s):
    R, D = s["rotary"], s["D"]
    table = s["cos_sin"][s["at"].long()]
    cos, sin = table[:, None, :R // 2], table[:, None, R // 2:]

    def turn(x, weight):
        x = x.reshape(s["T"], -1, D).float()
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(2, keepdim=True) + 1e-6) * weight
        a, b = (x[:, :, 0:R:2], x[:, :, 1:R:2]) if s["interleaved"] else (x[:, :, :R // 2], x[:, :, R // 2:R])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], 3).flatten(2) if s["interleaved"] else torch.cat([a, b], 2)
        return torch.cat([turned, x[:, :, R:]], 2).to(s["q_out"].dtype).flatten(1)

    return {"q": turn(s["q"], s["q_norm"]), "k": turn(s["k"], s["k_norm"])}


def _places(s):
    """Sequence and position of each of the call's tokens."""
    t = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(s["offsets"][1:].long(), t, right=True)
    start = s["lengths"].long() - (s["offsets"][1:] - s["offsets"][:-1]).long()
    return seq, start[seq] + t - s["offsets"].long()[seq], start


def _rows_of_keys(tiles):
    P, H, n, J = tiles.shape[:4]
    return tiles.permute(0, 1, 2, 5, 3, 4, 6).reshape(P, H, n * 16, J * 64)


def _rows_of_values(tiles):
    P, H, n, J = tiles.shape[:4]
    return tiles.permute(0, 1, 2, 4, 7, 3, 6, 5).reshape(P, H, n * 16, J * 64)


def _plain_append(s):
    H, D, page, fmt = s["Hk"], s["D"], s["page"], s["fmt"]
    seq, at, start = _places(s)
    where = s["table"].long()[seq, at // page]
    touched, which = torch.unique(where, return_inverse=True)
    # tokens that a touched page held before: those of its sequence before the call's first
    before = (start[seq] - at // page * page).clamp(0, page)
    held = torch.zeros(len(touched), dtype=torch.long, device="cuda").scatter_(0, which, before)
    old = torch.arange(page, device="cuda")[None, :] < held[:, None]
    qmax = torch.full((), QMAX[fmt], device="cuda")      # a tensor: dividing by it is one division

    def codes(x, scale):
        x = torch.where(scale == 0, 0.0, x / scale)
        return x.round().clamp(-127, 127).to(torch.int8) if fmt == INT8 else x.clamp(-448, 448).to(torch.float8_e4m3fn)

    def put(x, tiles, scales, rows_of, tiles_of):
        x = x.reshape(s["T"], H, D).float()
        most = torch.zeros(len(touched), H, device="cuda")
        most = most.scatter_reduce_(0, which[:, None].expand(-1, H), x.abs().amax(2), "amax")
        was = torch.where(held[:, None] > 0, scales[touched], 0.0)
        now = torch.maximum(was, most / qmax)
        rows = rows_of(tiles.view(torch.uint8)[touched]).view(tiles.dtype)
        again = codes(rows.float() * was[:, :, None, None], now[:, :, None, None])
        grown = (old[:, None, :] & (now > was)[:, :, None])[:, :, :, None]
        rows = torch.where(grown, again.view(torch.uint8), rows.view(torch.uint8))
        rows[which, :, at % page] = codes(x, now[which][:, :, None]).view(torch.uint8)
        tiles.view(torch.uint8)[touched] = tiles_of(rows)
        scales[touched] = now

    put(s["k"], s["kc"], s["ks"], _rows_of_keys, _key_tiles)
    put(s["v"], s["vc"], s["vs"], _rows_of_values, _value_tiles)
    return {"k": s["kc"], "v": s["vc"], "k_scales": s["ks"], "v_scales": s["vs"]}


def _plain_read(s):
    seq, at, _ = _places(s)
    where = s["table"].long()[seq, at // s["page"]]

    def get(tiles, scales, rows_of, out):
        rows = rows_of(tiles.view(torch.uint8)).view(tiles.dtype)
        x = rows.view(torch.uint8)[where, :, at % s["page"]].view(tiles.dtype).float() * scales[where][:, :, None]
        return x.to(out.dtype).flatten(1)

    return {"k": get(s["kc"], s["ks"], _rows_of_keys, s["k"]), "v": get(s["vc"], s["vs"], _rows_of_values, s["v"])}


def _plain_attention(s):
    """All sequences at once, padded to the longest."""
    B, Hq, Hk, D, page = s["B"], s["Hq"], s["Hk"], s["D"], s["page"]
    G, N, L = Hq // Hk, s["most_new"], -(-s["most"] // page) * page
    first, new = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    table = s["table"].long()[:, :L // page].clamp_min(0)

    def rows(tiles, scales, rows_of):
        x = rows_of(tiles.view(torch.uint8)[table.flatten()]).view(tiles.dtype).float()
        x = x * scales[table.flatten()][:, :, None, None]
        return x.view(B, L // page, Hk, page, D).permute(0, 2, 1, 3, 4).reshape(B * Hk, L, D)

    step = torch.arange(N, device="cuda")
    mine = step[None, :] < new[:, None]                                                         # [B, N]
    token = torch.where(mine, first[:, None] + step[None, :], 0)
    q = s["q"].float().view(s["T"], Hk, G, D)[token].permute(0, 2, 1, 3, 4).reshape(B * Hk, N * G, D)
    k = rows(s["kc"], s["ks"], _rows_of_keys)
    score = torch.bmm(q, k.transpose(1, 2).contiguous()).view(B, Hk, N, G, L) * s["scale"]
    del k
    length = s["lengths"].long()[:, None, None]
    at = torch.arange(L, device="cuda")[None, None, :]
    own_at = length - new[:, None, None] + step[None, :, None]
    seen = (at < length) & (at <= own_at if s["causal"] else True)
    if s["window"]:
        seen = seen & (at > own_at - s["window"])
    score = score.masked_fill(~seen[:, None, :, None, :], -math.inf)
    p = torch.exp(score - score.amax(4, keepdim=True).clamp_min(-1e30))
    del score
    total = p.sum(4, keepdim=True)
    v = rows(s["vc"], s["vs"], _rows_of_values)
    y = torch.bmm(p.view(B * Hk, N * G, L), v).view(B, Hk, N, G, D)
    y = torch.where(total > 0, y / total, 0.0)
    y = y.permute(0, 2, 1, 3, 4).reshape(B, N, Hq * D)[mine]
    return {"y": y.to(s["y"].dtype)}


# ------------------------------------------------------------- entry points

_handles = {}


def _workspace(nbytes):
    """One workspace for the stream, as large as the largest call so far needs."""
    ws = _handles.get("workspace")
    if ws is None or ws.numel() < nbytes:
        ws = _handles["workspace"] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device="cuda")
    return ws


def _type(q, dtype):
    return q.QLIN_OUT_F32_ACC if dtype == torch.float32 else q.QLIN_OUT_BF16


def _own(s):
    import skinny_bit_gemm_amd as q
    if s["op"] == "rope":
        if "rope" not in s:      # a program keeps one for each of its models
            s["rope"] = q.make_rope(s["Hq"], s["Hk"], s["D"], s["rotary"], s["positions"], int(s["interleaved"]), 1e-6)
        ld, D = s["qkv"].stride(0), s["D"]
        q.qlin_norm_rope(s["rope"], s["T"], s["q"], ld, s["k"], ld, _type(q, s["qkv"].dtype), s["q_norm"], s["k_norm"],
                         s["cos_sin"], s["at"], s["q_out"], s["Hq"] * D, s["k_out"], s["Hk"] * D, _type(q, s["q_out"].dtype))
        return {"q": s["q_out"], "k": s["k_out"]}
    if "cache" not in s:         # one cache for each layer, one description of a step's sequences
        s["cache"] = q.make_cache(s["fmt"], s["Hk"], s["D"], s["page"], s["pages"], s["kc"], s["vc"], s["ks"], s["vs"])
        s["sequences"] = q.make_sequences(s["B"], s["T"], s["offsets"], s["lengths"], s["table"], s["width"], s["most"])
    cache, sequences = s["cache"], s["sequences"]
    if s["op"] == "append":
        ld = s["qkv"].stride(0)
        q.qlin_cache_append(cache, sequences, s["k"], ld, s["v"], ld, _type(q, s["qkv"].dtype))
        return {"k": s["kc"], "v": s["vc"], "k_scales": s["ks"], "v_scales": s["vs"]}
    ld = s["Hk"] * s["D"]
    if s["op"] == "read":
        q.qlin_cache_read(cache, sequences, s["k"], ld, s["v"], ld, _type(q, s["k"].dtype))
        return {"k": s["k"], "v": s["v"]}
    if "attention" not in s:
        s["attention"] = q.make_attention(s["Hq"], s["scale"], int(s["causal"]), s["window"])
    a, ld = s["attention"], s["Hq"] * s["D"]
    q.qlin_cache_attention(a, cache, sequences, s["q"], ld, s["y"], ld, _type(q, s["y"].dtype),
                           _workspace(q.qlin_cache_attention_workspace_bytes(a, cache, sequences)))
    return {"y": s["y"]}


_PLAIN = {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "attention": _plain_attention}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work

def _pairs(case):
    """(query, cached token) pairs, and the cached tokens that any query sees."""
    pairs = seen = 0
    for n, length in zip(*_lengths(case)):
        low = length
        for i in range(n):
            at = length - n + i
            last = at + 1 if case["causal"] else length
            first = max(0, at - case["window"] + 1) if case["window"] else 0
            pairs += last - first
            low = min(low, first)
        seen += length - low if n else 0
    return pairs, seen


def work(case):
    D, Hk = case["D"], case["Hk"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        T, heads, out = case["T"], case["Hq"] + Hk, 4 if case["out"] == "f32" else 2
        rows = min(T, case["positions"])
        return {"bytes": T * heads * D * (size + out) + 4 * rows * case["rotary"] + 4 * T, "flops": 8 * T * heads * D}
    new, lengths = _lengths(case)
    T = sum(new)
    if case["op"] in ("append", "read"):
        pages = sum(-(-l // case["page"]) - (l - n) // case["page"] for n, l in zip(new, lengths) if n)
        return {"bytes": 2 * T * Hk * D * (size + 1) + 8 * pages * Hk + 8 * case["B"], "flops": 4 * T * Hk * D}
    pairs, seen = _pairs(case)
    return {"bytes": T * case["Hq"] * D * (2 + size) + 2 * seen * Hk * D + 8 * Hk * seen / case["page"] + 8 * case["B"],
            "flops": 4 * pairs * case["Hq"] * D}


# -------------------------------------------------------------------- exact

def _exact_rope(s):
    """As a product of complex numbers."""
    D, R = s["D"], s["rotary"]
    table = s["cos_sin"].double()[s["at"].long()]
    by = torch.complex(table[:, :R // 2].contiguous(), table[:, R // 2:].contiguous())[:, None]

    def turn(x, weight):
        x = x.double().reshape(s["T"], -1, D)
        if weight is not None:
            x = x * torch.rsqrt(x.pow(2).sum(2, keepdim=True) / D + 1e-6) * weight.double()
        pairs = x[:, :, :R].reshape(s["T"], -1, R // 2, 2) if s["interleaved"] else \
            x[:, :, :R].reshape(s["T"], -1, 2, R // 2).transpose(2, 3)
        z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * by)
        z = z.flatten(2) if s["interleaved"] else z.transpose(2, 3).flatten(2)
        return torch.cat([z, x[:, :, R:]], 2).flatten(1)

    return {"q": turn(s["q"], s["q_norm"]), "k": turn(s["k"], s["k_norm"])}


def _token_index(page, D, values):
    """Where (token, channel) of a page and head lies among its codes."""
    t, d = torch.arange(page, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    block = (t // 16) * (D // 64) + d // 64
    if values:
        return 1024 * block + 256 * (t % 16 // 4) + 16 * (d % 16) + 4 * (d % 64 // 16) + t % 4
    return 1024 * block + 256 * (d % 64 // 16) + 16 * (t % 16) + d % 16


def _exact_append(s):
    """Sequence by sequence and page by page; codes before their rounding."""
    H, D, page, fmt = s["Hk"], s["D"], s["page"], s["fmt"]
    table, offsets, lengths = s["table"].tolist(), s["offsets"].tolist(), s["lengths"].tolist()
    found = {}
    for name, x, values in (("k", s["k"], False), ("v", s["v"], True)):
        codes = s[name + "c"].float().double().view(s["pages"], H, page * D)
        scales = s[name + "s"].double().clone()
        index = _token_index(page, D, values)
        x = x.double().reshape(s["T"], H, D)
        for b in range(s["B"]):
            n = offsets[b + 1] - offsets[b]
            start = lengths[b] - n
            for c in range(start // page, -(-lengths[b] // page) if n else 0):
                lo, hi = max(start, c * page), min(lengths[b], (c + 1) * page)
                rows = x[offsets[b] + lo - start:offsets[b] + hi - start]
                p, had = table[b][c], lo - c * page
                was = scales[p].clone() if had else torch.zeros(H, dtype=torch.float64, device="cuda")
                now = torch.maximum(was, rows.abs().amax((0, 2)) / QMAX[fmt])
                scales[p] = now
                if had:
                    old = index[:had].flatten()
                    codes[p][:, old] *= (was / now)[:, None]
                codes[p][:, index[had:had + hi - lo].flatten()] = (rows / now[None, :, None]).permute(1, 0, 2).flatten(1)
        found[name] = None if fmt == INT8 else codes.view(s[name + "c"].shape)
        found[name + "_scales"] = scales
    return found


def _sequence(s, name, b, length):
    """A sequence's first tokens [length, H, D] from its pages."""
    H, D, page = s["Hk"], s["D"], s["page"]
    pages = s["table"][b, :-(-length // page)].long()
    codes = s[name + "c"].view(torch.uint8)[pages].view(s[name + "c"].dtype).float().double().view(len(pages), H, page * D)
    x = codes[:, :, _token_index(page, D, name == "v").flatten()].view(len(pages), H, page, D)
    x = x * s[name + "s"].double()[pages][:, :, None, None]
    return x.permute(0, 2, 1, 3).reshape(len(pages) * page, H, D)[:length]


def _exact_read(s):
    offsets, lengths = s["offsets"].tolist(), s["lengths"].tolist()
    return {name: torch.cat([_sequence(s, name, b, lengths[b])[lengths[b] - (offsets[b + 1] - offsets[b]):].flatten(1)
                             for b in range(s["B"]) if offsets[b + 1] > offsets[b]]) for name in ("k", "v")}


def _exact_attention(s):
    """Sequence by sequence and head by head."""
    offsets, lengths = s["offsets"].tolist(), s["lengths"].tolist()
    G, D = s["Hq"] // s["Hk"], s["D"]
    y = torch.zeros(s["T"], s["Hq"], D, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(s["T"], s["Hq"], D)
    for b in range(s["B"]):
        n, length = offsets[b + 1] - offsets[b], lengths[b]
        if not n:
            continue
        k, v = _sequence(s, "k", b, length), _sequence(s, "v", b, length)
        at = torch.arange(length, device="cuda")[None, :]
        me = torch.arange(length - n, length, device="cuda")[:, None]
        hidden = at > me if s["causal"] else torch.zeros(n, length, dtype=torch.bool, device="cuda")
        if s["window"]:
            hidden = hidden | (at <= me - s["window"])
        for h in range(s["Hq"]):
            rows = slice(offsets[b], offsets[b + 1])
            score = (q[rows, h] @ k[:, h // G].t().contiguous() * s["scale"]).masked_fill(hidden, -math.inf)
            y[rows, h] = torch.softmax(score, 1) @ v[:, h // G].contiguous()
    return {"y": y.flatten(1)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "read": _exact_read, "attention": _exact_attention}[case["op"]](s)
