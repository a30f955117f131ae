"""Measured cases of the per-row operators beside the shared linear layers:

  route     routing tokens to experts: scores, top-k choice, weights, and the
            rows grouped by expert that qlin_grouped_gemm takes
  dispatch  tokens quantized once and stored at their experts' rows
  combine   the weighted sum of the experts' rows back into tokens
  lora      low-rank adapters of many requests added to a shared projection

run() computes them with elementary torch operations in 32 bits (own =
False), or through the library's entry points (own = True).  exact() gives
the same from the definitions in 64 bits.

Sizes: the 128-expert top-8 layer of hidden size 2048 and the projections of
the dense layers of hidden size 2048, 4096 and 5120, which the workloads
name; 256 experts in 8 groups and 60 experts are the larger grouped and the
odd router that the same code has to serve.
"""
import math

import torch

own = False

FLT_MAX = 3.4028234663852886e38
FP8, INT8, BLOCK = 0, 1, 2
QMAX = {FP8: 448.0, INT8: 127.0, BLOCK: 448.0}


def _route(name, T, E, topk, score, dtype, bias=False, groups=1, topk_groups=1, top2=False, renorm=True, scale=1.0,
           closed=0.0):
    c = {"op": "route", "T": T, "E": E, "topk": topk, "score": score, "dtype": dtype, "bias": bias, "groups": groups,
         "topk_groups": topk_groups, "top2": top2, "renorm": renorm, "scale": scale, "closed": closed}
    return dict(c, name=name) if name else c


def _dispatch(name, fmt, T, E, topk, K):
    c = {"op": "dispatch", "fmt": fmt, "T": T, "E": E, "topk": topk, "K": K}
    return dict(c, name=name) if name else c


def _combine(name, T, E, topk, N, dtype, add):
    c = {"op": "combine", "T": T, "E": E, "topk": topk, "N": N, "dtype": dtype, "add": add}
    return dict(c, name=name) if name else c


def _lora(name, M, N, K, adapters, rank, present, run_rows, base=True, dtype="bf16"):
    """present: adapters that the batch uses; run_rows: consecutive rows of one
    request (1: single tokens, each row its own request)."""
    c = {"op": "lora", "M": M, "N": N, "K": K, "adapters": adapters, "rank": rank, "present": present,
         "run_rows": run_rows, "base": base, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one request: latency of the call
        _route("route_1_token", 1, 128, 8, "softmax", "f32"),
        # a decode batch, bf16 logits (ties are common), a few experts shut off
        _route("route_61_tokens_60_experts", 61, 60, 4, "softmax", "bf16", renorm=False, closed=0.05),
        # a prompt through a router with a balance bias and 4 of 8 groups
        _route("route_8192_tokens_grouped", 8192, 256, 8, "sigmoid", "f32", bias=True, groups=8, topk_groups=4, top2=True,
               scale=2.5),
        # a decode batch and a prompt on their way into the experts
        _dispatch("dispatch_32_fp8", FP8, 32, 128, 8, 2048),
        _dispatch("dispatch_4096_block", BLOCK, 4096, 128, 8, 2048),
        # and back out of them: one token in 32 bits, and a prompt beside a residual
        _combine("combine_1_token_f32", 1, 128, 8, 2048, "f32", False),
        _combine("combine_4096_bf16_add", 4096, 128, 8, 2048, "bf16", True),
        # adapters: one request's single token on the smallest qkv projection
        _lora("lora_1_token", 1, 4096, 2048, 8, 16, 1, 1),
        # a decode batch where each request has an adapter of its own, hidden 5120
        _lora("lora_32_requests", 32, 10240, 5120, 64, 16, 32, 1),
        # a large decode batch with ragged ranks on a wide projection, adapters shared by some rows
        _lora("lora_237_requests_wide", 237, 24576, 4096, 48, 64, 48, 1),
        # a prompt batch: long runs of rows of one adapter
        _lora("lora_4096_rows_rank64", 4096, 10240, 5120, 8, 64, 6, 700),
        # the same with small adapters and the sum kept in 32 bits
        _lora("lora_2048_rows_f32", 2048, 4096, 12288, 16, 8, 9, 251, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "combine", "lora", "lora"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = rng.choice([8, 60, 64, 72, 128, 160, 256, 384]) if groups == 1 else groups * rng.randint(4, 40)
        return _route(None, _log(rng, 1, 8192), E, min(E, rng.randint(1, 10)) if groups == 1 else rng.randint(1, 6),
                      rng.choice(["softmax", "sigmoid"]), rng.choice(["f32", "bf16"]), rng.random() < 0.5, groups,
                      rng.randint(2, groups) if groups > 1 else 1, groups > 1 and rng.random() < 0.5,
                      rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.choice([0.0, 0.0, 0.1]))
    if op == "dispatch":
        return _dispatch(None, rng.choice([FP8, INT8, BLOCK]), _log(rng, 1, 4096), rng.choice([8, 60, 128]),
                         rng.randint(1, 8), rng.choice([640, 768, 2048, 2688, 4096, 5120]))
    if op == "combine":
        dtype = rng.choice(["f32", "bf16"])
        return _combine(None, _log(rng, 1, 2048 if dtype == "f32" else 4096), rng.choice([8, 60, 128]), rng.randint(1, 8),
                        16 * rng.randint(40, 160), dtype, rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    M = _log(rng, 1, 1500 if dtype == "f32" else 3000)
    run_rows = rng.choice([1, 1, 16, 131])
    present = rng.randint(1, min(32, (M + run_rows - 1) // run_rows))
    N, K = rng.choice([(4096, 2048), (2048, 2048), (2048, 6144), (6144, 4096), (4096, 4096), (10240, 5120), (5120, 8192)])
    return _lora(None, M, N, K, present + rng.randint(0, 32), rng.choice([8, 16, 32, 64]), present,
                 run_rows, rng.random() < 0.8, dtype)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _slots(g, T, E, topk):
    """The rows that T tokens' pairs take when they are grouped by expert:
    topk distinct experts drawn for each token."""
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(dim=1)[:, :topk].reshape(-1)
    order = torch.argsort(ids, stable=True)
    slots = torch.empty(T * topk, dtype=torch.int32, device="cuda")
    slots[order] = torch.arange(T * topk, dtype=torch.int32, device="cuda")
    return slots.view(T, topk)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dev = {"device": "cuda"}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        logits = _normal(g, T, E, std=1.5)
        if case["closed"]:
            shut = torch.rand(T, E, generator=g, device="cuda") < case["closed"]
            logits = logits.masked_fill(shut, -math.inf)
        s["logits"] = logits.to(_dtype(case))
        # balance biases move in small fixed steps
        s["b"] = torch.randint(-80, 81, (E,), generator=g, device="cuda").float() * 1e-3 if case["bias"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, **dev)
        s["weights"] = torch.empty(T, k, **dev)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, **dev)
        s["rows"] = torch.empty(T * k, dtype=torch.int32, **dev)
        s["slots"] = torch.empty(T, k, dtype=torch.int32, **dev)
    elif case["op"] == "dispatch":
        T, k, K = case["T"], case["topk"], case["K"]
        s["x"] = _normal(g, T, K)
        s["x"][:, torch.randint(0, K, (K // 100 + 1,), generator=g, device="cuda")] *= 20.0   # outlier channels
        s["x"] = s["x"].to(torch.bfloat16)
        s["slots"] = _slots(g, T, case["E"], k)
        s["xq"] = torch.empty(T * k, K, dtype=torch.int8 if case["fmt"] == INT8 else torch.float8_e4m3fn, **dev)
        s["xs"] = torch.empty((T * k, K // 128) if case["fmt"] == BLOCK else (T * k,), **dev)
    elif case["op"] == "combine":
        T, k, N = case["T"], case["topk"], case["N"]
        s["h"] = _normal(g, T * k, N, dtype=_dtype(case))
        s["slots"] = _slots(g, T, case["E"], k)
        s["weights"] = torch.softmax(_normal(g, T, k), 1)
        s["res"] = _normal(g, T, N, dtype=torch.bfloat16) if case["add"] else None
        s["y"] = torch.empty(T, N, dtype=torch.bfloat16, **dev)
    else:
        M, N, K, n, R = case["M"], case["N"], case["K"], case["adapters"], case["rank"]
        s["x"] = _normal(g, M, K, dtype=torch.bfloat16)
        s["A"] = _normal(g, n, R, K, std=K ** -0.5, dtype=torch.bfloat16)
        s["B"] = _normal(g, n, N, R, std=R ** -0.5, dtype=torch.bfloat16)
        # ranks: all of them, half of them, or an odd one
        ranks = torch.tensor([R, R, max(1, R // 2), max(1, R - 3)], dtype=torch.int32, device="cuda")
        s["ranks"] = ranks[torch.randint(0, 4, (n,), generator=g, device="cuda")]
        s["scales"] = 0.25 + torch.rand(n, generator=g, device="cuda")
        used = torch.randperm(n, generator=g, device="cuda")[:case["present"]]
        runs = (M + case["run_rows"] - 1) // case["run_rows"]
        who = torch.cat([torch.arange(case["present"], device="cuda"),
                         torch.randint(0, case["present"], (max(0, runs - case["present"]),), generator=g, device="cuda")])
        ids = used[who[:runs]].repeat_interleave(case["run_rows"])[:M]
        # about one request in sixteen has no adapter
        none = (torch.rand(runs, generator=g, device="cuda") < 1 / 16).repeat_interleave(case["run_rows"])[:M]
        s["ids"] = (ids.masked_fill(none, -1) if M > 1 else ids).to(torch.int32).contiguous()
        s["base_y"] = _normal(g, M, N, dtype=_dtype(case)) if case["base"] else None
        s["y"] = torch.empty(M, N, dtype=_dtype(case), **dev)
    return s


# -------------------------------------------------------------- plain forms

def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["topk"], s["groups"]
    l = s["logits"].float()
    closed = l.isnan() | (l == -math.inf)
    l = l.clamp(max=FLT_MAX).masked_fill(closed, -math.inf)
    none = torch.full_like(l, -math.inf)

    def scores(l):
        if s["score"] == "sigmoid":
            return 1 / (1 + torch.exp(-l))
        top = l.amax(1, keepdim=True)
        p = torch.exp(l - torch.where(top == -math.inf, 0.0, top)).masked_fill(closed, 0.0)
        return p / p.sum(1, keepdim=True).clamp_min(1e-30)

    score = scores(l)
    # whole numbers have to be equal: the choice goes by the logits where the scores have their order, and
    # by scores in 64 bits where a sum comes in, so that no rounding of a score decides it
    if s["b"] is None and not s["top2"]:
        key = l
    else:
        key = scores(l.double())
        if s["b"] is not None:
            key = key + s["b"].double()
        key = torch.where(closed, none.double(), key)
    if G > 1:
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        gs = best[:, :, 0]
        if s["top2"]:
            gs = gs + torch.where(best[:, :, 1] == -math.inf, 0.0, best[:, :, 1])
        kept = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = key.masked_fill(~stays.repeat_interleave(E // G, dim=1), -math.inf)
    got = torch.sort(key, dim=1, descending=True, stable=True)
    ids, there = got.indices[:, :k], got.values[:, :k] > -math.inf
    w = score.gather(1, ids).masked_fill(~there, 0.0)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = w * s["scale"]
    ids = torch.where(there, ids, -1)
    # rows grouped by expert, in token order
    flat = torch.where(there, ids, E).reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = (flat[:, None] == torch.arange(E, device=l.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(T * k, device=l.device)
    rows = torch.where(place < offsets[E], order // k, -1)
    slots = torch.empty_like(place)
    slots[order] = place
    slots = torch.where(there, slots.view(T, k), -1)
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": w, "offsets": offsets.to(i32), "rows": rows.to(i32), "slots": slots.to(i32)}


def _plain_dispatch(s):
    T, k, K, fmt = s["T"], s["topk"], s["K"], s["fmt"]
    x = s["x"].float()
    g = x.view(T, K // 128, 128) if fmt == BLOCK else x.view(T, 1, K)
    qmax = torch.full((), QMAX[fmt], device=x.device)   # a tensor: dividing by it is one division
    scale = g.abs().amax(2, keepdim=True) / qmax
    q = torch.where(scale == 0, 0.0, g / scale).view(T, K)
    q = q.round().clamp(-127, 127).to(torch.int8) if fmt == INT8 else q.clamp(-448, 448).to(torch.float8_e4m3fn)
    place = s["slots"].reshape(-1).long()
    xq = torch.empty_like(s["xq"])
    xq.view(torch.uint8)[place] = q.view(torch.uint8).repeat_interleave(k, dim=0)
    xs = torch.empty_like(s["xs"])
    xs[place] = scale.view((T,) + s["xs"].shape[1:]).repeat_interleave(k, dim=0)
    return {"xq": xq, "xs": xs}


def _plain_combine(s):
    T, k, N = s["T"], s["topk"], s["N"]
    h = s["h"].float()[s["slots"].reshape(-1).long()].view(T, k, N)
    y = (h * s["weights"][:, :, None]).sum(1)
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(s["y"].dtype)}


def _plain_lora(s):
    """Every adapter's product for every row at once, the other adapters' part
    set to zero between the two."""
    M, N, K, n, R = s["M"], s["N"], s["K"], s["adapters"], s["rank"]
    here = torch.arange(R, device="cuda")[None, :] < s["ranks"][:, None]                       # [n, R]
    A = torch.where(here[:, :, None], s["A"].float(), 0.0).view(n * R, K)
    B = torch.where(here[:, None, :], s["B"].float(), 0.0).permute(0, 2, 1).reshape(n * R, N)
    mine = s["ids"][:, None] == torch.arange(n, device="cuda", dtype=torch.int32)[None, :]     # [M, n]
    v = (s["x"].float() @ A.t()).view(M, n, R) * (mine * s["scales"])[:, :, None]
    y = v.view(M, n * R) @ B
    if s["base_y"] is not None:
        y = y + s["base_y"].float()
    return {"y": y.to(s["y"].dtype)}


# ------------------------------------------------------------- entry points

_handles = {}


def _router(q, s):
    """A program keeps one router description for each of its models."""
    key = (s["E"], s["topk"], s["score"], s["groups"], s["topk_groups"], s["top2"], s["renorm"], s["scale"])
    if key not in _handles:
        _handles[key] = q.make_router(s["E"], s["topk"], q.QLIN_SCORE_SIGMOID if s["score"] == "sigmoid" else
                                      q.QLIN_SCORE_SOFTMAX, s["groups"], s["topk_groups"],
                                      q.QLIN_GROUP_TOP2 if s["top2"] else q.QLIN_GROUP_MAX, int(s["renorm"]), s["scale"])
    return _handles[key]


def _workspace(nbytes):
    """One workspace for the stream, as large as the largest call so far needs."""
    ws = _handles.get("workspace")
    if ws is None or ws.numel() < nbytes:
        ws = _handles["workspace"] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device="cuda")
    return ws


def _own(s):
    import skinny_bit_gemm_amd as q
    if s["op"] == "route":
        r = _router(q, s)
        t = q.QLIN_OUT_F32_ACC if s["dtype"] == "f32" else q.QLIN_OUT_BF16
        q.qlin_route(r, s["T"], s["logits"], s["E"], t, s["b"], s["ids"], s["weights"], s["offsets"], s["rows"],
                     s["slots"], _workspace(q.qlin_route_workspace_bytes(r, s["T"])))
        return {name: s[name] for name in ("ids", "weights", "offsets", "rows", "slots")}
    if s["op"] == "dispatch":
        q.qlin_dispatch_quantize(s["fmt"], s["T"], s["topk"], s["K"], s["x"], s["K"], s["slots"], s["T"] * s["topk"],
                                 s["xq"], s["xs"])
        return {"xq": s["xq"], "xs": s["xs"]}
    if s["op"] == "combine":
        q.qlin_combine(s["T"], s["topk"], s["N"], s["h"], s["N"], q.QLIN_OUT_F32_ACC if s["dtype"] == "f32" else
                       q.QLIN_OUT_BF16, s["slots"], s["weights"], s["T"] * s["topk"], s["res"], s["N"], s["y"], s["N"],
                       q.QLIN_OUT_BF16)
        return {"y": s["y"]}
    M, N, K, n, R = s["M"], s["N"], s["K"], s["adapters"], s["rank"]
    q.qlin_lora(M, N, K, n, R, s["x"], K, s["ids"], s["A"], s["B"], s["ranks"], s["scales"], s["base_y"], N, s["y"], N,
                q.QLIN_OUT_F32_ACC if s["dtype"] == "f32" else q.QLIN_OUT_BF16,
                _workspace(q.qlin_lora_workspace_bytes(M, N, K, n, R)))
    return {"y": s["y"]}


_PLAIN = {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine, "lora": _plain_lora}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work

def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    if case["op"] == "dispatch":
        T, k, K = case["T"], case["topk"], case["K"]
        return {"bytes": 2 * T * K + 4 * T * k + T * k * (K + 4 * (K // 128 if case["fmt"] == BLOCK else 1)),
                "flops": 3 * T * K}
    if case["op"] == "combine":
        T, k, N = case["T"], case["topk"], case["N"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * k * N * size + 8 * T * k + (2 * T * N if case["add"] else 0) + 2 * T * N, "flops": 2 * T * k * N}
    M, N, K, R = case["M"], case["N"], case["K"], case["rank"]
    size = 4 if case["dtype"] == "f32" else 2
    r = (R + R + max(1, R // 2) + max(1, R - 3)) / 4   # an adapter's rank, on average
    return {"bytes": 2 * M * K + (2 if case["base"] else 1) * size * M * N + 2 * case["present"] * r * (K + N) + 4 * M,
            "flops": 2 * M * r * (K + N)}


# -------------------------------------------------------------------- exact

def _exact_route(s):
    """Token by token, from the definition."""
    import numpy as np
    T, E, k, G = s["T"], s["E"], s["topk"], s["groups"]
    logits = s["logits"].double().cpu().numpy()
    bias = None if s["b"] is None else s["b"].double().cpu().numpy()
    w = np.zeros((T, k))
    for t in range(T):
        l = np.minimum(logits[t], FLT_MAX)
        is_open = ~np.isnan(l) & (l > -np.inf)
        if not is_open.any():
            continue
        score = np.zeros(E)
        if s["score"] == "sigmoid":
            score[is_open] = 1 / (1 + np.exp(-l[is_open]))
        else:
            e = np.exp(l[is_open] - l[is_open].max())
            score[is_open] = e / e.sum()
        key = np.where(is_open, score if bias is None else score + bias, -np.inf)
        if G > 1:
            top = -np.sort(-key.reshape(G, E // G), axis=1)[:, :2]
            gs = top[:, 0] + np.where(np.isinf(top[:, 1]), 0, top[:, 1]) if s["top2"] else top[:, 0]
            kept = np.argsort(-gs, kind="stable")[:s["topk_groups"]]
            key = np.where(np.isin(np.arange(E) // (E // G), kept), key, -np.inf)
        ids = [e for e in np.argsort(-key, kind="stable")[:k] if key[e] > -np.inf]
        chosen = score[ids]
        if s["renorm"]:
            chosen = chosen / chosen.sum() if chosen.sum() > 0 else 0 * chosen
        w[t, :len(ids)] = chosen * s["scale"]
    return {"ids": None, "weights": torch.from_numpy(w), "offsets": None, "rows": None, "slots": None}


def _exact_dispatch(s):
    """The scales, and the quotients before they are rounded to 8 bits."""
    T, k, K, fmt = s["T"], s["topk"], s["K"], s["fmt"]
    width = 128 if fmt == BLOCK else K
    x = s["x"].double().view(T, K // width, width)
    scale = x.abs().amax(2) / QMAX[fmt]
    quotient = (x / scale[:, :, None]).nan_to_num(0.0).view(T, K)
    token = torch.empty(T * k, dtype=torch.long, device="cuda")
    token[s["slots"].reshape(-1).long()] = torch.arange(T * k, device="cuda") // k
    xs = scale[token]
    return {"xq": None if fmt == INT8 else quotient[token], "xs": xs if fmt == BLOCK else xs[:, 0]}


def _exact_combine(s):
    y = torch.zeros(s["T"], s["N"], dtype=torch.float64, device="cuda")
    for j in range(s["topk"]):
        y += s["weights"][:, j, None].double() * s["h"][s["slots"][:, j].long()].double()
    return {"y": y if s["res"] is None else y + s["res"].double()}


def _exact_lora(s):
    """Adapter by adapter, on its own rows."""
    y = torch.zeros(s["M"], s["N"], dtype=torch.float64, device="cuda")
    if s["base_y"] is not None:
        y += s["base_y"].double()
    ids = s["ids"].cpu()
    for a in sorted(set(ids.tolist()) - {-1}):
        r = int(s["ranks"][a])
        m = (ids == a).nonzero()[:, 0].cuda()
        v = s["x"][m].double() @ s["A"][a, :r].double().t()
        y[m] += float(s["scales"][a]) * (v @ s["B"][a, :, :r].double().t())
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine, "lora": _exact_lora}[case["op"]](s)
