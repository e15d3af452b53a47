"""Cases that measure the products whose matrix depends on the row: the top-k
router with its row grouping, the int8 expert products and the low-rank
adapters.  With ``own`` false ``run`` computes them in elementary torch
operations (fp32 sums); with ``own`` true it calls the library."""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's router: 16 sequences, fine-grained experts; pure latency
        dict(name="route_decode", op="route", t=16, e=64, top=8, bf16=False, renorm=True, masked=0.0),
        # a prefill batch's router; some experts are out of service (their logits are -inf)
        dict(name="route_prefill", op="route", t=8192, e=128, top=8, bf16=True, renorm=False, masked=0.1),
        # one sequence decoding on a few wide experts: gate and up of the 4096 / 11008 layer
        dict(name="swiglu_one_token", op="swiglu", t=1, e=8, top=2, k=4096, n=11008, act="bf16", ybf16=True, tiled=True),
        # 16 sequences decoding on many narrow experts: two rows per expert
        dict(name="swiglu_decode", op="swiglu", t=16, e=64, top=8, k=2048, n=1024, act="bf16", ybf16=True, tiled=True),
        # the same layer's way down, combined per token; weights as quantized (row-major)
        dict(name="combine_decode", op="combine", t=16, e=64, top=8, k=1024, n=2048, act="bf16", ybf16=False, tiled=False),
        # a mid-size batch (speculative or chunked decode), odd row counts and an odd width
        dict(name="experts_odd", op="experts", t=61, e=32, top=4, k=2048, n=1411, act="bf16", ybf16=False, tiled=False),
        # prefill on wide experts, weight-only
        dict(name="swiglu_prefill", op="swiglu", t=2048, e=8, top=2, k=4096, n=11008, act="bf16", ybf16=True, tiled=True),
        # prefill on narrow experts with int8 activations (per-token scales)
        dict(name="experts_prefill_w8a8", op="experts", t=4096, e=64, top=8, k=2048, n=2048, act="int8", ybf16=False, tiled=True),
        dict(name="combine_prefill_w8a8", op="combine", t=2048, e=64, top=8, k=1024, n=2048, act="int8", ybf16=False, tiled=True),
        # decode: 16 sequences of different tenants, an adapter on one projection
        dict(name="adapters_decode", op="adapters", m=16, groups=64, count=1, r=16, k=4096, n=4096, none=0.0, ybf16=False),
        # the q, k, v projections of a mixed batch, a quarter of it without an adapter
        dict(name="adapters_qkv", op="adapters", m=61, groups=64, count=3, r=32, k=4096, n=4096, none=0.25, ybf16=True),
        # prefill: a few requests' prompts through a wide projection
        dict(name="adapters_prefill", op="adapters", m=4129, groups=8, count=1, r=64, k=4096, n=11008, none=0.1, ybf16=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(("route", "experts", "swiglu", "combine", "adapters"))
    if op == "route":
        e = rng.randint(4, 256)
        return dict(op=op, t=_log(rng, 1, 8192), e=e, top=rng.randint(1, min(8, e)), bf16=rng.random() < 0.5,
                    renorm=rng.random() < 0.5, masked=rng.choice((0.0, 0.1)))
    if op == "adapters":
        return dict(op=op, m=_log(rng, 1, 4129), groups=_log(rng, 1, 64), count=rng.randint(1, 3),
                    r=rng.choice((8, 16, 32, 64, 128)), k=128 * rng.randint(4, 64), n=_log(rng, 256, 11008),
                    none=rng.choice((0.0, 0.25)), ybf16=rng.random() < 0.5)
    e = _log(rng, 4, 64)
    return dict(op=op, t=_log(rng, 1, 4096), e=e, top=rng.randint(1, min(8, e)), k=128 * rng.randint(4, 32),
                n=_log(rng, 256, 11008), act=rng.choice(("bf16", "int8")), ybf16=rng.random() < 0.5,
                tiled=rng.random() < 0.5)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _cost(c) <= most:
            return c


def work(case):
    c = case
    if c["op"] == "route":
        pairs = c["t"] * c["top"]
        return {"bytes": c["t"] * c["e"] * (2 if c["bf16"] else 4) + 16 * pairs + 4 * (c["e"] + 1),
                "flops": 4 * c["t"] * c["e"]}
    ysize = 2 if c["ybf16"] else 4
    if c["op"] == "adapters":
        rows = c["m"] * (1 - c["none"])
        active = c["groups"] * (1 - (1 - 1 / c["groups"]) ** rows)
        per = active * c["r"] * (c["k"] + c["n"]) * 2 + 2 * rows * c["n"] * ysize
        return {"bytes": int(rows * c["k"] * 2 + c["count"] * per),
                "flops": int(2 * c["count"] * rows * c["r"] * (c["k"] + c["n"]))}
    rows = c["t"] * c["top"]
    active = c["e"] * (1 - (1 - c["top"] / c["e"]) ** c["t"])
    mats = 2 if c["op"] == "swiglu" else 1
    xrows = rows if c["op"] == "combine" else c["t"]
    yrows = c["t"] if c["op"] == "combine" else rows
    xsize = 2 if c["act"] == "bf16" else 1
    return {"bytes": int(mats * active * c["n"] * (c["k"] + 4) + xrows * c["k"] * xsize + yrows * c["n"] * ysize),
            "flops": 2 * mats * rows * c["n"] * c["k"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(g, shape, sd):
    """int8 codes as absmax quantization of Gaussian rows gives them."""
    return torch.randn(shape, generator=g, device="cuda").mul_(sd).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, shape, mean):
    return (0.8 + 0.4 * torch.rand(shape, generator=g, device="cuda")) * mean


def _tiles16(codes):
    """[e][n][k] int8 -> 16-row tiles per expert: [e][ceil(n/16)][k/64][4][16][16]."""
    e, n, k = codes.shape
    pad = -n % 16
    if pad:
        codes = torch.cat((codes, codes.new_zeros((e, pad, k))), 1)
    return codes.view(e, (n + pad) // 16, 16, k // 64, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous()


def _plan(ids, groups):
    """Rows grouped by id: order (pair numbers), offsets, pos."""
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    order = torch.sort(key, stable=True)[1]
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.cumsum(torch.zeros(groups + 1, dtype=torch.int64, device=flat.device)
                               .index_add_(0, key, torch.ones_like(key))[:groups], 0)
    at = torch.arange(flat.numel(), device=flat.device)
    pos = torch.empty_like(order)
    pos[order] = at
    live = at < offsets[groups]
    return (torch.where(live, order, -1).to(torch.int32), offsets.to(torch.int32),
            torch.where(key < groups, pos, -1).to(torch.int32))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "route":
        bias = 0.5 * torch.randn(c["e"], generator=g, device="cuda")
        logits = 2.0 * torch.randn((c["t"], c["e"]), generator=g, device="cuda") + bias
        if c["masked"]:
            out = torch.rand(c["e"], generator=g, device="cuda") < c["masked"]
            logits = logits.masked_fill(out, -math.inf)
        s["logits"] = logits.bfloat16() if c["bf16"] else logits
        return s
    if c["op"] == "adapters":
        m, r, k, n, G = c["m"], c["r"], c["k"], c["n"], c["groups"]
        # prompts are runs of tokens of one request; decode rows are single tokens
        run = 1 if m <= 64 else max(1, m // 12)
        ids = torch.randint(0, G, (-(-m // run),), generator=g, device="cuda")
        none = torch.rand(ids.shape, generator=g, device="cuda") < c["none"]
        ids = torch.where(none, -1, ids).repeat_interleave(run)[:m].to(torch.int32)
        s["x"] = torch.randn((m, k), generator=g, device="cuda").bfloat16()
        s["ids"] = ids
        s["order"], s["offsets"], s["pos"] = _plan(ids, G)
        s["a"] = [(torch.randn((G, r, k), generator=g, device="cuda") / math.sqrt(k)).bfloat16() for _ in range(c["count"])]
        s["b"] = [(0.5 * torch.randn((G, n, r), generator=g, device="cuda")).bfloat16() for _ in range(c["count"])]
        s["scale"] = [0.5 + torch.rand(G, generator=g, device="cuda") for _ in range(c["count"])]
        s["y"] = [torch.randn((m, n), generator=g, device="cuda").to(torch.bfloat16 if c["ybf16"] else torch.float32)
                  for _ in range(c["count"])]
        return s
    t, e, top, k, n = c["t"], c["e"], c["top"], c["k"], c["n"]
    logits = torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
    v, ids = torch.topk(logits, top, dim=1)
    s["weights"] = torch.softmax(v, 1).contiguous()
    s["ids"] = ids.to(torch.int32)
    s["order"], s["offsets"], s["pos"] = _plan(ids, e)
    s["capacity"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    rows = t * top if c["op"] == "combine" else t
    if c["act"] == "bf16":
        s["x"], s["s_x"] = torch.randn((rows, k), generator=g, device="cuda").bfloat16(), None
    else:
        s["x"], s["s_x"] = _codes(g, (rows, k), 36.0), _scales(g, (rows,), 36.0)
    s["codes"] = [_codes(g, (e, n, k), 30.0) for _ in range(2 if c["op"] == "swiglu" else 1)]
    s["scale"] = [_scales(g, (e, n), 30.0 * math.sqrt(k)) for _ in s["codes"]]
    if c["tiled"]:
        s["tiles"] = [_tiles16(w) for w in s["codes"]]
    return s


# ------------------------------------------------------------------ plain forms

def _plain_route(s):
    c = s["case"]
    l = s["logits"].float()
    l = torch.where(torch.isnan(l), -math.inf, l).clamp(max=torch.finfo(torch.float32).max)
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    v, i = v[:, :c["top"]], i[:, :c["top"]]
    live = v > -math.inf
    top = torch.where(live[:, :1], v[:, :1], 0.0)
    p = torch.where(live, torch.exp(v - top), 0.0)
    total = p.sum(1, keepdim=True) if c["renorm"] else torch.exp(l - top).sum(1, keepdim=True)
    weights = torch.where(live, p / total, 0.0)
    ids = torch.where(live, i, -1).to(torch.int32)
    order, offsets, pos = _plan(ids, c["e"])
    return dict(ids=ids, weights=weights, order=order, offsets=offsets, pos=pos.view(ids.shape))


def _plain_products(s, j):
    """Sorted rows' products with matrix j in fp32: [rows][n]."""
    c = s["case"]
    rows = c["t"] * c["top"]
    at = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].to(torch.int64), at, right=True)
    x = s["x"] if c["op"] == "combine" else s["x"][(s["order"] // c["top"]).to(torch.int64)]
    x = x.float()
    if rows < c["e"]:  # fewer rows than experts: only the chosen matrices
        y = torch.bmm(s["codes"][j][expert].float(), x[:, :, None])[:, :, 0]
    else:  # every expert's rows padded to the largest share
        slot = at - s["offsets"].to(torch.int64)[expert]
        xp = torch.zeros((c["e"], s["capacity"], c["k"]), device="cuda")
        xp[expert, slot] = x
        y = torch.bmm(xp, s["codes"][j].float().transpose(1, 2))[expert, slot]
    y = y / s["scale"][j][expert]
    if s["s_x"] is not None:
        sx = s["s_x"] if c["op"] == "combine" else s["s_x"][(s["order"] // c["top"]).to(torch.int64)]
        y = y / sx[:, None]
    return y


def _plain_experts(s):
    c = s["case"]
    y = _plain_products(s, 0)
    if c["op"] == "swiglu":
        y = y / (1 + torch.exp(-y)) * _plain_products(s, 1)
    if c["op"] == "combine":
        y = (y[s["pos"].to(torch.int64)].view(c["t"], c["top"], c["n"]) * s["weights"][:, :, None]).sum(1)
    return y.to(torch.bfloat16 if c["ybf16"] else torch.float32)


def _plain_adapters(s):
    c = s["case"]
    live = s["ids"] >= 0
    g = s["ids"].clamp(min=0).to(torch.int64)
    x = s["x"].float()
    for a, b, scale, y in zip(s["a"], s["b"], s["scale"], s["y"]):
        if c["m"] <= c["groups"]:  # each row's own matrices
            d = torch.bmm(b[g].float(), torch.bmm(a[g].float(), x[:, :, None]))[:, :, 0]
        else:  # every adapter's low-rank rows of all tokens, then the token's own
            v = torch.matmul(x, a.float().reshape(-1, c["k"]).t()).view(c["m"], c["groups"], c["r"])
            v = v * (torch.arange(c["groups"], device="cuda")[None, :] == g[:, None])[:, :, None]
            d = torch.matmul(v.reshape(c["m"], -1), b.float().permute(0, 2, 1).reshape(-1, c["n"]))
        d = torch.where(live[:, None], d * scale[g][:, None], 0.0)
        y.copy_((y.float() + d).to(y.dtype))
    return s["y"]


# ------------------------------------------------------------------ the library's calls

def _own_groups(qg, s):
    if "groups" not in s:
        c = s["case"]
        s["groups"] = qg.RowGroups(s["offsets"], s["order"], s["pos"], c.get("top", 1))
    return s["groups"]


def _own_experts(qg, s):
    c = s["case"]
    groups = _own_groups(qg, s)
    if "w" not in s:
        fmt = qg.QG_WFMT_INT8_T16 if c["tiled"] else qg.QG_WFMT_INT8
        s["w"] = [qg.QExperts(fmt, c["e"], c["n"], c["k"], w, sc)
                  for w, sc in zip(s["tiles"] if c["tiled"] else s["codes"], s["scale"])]
    dt = torch.bfloat16 if c["ybf16"] else torch.float32
    if c["op"] == "swiglu":
        s["out"] = qg.qgemm_experts_swiglu(s["w"][0], s["w"][1], s["x"], groups, s_x=s["s_x"], y_dtype=dt, y=s.get("out"))
    elif c["op"] == "combine":
        s["out"] = qg.qgemm_experts_combine(s["w"][0], s["x"], groups, s["weights"], s_x=s["s_x"], y_dtype=dt, y=s.get("out"))
    else:
        s["out"] = qg.qgemm_experts(s["w"][0], s["x"], groups, s_x=s["s_x"], y_dtype=dt, y=s.get("out"))
    return s["out"]


def _own_adapters(qg, s):
    if "launch" not in s:
        ad = [qg.LoraAdapters(a, b, sc) for a, b, sc in zip(s["a"], s["b"], s["scale"])]
        s["launch"] = qg.LoraLaunch(s["x"], _own_groups(qg, s), ad, s["y"])
    s["launch"].launch()
    return s["y"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import quantized_gemv_amd as qg
        if op == "route":
            r = s["kept"] = qg.moe_route(s["logits"], s["case"]["top"], renorm=s["case"]["renorm"], out=s.get("kept"))
            return dict(ids=r.ids, weights=r.weights, order=r.groups.order, offsets=r.groups.offsets, pos=r.groups.pos.view(r.ids.shape))
        return _own_adapters(qg, s) if op == "adapters" else _own_experts(qg, s)
    if op == "route":
        return _plain_route(s)
    return _plain_adapters(s) if op == "adapters" else _plain_experts(s)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        l = s["logits"].double().cpu().numpy()
        ids = np.full((c["t"], c["top"]), -1, np.int64)
        weights = np.zeros((c["t"], c["top"]))
        for t in range(c["t"]):
            best = np.argsort(-l[t], kind="stable")[:c["top"]]
            best = best[l[t][best] > -np.inf]
            if len(best):
                p = np.exp(l[t][best] - l[t][best[0]])
                weights[t, :len(best)] = p / (p.sum() if c["renorm"] else np.exp(l[t] - l[t][best[0]]).sum())
                ids[t, :len(best)] = best
        return dict(ids=None, weights=weights, order=None, offsets=None, pos=None)
    if c["op"] == "adapters":
        ids, x = s["ids"].cpu().tolist(), s["x"].double()
        outs = []
        for a, b, scale, y in zip(s["a"], s["b"], s["scale"], s["y"]):
            o = y.double()
            for g in sorted(set(ids) - {-1}):
                rows = torch.tensor([i for i, v in enumerate(ids) if v == g], device="cuda")
                o[rows] += float(scale[g].double()) * (x[rows] @ a[g].double().t()) @ b[g].double().t()
            outs.append(o)
        return outs
    off, order = s["offsets"].cpu().tolist(), s["order"].to(torch.int64)
    rows = c["t"] * c["top"]
    ys = []
    for codes, scale in zip(s["codes"], s["scale"]):
        y = torch.zeros((rows, c["n"]), dtype=torch.float64, device="cuda")
        for e in range(c["e"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            src = torch.arange(lo, hi, device="cuda") if c["op"] == "combine" else order[lo:hi] // c["top"]
            d = s["x"][src].double() @ codes[e].double().t() / scale[e].double()
            y[lo:hi] = d if s["s_x"] is None else d / s["s_x"][src].double()[:, None]
        ys.append(y)
    if c["op"] == "swiglu":
        return ys[0] * torch.sigmoid(ys[0]) * ys[1]
    if c["op"] == "combine":
        out = torch.zeros((c["t"], c["n"]), dtype=torch.float64, device="cuda")
        pair = order[:off[-1]]
        out.index_add_(0, pair // c["top"], ys[0][:off[-1]] * s["weights"].double().reshape(-1)[pair][:, None])
        return out
    return ys[0]
