"""Cases that measure the 8-bit path between two layers: the root-mean-square
norm with the residual's addition and SwiGLU, both with 8-bit outputs and their
scales, quantization to 8-bit floating point (e4m3) in blocks of 128, and the
matrix product of such operands.  With ``own`` false ``run`` computes them in
elementary torch operations (fp32); with ``own`` true it calls the library."""
import math

import numpy as np
import torch

own = False

BLOCK = 128     # values of a row under one step; a weight matrix's blocks are 128 x 128
FP8_MAX = 448.0
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence decoding: the norm before a projection, with the residual; pure latency
        dict(name="norm_token", op="norm", m=1, k=4096, bf16=True, residual=True, out="fp8"),
        # 16 sequences decoding on a wide model, for W8A8 products (int8, a scale per row)
        dict(name="norm_decode_int8", op="norm", m=16, k=8192, bf16=True, residual=True, out="int8"),
        # a prefill batch's norm, an odd number of rows
        dict(name="norm_prefill", op="norm", m=4129, k=4096, bf16=True, residual=True, out="fp8"),
        # weights when they are loaded: fp32, 128 x 128 blocks, the last ones of fewer rows
        dict(name="quantize_weight", op="quantw", n=11000, k=4096),
        # a prefill batch's activations that come without a norm (the attention's output)
        dict(name="quantize_rows", op="quant", m=2048, k=4096, bf16=True),
        # the feed-forward's activation in a decode step and in prefill
        dict(name="swiglu_decode", op="swiglu", m=16, k=11008, bf16=True, out="fp8"),
        dict(name="swiglu_prefill", op="swiglu", m=2048, k=11008, bf16=True, out="fp8"),
        # products: one sequence decoding, weights laid out in tiles when they were loaded
        dict(name="product_token", op="product", m=1, n=4096, k=4096, ybf16=True, tiled=True),
        # 16 sequences decoding through the feed-forward's gate and up, weights as quantized (row-major)
        dict(name="product_decode", op="product", m=16, n=22016, k=4096, ybf16=True, tiled=False),
        # odd counts of rows and columns, fp32 outputs
        dict(name="product_odd", op="product", m=61, n=1411, k=2048, ybf16=False, tiled=False),
        # a chunk of a prompt beside decoding sequences
        dict(name="product_chunk", op="product", m=300, n=4096, k=11008, ybf16=True, tiled=True),
        # prefill
        dict(name="product_prefill", op="product", m=2048, n=11008, k=4096, ybf16=True, tiled=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(("norm", "norm", "quant", "quantw", "swiglu", "product", "product", "product"))
    if op == "quantw":
        return dict(op=op, n=_log(rng, 64, 28672), k=BLOCK * rng.randint(1, 86))
    if op == "product":
        return dict(op=op, m=_log(rng, 1, 4129), n=_log(rng, 128, 28672), k=BLOCK * rng.randint(2, 86),
                    ybf16=rng.random() < 0.5, tiled=rng.random() < 0.5)
    c = dict(op=op, m=_log(rng, 1, 8192), k=BLOCK * _log(rng, 1, 86), bf16=rng.random() < 0.7)
    if op == "norm":
        c["residual"] = rng.random() < 0.7
        c["out"] = rng.choice(("fp8", "fp8", "int8", "bf16"))
    if op == "swiglu":
        c["out"] = rng.choice(("fp8", "fp8", "int8"))
    return c


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
    if c["op"] == "quantw":
        return {"bytes": c["n"] * c["k"] * 5 + 4 * -(-c["n"] // BLOCK) * (c["k"] // BLOCK), "flops": 3 * c["n"] * c["k"]}
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * k + 4 * (m + -(-n // BLOCK)) * (k // BLOCK) + m * n * (2 if c["ybf16"] else 4),
                "flops": 2 * m * n * k}
    size = 2 if c["bf16"] else 4
    out = 2 * c["k"] if c.get("out") == "bf16" else c["k"] + (4 if c.get("out") == "int8" else 4 * (c["k"] // BLOCK))
    if c["op"] == "norm":
        return {"bytes": c["m"] * (c["k"] * size * (3 if c["residual"] else 1) + out) + c["k"] * size,
                "flops": 8 * c["m"] * c["k"]}
    ins = 2 if c["op"] == "swiglu" else 1
    return {"bytes": c["m"] * (c["k"] * size * ins + out), "flops": (8 if c["op"] == "swiglu" else 3) * c["m"] * c["k"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _act(g, m, k, bf16, sd=1.0):
    """Activations: rows of different size, some channels larger than the rest."""
    x = torch.randn((m, k), generator=g, device="cuda")
    x *= sd * torch.exp(0.5 * torch.randn((m, 1), generator=g, device="cuda"))
    big = torch.rand(k, generator=g, device="cuda") < 0.005
    x = torch.where(big, 12.0 * x, x)
    return x.bfloat16() if bf16 else x


def _tiles16(codes):
    """[n][k] bytes -> 16-row tiles: [ceil(n/16)][k/64][4][16][16]."""
    n, k = codes.shape
    pad = -n % 16
    b = codes.view(torch.uint8)
    if pad:
        b = torch.cat((b, b.new_zeros((pad, k))), 0)
    return b.view((n + pad) // 16, 16, k // 64, 4, 16).permute(0, 2, 3, 1, 4).contiguous().view(-1).view(codes.dtype)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    if c["op"] == "quantw":
        s["w"] = torch.randn((c["n"], c["k"]), generator=g, device="cuda") * 0.02
        s["w"] *= torch.exp(0.3 * torch.randn((c["n"], 1), generator=g, device="cuda"))
        return s
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        # as absmax steps per block leave them: the largest code near 448, the rest Gaussian
        s["x"] = (150.0 * torch.randn((m, k), generator=g, device="cuda")).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        s["s_x"] = (0.5 + torch.rand((k // BLOCK, m), generator=g, device="cuda")) * (3.0 / FP8_MAX)
        s["codes"] = (130.0 * torch.randn((n, k), generator=g, device="cuda")).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        s["scale"] = (0.5 + torch.rand((-(-n // BLOCK), k // BLOCK), generator=g, device="cuda")) * (0.08 / FP8_MAX)
        if c["tiled"]:
            s["tiles"] = _tiles16(s["codes"])
        return s
    m, k = c["m"], c["k"]
    if c["op"] == "swiglu":
        s["x"] = _act(g, m, 2 * k, c["bf16"])  # gate's columns, then up's
        return s
    s["x"] = _act(g, m, k, c["bf16"])
    if c["op"] == "norm":
        s["weight"] = 1.0 + 0.2 * torch.randn(k, generator=g, device="cuda")
        if c["bf16"]:
            s["weight"] = s["weight"].bfloat16()
        s["residual"] = _act(g, m, k, c["bf16"], 3.0) if c["residual"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _blocks8(v):
    """Rows in fp32 -> e4m3 codes and the step of every 128 values, [k/128][m]."""
    m, k = v.shape
    b = v.view(m, k // BLOCK, BLOCK)
    step = (b.abs().amax(2) / FP8_MAX).clamp(min=2.0 ** -126)
    return (b * (1.0 / step)[:, :, None]).view(m, k).to(torch.float8_e4m3fn), step.t().contiguous()


def _rows8(v):
    """Rows in fp32 -> int8 codes (as numbers in bf16, which holds them) and the multiplier of each row."""
    mult = 127.0 / v.abs().amax(1)
    return torch.round(v * mult[:, None]).clamp(-127, 127).bfloat16(), mult


def _finish(v, out):
    if out == "bf16":
        return dict(y=v.bfloat16())
    y, s = _rows8(v) if out == "int8" else _blocks8(v)
    return dict(y=y, s=s)


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    v = h * (1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * s["weight"].float()
    r = _finish(v, c["out"])
    if c["residual"]:
        r["residual"] = h.to(s["x"].dtype)
    return r


def _plain_swiglu(s):
    c = s["case"]
    g, u = s["x"][:, :c["k"]].float(), s["x"][:, c["k"]:].float()
    return _finish(g / (1 + torch.exp(-g)) * u, c["out"])


def _plain_weight(s):
    n, k = s["w"].shape
    nb = -(-n // BLOCK)
    w = s["w"] if n % BLOCK == 0 else torch.cat((s["w"], s["w"].new_zeros((nb * BLOCK - n, k))), 0)
    b = w.view(nb, BLOCK, k // BLOCK, BLOCK)
    step = (b.abs().amax((1, 3)) / FP8_MAX).clamp(min=2.0 ** -126)
    codes = (b * (1.0 / step)[:, None, :, None]).view(nb * BLOCK, k)[:n].to(torch.float8_e4m3fn)
    return dict(codes=codes, scale=step)


def _plain_product(s):
    c = s["case"]
    m, n, k = c["m"], c["n"], c["k"]
    x = (s["x"].float().view(m, k // BLOCK, BLOCK) * s["s_x"].t()[:, :, None]).view(m, k)
    rows = s["scale"].repeat_interleave(BLOCK, 0)[:n]
    w = (s["codes"].float().view(n, k // BLOCK, BLOCK) * rows[:, :, None]).view(n, k)
    return torch.matmul(x, w.t()).to(torch.bfloat16 if c["ybf16"] else torch.float32)


# ------------------------------------------------------------------ the library's calls

def _own_launch(qg, s):
    """The launch object that a serving program keeps beside its buffers."""
    c, x = s["case"], s.get("x")
    out = {"fp8": torch.float8_e4m3fn, "int8": torch.int8, "bf16": torch.bfloat16}[c.get("out", "fp8")]
    if c["op"] == "norm":
        ro = torch.empty_like(x) if c["residual"] else None
        return qg.RmsNormLaunch(x, s["weight"], EPS, residual=s["residual"], residual_out=ro, out_dtype=out)
    if c["op"] == "swiglu":
        return qg.SwigluLaunch(x, out_dtype=out)
    fmt = qg.QG_WFMT_FP8_T16 if c["tiled"] else qg.QG_WFMT_FP8
    w = qg.QWeight(fmt, c["n"], c["k"], s["tiles"] if c["tiled"] else s["codes"], s["scale"])
    return qg.QgemmFp8Launch(w, x, s["s_x"], y_dtype=torch.bfloat16 if c["ybf16"] else torch.float32)


def _run_own(qg, s):
    c = s["case"]
    if c["op"] == "quantw":
        w = qg.quantize_fp8_weight(s["w"])
        return dict(codes=w.codes, scale=w.scale)
    if c["op"] == "quant":
        y, step = qg.quantize_fp8(s["x"])
        return dict(y=y, s=step)
    if "launch" not in s:
        s["launch"] = _own_launch(qg, s)
    a = s["launch"]
    a.launch()
    if c["op"] == "product":
        return a.y
    r = dict(y=a.y.bfloat16() if c["out"] == "int8" else a.y)
    if c["out"] != "bf16":
        r["s"] = a.s
    if c.get("residual"):
        r["residual"] = a.residual_out
    return r


def run(state):
    op = state["case"]["op"]
    if own:
        import quantized_gemv_amd as qg
        return _run_own(qg, state)
    if op == "quant":
        y, step = _blocks8(state["x"].float())
        return dict(y=y, s=step)
    return {"norm": _plain_norm, "swiglu": _plain_swiglu, "quantw": _plain_weight, "product": _plain_product}[op](state)


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_codes(v, out):
    """Codes before their rounding, and steps or multipliers, in 64 bits.  None for
    int8 codes: they are whole numbers, and half a step is more than a number in
    bf16 may be off; their multipliers have a value."""
    if out == "bf16":
        return dict(y=v)
    if out == "int8":
        top = np.abs(v).max(1)
        return dict(y=None, s=127.0 / top)
    m, k = v.shape
    top = np.maximum(np.abs(v).reshape(m, k // BLOCK, BLOCK).max(2) / 448.0, 2.0 ** -126)
    return dict(y=v / np.repeat(top, BLOCK, 1), s=np.ascontiguousarray(top.T))


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "product":
        x, w = s["x"].double(), s["codes"].double()
        y = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device="cuda")
        for b in range(c["k"] // BLOCK):
            cols = slice(b * BLOCK, (b + 1) * BLOCK)
            part = torch.matmul(x[:, cols].contiguous(), w[:, cols].t().contiguous())
            per_row = s["scale"][:, b].double()[torch.arange(c["n"], device="cuda") // BLOCK]
            y += part * s["s_x"][b].double()[:, None] * per_row[None, :]
        return y
    if c["op"] == "quantw":
        w = s["w"].double().cpu().numpy()
        nb, kb = -(-c["n"] // BLOCK), c["k"] // BLOCK
        codes, scale = np.empty_like(w), np.empty((nb, kb))
        for i in range(nb):
            rows = w[i * BLOCK:(i + 1) * BLOCK]
            step = np.maximum(np.abs(rows).max(0).reshape(kb, BLOCK).max(1) / 448.0, 2.0 ** -126)
            scale[i] = step
            codes[i * BLOCK:(i + 1) * BLOCK] = rows / np.repeat(step, BLOCK)[None, :]
        return dict(codes=codes, scale=scale)
    x = s["x"].double().cpu().numpy()
    if c["op"] == "quant":
        return _exact_codes(x, "fp8")
    if c["op"] == "swiglu":
        g, u = x[:, :c["k"]], x[:, c["k"]:]
        with np.errstate(over="ignore"):
            return _exact_codes(g * u / (1.0 + np.exp(-g)), c["out"])
    h = x + s["residual"].double().cpu().numpy() if c["residual"] else x
    v = h / np.sqrt((h * h).sum(1, keepdims=True) / c["k"] + EPS) * s["weight"].double().cpu().numpy()
    r = _exact_codes(v, c["out"])
    if c["residual"]:
        r["residual"] = h
    return r
