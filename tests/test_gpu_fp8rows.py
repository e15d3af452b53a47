"""GPU norm, SwiGLU and e4m3 quantization against the fp64 oracle.

Float outputs are compared with the formula in fp64, elementwise, in half steps
of fp32 (HALF = 2^-24).  Norm: the sum of squares runs through at most 8
multiply-adds and 4 sums in a lane, 6 across the wave and 15 across a
workgroup, 1 / k and its product, eps and h's own rounding (twice in h^2): the
root halves these 38; then root, quotient, two products and h: 19 + 5, so 26.
SwiGLU (see the kernel): the exponent is off by 2 |g| half steps, then 8 more
for exp, sum, reciprocal (1 ulp each at most) and products; where exp(-g) exceeds
2^126 its reciprocal may be flushed to zero: |g u| 2^-126.
8-bit outputs and scales have to equal, bit for bit, the oracle's quantization
of the fp32 output of the same kernel."""
import sys

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import bf16_to_f64, canaries_intact, dev, dev_bf16, f32_to_bf16_rne, guarded, host
from oracle import fp8

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24
E4 = torch.float8_e4m3fn


def note(msg):
    print("[case] " + msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantized_gemv_amd as q
    q.lib()
    return q


def rows_of(g, m, k, bf16, sd=1.0):
    """(values, device tensor) of rows of different size."""
    x = (g.standard_normal((m, k)) * sd * np.exp(g.standard_normal((m, 1)))).astype(np.float32)
    if not bf16:
        return x, dev(x)
    bits = synth.to_bf16_bits(x)
    return synth.bf16_bits_to_f32(bits), dev_bf16(bits)


def codes_of(t):
    return host(t.view(torch.uint8))


def check_fp8(y32, q, s):
    ref_q, ref_s = fp8.quantize(y32)
    assert np.array_equal(host(s), ref_s, equal_nan=True)
    nan = lambda c: np.where(c & 127 == 127, 127, c)  # either sign is NaN
    assert np.array_equal(nan(codes_of(q)), nan(ref_q))


def check_int8(y32, q, s):
    ref_q, ref_s = oracle.quantize_absmax(y32, per_row=True)
    assert np.array_equal(host(s), ref_s) and np.array_equal(host(q), ref_q)


# lanes per row: 16, 64, 256 and more; ends inside a chunk of lanes; one row to many
NORMS = [(1, 8), (3, 128), (17, 120), (5, 136), (16, 512), (4, 520), (33, 1024), (1, 4096), (7, 4104), (130, 5120),
         (2, 8192), (3, 11008), (1, 16384), (2, 24320), (2, 32768), (2, 32760), (1031, 256), (515, 2048), (300, 4096), (257, 6016),
         (258, 8192), (259, 11008), (261, 16376), (257, 24576), (257, 28672)]


@pytest.mark.parametrize("m,k", NORMS)
@pytest.mark.parametrize("bf16,wbf16,res", [(True, True, True), (True, False, False), (False, False, True), (False, True, False)])
def test_rms_norm(qg, m, k, bf16, wbf16, res):
    note("norm m=%d k=%d bf16=%s wbf16=%s res=%s" % (m, k, bf16, wbf16, res))
    g = synth.rng(m * 40000 + k)
    x, xd = rows_of(g, m, k, bf16)
    w, wd = rows_of(g, 1, k, wbf16)
    w, wd = w[0], wd.view(-1)
    r, rd = rows_of(g, m, k, bf16, 3.0) if res else (None, None)
    ro = torch.empty_like(xd) if res else None
    eps = 1e-5
    v, h = fp8.rms_norm(x, w, eps, r)
    full, y32 = guarded(m * k, torch.float32)
    y32 = y32.view(m, k)
    qg.rms_norm(xd, wd, eps, rd, ro, y=y32)
    assert canaries_intact(full, m * k)
    y = host(y32)
    # h's own rounding acts on x and r of opposite sign, too: relative to h, as everything here
    assert np.all(np.abs(y - v) <= 26 * HALF * np.abs(v))
    if res:
        h32 = (x + r).astype(np.float32)
        assert np.array_equal(host(ro), f32_to_bf16_rne(h32) if bf16 else h32)
        assert np.array_equal(host(rd), synth.to_bf16_bits(r) if bf16 else r)
    yb = qg.rms_norm(xd, wd, eps, rd, ro)
    assert yb.dtype == torch.bfloat16 and np.array_equal(host(yb), f32_to_bf16_rne(y))
    full, q = guarded(m * k, torch.int8)
    q, s = qg.rms_norm(xd, wd, eps, rd, ro, y=q.view(m, k))
    check_int8(y, q, s)
    assert canaries_intact(full, m * k)
    if k % 128 == 0:
        fs, s = guarded(k // 128 * m, torch.float32)
        q, s = qg.rms_norm(xd, wd, eps, rd, ro, out_dtype=E4, s=s.view(k // 128, m))
        check_fp8(y, q, s)
        assert canaries_intact(fs, k // 128 * m)


@pytest.mark.parametrize("m,k", [(1, 128), (9, 136), (6, 4096), (5, 4104), (3, 20000)])
@pytest.mark.parametrize("where", ["residual", "x"])
def test_rms_norm_in_place(qg, m, k, where):
    note("in place m=%d k=%d %s" % (m, k, where))
    g = synth.rng(k + m)
    x, xd = rows_of(g, m, k, True)
    r, rd = rows_of(g, m, k, True)
    w = dev(np.ones(k, np.float32))
    apart = torch.empty_like(rd)
    y, s = qg.rms_norm(xd, w, 1e-6, rd, apart, out_dtype=torch.int8)
    y2, s2 = qg.rms_norm(xd, w, 1e-6, rd, None if where == "residual" else xd, out_dtype=torch.int8)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    assert torch.equal(rd if where == "residual" else xd, apart)


def test_rms_norm_over_the_range_of_fp32(qg):
    """Rows whose squares leave fp32's range upwards or downwards; zeros."""
    note("norm range")
    g = synth.rng(5)
    for k in (128, 384, 4096):
        base = g.standard_normal((6, k))
        scale = np.array([1e19, 3e37, 1e-19, 1e-38, 0.0, 1.0])[:, None]
        x = (base * scale).astype(np.float32)
        w = (1 + g.random(k)).astype(np.float32)
        for eps in (1e-6, float(np.float32(1.2e-38))):
            v, _ = fp8.rms_norm(x, w, float(np.float32(eps)))
            y = host(qg.rms_norm(dev(x), dev(w), eps, out_dtype=torch.float32))
            # values below 2^-126 keep steps of 2^-149; squares below it vanish beside eps:
            # k of them add less than 2^-149 (1 + k) / k to a mean of eps >= 2^-126
            assert np.all(np.abs(y - v) <= 27 * HALF * np.abs(v) + 2.0 ** -149), (k, eps)
            q, s = qg.rms_norm(dev(x), dev(w), eps, out_dtype=E4)
            check_fp8(y, q, s)


@pytest.mark.parametrize("k", [128, 512, 4096])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_rows_that_are_not_finite(qg, k, bad):
    note("not finite k=%d %s" % (k, bad))
    g = synth.rng(k)
    x = g.standard_normal((20, k)).astype(np.float32)
    x[7, k - 1] = bad
    w = np.ones(k, np.float32)
    xd, wd = dev(x), dev(w)
    clean = np.arange(20) != 7
    y = host(qg.rms_norm(xd, wd, out_dtype=torch.float32))
    ref, _ = fp8.rms_norm(x[clean], w, 1e-6)
    assert np.all(np.abs(y[clean] - ref) <= 26 * HALF * np.abs(ref)) and np.isnan(y[7, k - 1])
    q, s = qg.rms_norm(xd, wd, out_dtype=torch.int8)
    assert np.isnan(host(s)[7]) and np.all(np.isfinite(host(s)[clean]))
    check_int8(y[clean], q[torch.from_numpy(clean).cuda()], s[torch.from_numpy(clean).cuda()])
    q, s = qg.rms_norm(xd, wd, out_dtype=E4)
    check_fp8(y, q, s)
    assert np.all(codes_of(q)[7, k - 128:] & 127 == 127)
    q, s = qg.quantize_fp8(xd)
    check_fp8(x, q, s)
    assert np.isnan(host(s)[k // 128 - 1, 7]) and np.isfinite(host(s)).sum() == 20 * (k // 128) - 1
    W = qg.quantize_fp8_weight(xd)
    assert np.isnan(host(W.scale)[0, k // 128 - 1]) and np.all(np.isfinite(host(W.scale)[0, :-1]))
    gu = np.concatenate([x, np.ones_like(x)], 1)
    q, s = qg.swiglu(dev(gu), out_dtype=torch.int8)
    # silu(-inf) is -inf / inf: NaN, as the formula has it
    assert np.isnan(host(s)[7]) and np.all(np.isfinite(host(s)[clean]))


SWIGLUS = [(1, 8), (1, 128), (3, 1024), (16, 11008), (7, 136), (65, 384), (2, 32768), (300, 1408), (1, 40064)]


@pytest.mark.parametrize("m,n", SWIGLUS)
@pytest.mark.parametrize("bf16", [True, False])
def test_swiglu(qg, m, n, bf16):
    note("swiglu m=%d n=%d bf16=%s" % (m, n, bf16))
    g = synth.rng(m * 50000 + n)
    x, xd = rows_of(g, m, 2 * n, bf16, 2.0)
    if n >= 128:  # gates far on either side
        x[0, :6] = [100.0, -100.0, 88.5, -88.5, -87.0, -20.0]
        xd = dev_bf16(synth.to_bf16_bits(x)) if bf16 else dev(x)
    ref = fp8.swiglu(x)
    full, y32 = guarded(m * n, torch.float32)
    y32 = y32.view(m, n)
    qg.swiglu(xd, y=y32)
    assert canaries_intact(full, m * n)
    y = host(y32)
    gate, up = np.abs(x[:, :n]), np.abs(x[:, n:])
    assert np.all(np.abs(y - ref) <= (2 * gate + 8) * HALF * np.abs(ref) + gate * up * 2.0 ** -126)
    assert np.array_equal(host(qg.swiglu(xd)), f32_to_bf16_rne(y))
    if n <= qg.QG_ROW_MAX_K:
        q, s = qg.swiglu(xd, out_dtype=torch.int8)
        check_int8(y, q, s)
    if n % 128 == 0:
        full, q = guarded(m * n, torch.uint8)
        q, s = qg.swiglu(xd, y=q.view(E4).view(m, n))
        check_fp8(y, q, s)
        assert canaries_intact(full, m * n)


@pytest.mark.parametrize("m,k", [(1, 128), (2, 256), (5, 640), (31, 128), (2048, 512), (77, 11008)])
@pytest.mark.parametrize("bf16", [True, False])
def test_quantize_fp8(qg, m, k, bf16):
    note("quantize m=%d k=%d bf16=%s" % (m, k, bf16))
    g = synth.rng(m + k)
    x, _ = rows_of(g, m, k, True)
    x[0, :128] = 0.0
    x[m - 1, k - 128:] *= np.float32(2.0 ** -124)  # steps at their lower bound
    x[m // 2, :7] = [448.0, -448.0, 0.0, -0.0, 26.0, 2.0 ** -9, 1.5 * 2.0 ** -9]
    bits = synth.to_bf16_bits(x)
    x = synth.bf16_bits_to_f32(bits)
    full, q = guarded(m * k, torch.uint8)
    fs, s = guarded(m * (k // 128), torch.float32)
    q, s = qg.quantize_fp8(dev_bf16(bits) if bf16 else dev(x), q.view(E4).view(m, k), s.view(k // 128, m))
    check_fp8(x, q, s)
    assert canaries_intact(full, m * k) and canaries_intact(fs, m * (k // 128))


@pytest.mark.parametrize("n,k", [(1, 128), (127, 128), (128, 256), (129, 384), (1000, 1408)])
@pytest.mark.parametrize("bf16", [True, False])
def test_quantize_fp8_weight(qg, n, k, bf16):
    note("weight n=%d k=%d bf16=%s" % (n, k, bf16))
    w, wd = rows_of(synth.rng(n + k), n, k, bf16, 0.02)
    W = qg.quantize_fp8_weight(wd)
    codes, scale = fp8.quantize_weight(w)
    assert W.fmt == qg.QG_WFMT_FP8 and np.array_equal(host(W.scale), scale) and np.array_equal(codes_of(W.codes), codes)
    T = qg.tiled16(W)
    t = codes_of(T.codes).reshape(-(-n // 16), k // 64, 4, 16, 16).transpose(0, 3, 1, 2, 4).reshape(-1, k)
    assert T.fmt == qg.QG_WFMT_FP8_T16 and np.array_equal(t[:n], codes) and not t[n:].any() and T.scale is W.scale


def test_codes_are_torchs_rounding(qg):
    """Every bf16 value of a block whose step is 1, against torch's narrowing."""
    note("all bf16 values up to 448")
    bits = np.arange(1 << 16).astype(np.uint16)
    v = synth.bf16_bits_to_f32(bits)
    v = v[np.isfinite(v) & (np.abs(v) <= 448)]
    v = np.concatenate([v, np.zeros(-len(v) % 127, np.float32)]).reshape(-1, 127)
    v = np.concatenate([v, np.full((len(v), 1), 448, np.float32)], 1)
    q, s = qg.quantize_fp8(dev(v))
    assert np.all(host(s) == 1)
    assert torch.equal(q.cpu().view(torch.uint8), torch.from_numpy(v).to(E4).view(torch.uint8))


def test_launches_on_a_stream_and_in_a_graph(qg):
    note("graph")
    g = synth.rng(9)
    _, x = rows_of(g, 16, 4096, True)
    _, r = rows_of(g, 16, 4096, True)
    w = dev(np.ones(4096, np.float32))
    norm = qg.RmsNormLaunch(x, w, residual=r, residual_out=torch.empty_like(r), out_dtype=E4)
    gu = torch.randn(16, 2048, device="cuda")
    act = qg.SwigluLaunch(gu, out_dtype=torch.int8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norm.launch()
        act.launch()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in (norm.y.view(torch.uint8), norm.s, norm.residual_out, act.y, act.s)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm.launch()
        act.launch()
    for step in range(3):
        for t in (norm.y.view(torch.uint8), norm.s, norm.residual_out, act.y, act.s):
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((norm.y.view(torch.uint8), norm.s, norm.residual_out, act.y, act.s), want):
            assert torch.equal(a, b)
        # new inputs in the same memory
        x.copy_(torch.randn_like(x))
        gu.copy_(torch.randn_like(gu))
        norm.launch()
        act.launch()
        want = [t.clone() for t in (norm.y.view(torch.uint8), norm.s, norm.residual_out, act.y, act.s)]


def test_many_rows(qg):
    """More workgroups than a launch starts, and offsets past 32 bits."""
    note("many rows")
    m, k = 18000001, 128
    x = torch.randn(m, k, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(k, device="cuda")
    y, s = qg.rms_norm(x, w, out_dtype=E4)
    for lo in (0, m // 2, (1 << 24) - 3, m - 1000):
        part, sp = qg.rms_norm(x[lo:lo + 1000].clone(), w, out_dtype=E4)
        assert torch.equal(y[lo:lo + 1000].view(torch.uint8), part.view(torch.uint8)) and torch.equal(s[:, lo:lo + 1000], sp)
    y, s = qg.quantize_fp8(x)
    for lo in (0, m // 2, (1 << 24) - 3, m - 1000):
        part, sp = qg.quantize_fp8(x[lo:lo + 1000].clone())
        assert torch.equal(y[lo:lo + 1000].view(torch.uint8), part.view(torch.uint8)) and torch.equal(s[:, lo:lo + 1000], sp)
