"""GPU product of e4m3 operands in blocks of 128 against the fp64 oracle.

Tolerance of fp32 outputs, elementwise against the sum T of the terms' absolute
values: the matrix instruction adds the 128 products of a block in fp32 in an
order of its own, rounded or cut off (at most 127 whole steps of 2^-23), then
one rounding of the steps' product, k / 128 multiply-adds and up to 8 sums
across waves: (254 + 1 + k / 128 + 8) half steps of 2^-24 of T.  bf16 outputs:
of every eight consecutive products each may lose less than 2^-13 of the
largest's binade, seven of them at most (the largest itself is whole), so
7 2^-13 of the sum of those binades; then the rounding, 2^-8 of the result.
Where every sum is a whole number below 2^24, products reach over fewer than 13
binades and the steps are powers of two, outputs are exact."""
import sys

import numpy as np
import pytest
import torch

import synth
from gpu_util import canaries_intact, dev, f32_to_bf16_rne, guarded, host
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


def e4(codes):
    return dev(codes).view(E4)


def operands(g, m, n, k):
    """Codes of Gaussian values (largest code in use, some subnormal) and steps."""
    x = fp8.encode(np.clip(g.standard_normal((m, k)) * 130, -448, 448))
    w = fp8.encode(np.clip(g.standard_normal((n, k)) * 130 * 2.0 ** -g.integers(0, 12, (n, 1)), -448, 448))
    s_x = (g.random((k // 128, m)) + 0.1).astype(np.float32) * np.float32(0.01)
    s_w = (g.random((-(-n // 128), k // 128)) + 0.1).astype(np.float32) * np.float32(0.001)
    return x, s_x, w, s_w


def weights(qg, w, s_w, tiled):
    W = qg.QWeight(qg.QG_WFMT_FP8, w.shape[0], w.shape[1], e4(w), dev(s_w))
    return qg.tiled16(W) if tiled else W


def bf16_close(y, ref, size, top, k):
    """A bf16 output within its tolerance."""
    off = (263 + k // 128) * HALF * size + 7 * 2.0 ** -13 * top
    return np.all(np.abs(y.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + off * (1 + 2.0 ** -8))


def run(qg, W, x, s_x, dtype=torch.float32):
    """y with canaries around it."""
    m, n = x.shape[0], W.n
    full, y = guarded(m * n, dtype)
    y = y.view(m, n)
    qg.qgemm_fp8(W, x, s_x, y=y)
    assert canaries_intact(full, m * n)
    return y


# m: every number of 16-row tiles, both sides of the kernels' borders; n: ends inside tiles, blocks, four columns
SHAPES = [(1, 1, 128), (1, 16, 256), (1, 4096, 4096), (2, 130, 1152), (5, 257, 128), (15, 1411, 2048), (16, 384, 11008),
          (17, 130, 256), (31, 64, 1024), (32, 515, 640), (33, 128, 2176), (47, 2000, 384), (48, 36, 4096), (49, 16, 128),
          (61, 1411, 2048), (64, 256, 1024), (65, 130, 384), (100, 384, 512), (127, 250, 256), (128, 128, 128),
          (129, 129, 1408), (200, 1000, 2048), (255, 33, 640), (256, 256, 4096), (257, 258, 384), (300, 640, 1152),
          (513, 511, 256), (700, 96, 2048), (1025, 300, 128), (7, 100, 8320), (16, 4200, 256), (3, 9000, 128),
          (12, 11000, 384), (18, 4200, 128), (29, 9010, 256), (32, 4097, 256), (40, 4200, 256), (64, 3000, 128),
          (129, 129, 11008), (150, 203, 8192), (333, 1500, 1408), (600, 1300, 1152)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(qg, m, n, k):
    g = synth.rng(m * 1000003 + n * 1009 + k)
    x, s_x, w, s_w = operands(g, m, n, k)
    ref, size, top = fp8.product(x, s_x, w, s_w)
    for tiled in (False, True):
        note("product m=%d n=%d k=%d tiled=%s" % (m, n, k, tiled))
        W, xd, sd = weights(qg, w, s_w, tiled), e4(x), dev(s_x)
        y = host(run(qg, W, xd, sd))
        assert np.all(np.abs(y - ref) <= (263 + k // 128) * HALF * size)
        assert np.max(np.abs(y - ref)) <= 1e-5 * np.max(np.abs(ref))
        assert torch.equal(run(qg, W, xd, sd), dev(y))  # the same bits again
        yb = run(qg, W, xd, sd, torch.bfloat16)
        assert bf16_close(yb, ref, size, top, k)
        assert torch.equal(run(qg, W, xd, sd, torch.bfloat16), yb)


@pytest.mark.parametrize("m,n,k", [(1, 300, 1024), (16, 48, 4096), (40, 130, 512), (64, 500, 256), (130, 260, 1152),
                                   (300, 700, 640), (512, 512, 512), (600, 1300, 1152), (1300, 2100, 640), (332, 13999, 256),
                                   (200, 300, 8192)])
@pytest.mark.parametrize("tiled", [False, True])
def test_exact_where_sums_are_whole(qg, m, n, k, tiled):
    """Every output told apart: whole codes, steps that are powers of two."""
    note("whole m=%d n=%d k=%d tiled=%s" % (m, n, k, tiled))
    g = synth.rng(m + n + k)
    x, w = fp8.encode(g.integers(-8, 9, (m, k))), fp8.encode(g.integers(-8, 9, (n, k)))
    s_x = 2.0 ** g.integers(-2, 3, (k // 128, m)).astype(np.float32)
    s_w = 2.0 ** g.integers(-2, 3, (-(-n // 128), k // 128)).astype(np.float32)
    ref, size, _ = fp8.product(x, s_x, w, s_w, cut=False)
    assert size.max() * 16 < 2 ** 24  # in units of 2^-4
    W = weights(qg, w, s_w, tiled)
    y = host(run(qg, W, e4(x), dev(s_x)))
    assert np.array_equal(y, ref.astype(np.float32))
    assert np.array_equal(host(run(qg, W, e4(x), dev(s_x), torch.bfloat16)), f32_to_bf16_rne(y))


# every kind of tile, in parts of k and not, and two kinds in one launch; ends
# inside tiles in both directions
LARGE = [(300, 4096, 11008), (2048, 512, 8192), (700, 4100, 1152), (1000, 1003, 8192), (4096, 4352, 128), (4100, 4611, 256),
         (2048, 2050, 4096), (513, 11008, 640), (9000, 128, 384), (130, 20001, 256), (4096, 8192, 384), (1029, 2050, 1152),
         (2500, 2601, 384), (600, 1100, 4096), (1683, 11827, 640), (200000, 16, 128),
         (785, 23363, 640), (387, 11809, 640), (197, 8343, 4864), (969, 1318, 4480), (450, 10265, 384), (162, 5545, 3712),
         (70000, 250, 256), (1100000, 16, 128)]


@pytest.mark.parametrize("m,n,k", LARGE)
def test_large_exact(qg, m, n, k):
    """Whole codes again; the reference is the fp64 product on the GPU, exact here."""
    torch.manual_seed(m + n + k)
    x = torch.randint(-4, 5, (m, k), device="cuda").float().to(E4)
    w = torch.randint(-4, 5, (n, k), device="cuda").float().to(E4)
    s_x = 2.0 ** torch.randint(-1, 2, (k // 128, m), device="cuda").float()
    s_w = 2.0 ** torch.randint(-1, 2, (-(-n // 128), k // 128), device="cuda").float()
    xs = x.double().view(m, k // 128, 128) * s_x.t().double()[:, :, None]
    ws = w.double().view(n, k // 128, 128) * s_w.double().repeat_interleave(128, 0)[:n, :, None]
    ref = torch.matmul(xs.view(m, k), ws.view(n, k).t().contiguous())
    del xs, ws
    assert 16 * 4 * 4 * k < 2 ** 24 * 4  # |terms| <= 16, times steps of 1/4 .. 4, in units of 1/4
    W = qg.QWeight(qg.QG_WFMT_FP8, n, k, w, s_w)
    for tiled in (False, True):
        note("large m=%d n=%d k=%d tiled=%s" % (m, n, k, tiled))
        L = qg.tiled16(W) if tiled else W
        assert torch.equal(run(qg, L, x, s_x), ref.float())
        assert torch.equal(run(qg, L, x, s_x, torch.bfloat16), ref.float().bfloat16())


def test_workspaces(qg):
    """A workspace of the caller's, whatever it holds; an object's own on another
    stream; too small a one."""
    note("workspaces")
    m, n, k = 300, 4096, 11008
    x = torch.randint(0, 0x48, (m, k), dtype=torch.uint8, device="cuda").view(E4)
    W = qg.QWeight(qg.QG_WFMT_FP8, n, k, torch.randint(0, 0x48, (n, k), dtype=torch.uint8, device="cuda").view(E4),
                   torch.rand(n // 128, k // 128, device="cuda"))
    s_x = torch.rand(k // 128, m, device="cuda")
    y = qg.qgemm_fp8(W, x, s_x, y_dtype=torch.float32)
    need = qg.lib().qg_qgemm_fp8_workspace_bytes(m, n, k, qg.QG_F32)
    assert need > 0
    for fill in (0, 255):
        full, ws = guarded(need, torch.uint8)
        ws.fill_(fill)
        assert torch.equal(qg.qgemm_fp8(W, x, s_x, y_dtype=torch.float32, ws=ws), y)
        assert canaries_intact(full, need)
    with pytest.raises(qg.QgError):
        qg.qgemm_fp8(W, x, s_x, y_dtype=torch.float32, ws=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = qg.QgemmFp8Launch(W, x, s_x, y_dtype=torch.float32)
    out = a.y
    with torch.cuda.stream(side):
        for _ in range(3):
            a.launch()
    del a  # its workspace must not be given out while the side stream works
    junk = [torch.full((need // 4,), float("nan"), device="cuda") for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    del junk


@pytest.mark.parametrize("m", [1, 16, 61, 130, 300, 9000])
@pytest.mark.parametrize("tiled", [False, True])
def test_all_codes(qg, m, tiled):
    """Every pair of finite codes meets at least once; one-hot rows pick them."""
    note("all codes m=%d tiled=%s" % (m, tiled))
    fin = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    k, n = 256, len(fin)
    g = synth.rng(m)
    w = np.zeros((n, k), np.uint8)
    at = g.integers(0, k, m)
    x = np.zeros((m, k), np.uint8)
    x[np.arange(m), at] = g.choice(fin, m)
    w[:, :] = fin[:, None]
    s_x = np.ones((2, m), np.float32)
    s_w = np.ones((2, 2), np.float32)
    ref, _, _ = fp8.product(x, s_x, w, s_w, cut=False)
    W = weights(qg, w, s_w, tiled)
    y = host(run(qg, W, e4(x), dev(s_x)))
    assert np.array_equal(y, ref.astype(np.float32))
    assert np.array_equal(host(run(qg, W, e4(x), dev(s_x), torch.bfloat16)), f32_to_bf16_rne(y))


@pytest.mark.parametrize("m,n,k", [(1, 200, 1024), (20, 200, 512), (130, 200, 1024), (300, 300, 384),
                                   (260, 260, 8192), (600, 1300, 1152), (136, 5641, 3456)])
@pytest.mark.parametrize("tiled", [False, True])
def test_nan_reaches_its_outputs_only(qg, m, n, k, tiled):
    note("nan m=%d n=%d tiled=%s" % (m, n, tiled))
    g = synth.rng(m + n)
    x, s_x, w, s_w = operands(g, m, n, k)
    clean = host(run(qg, weights(qg, w, s_w, tiled), e4(x), dev(s_x)))
    i, j = m - 1, n - 1
    x2, w2, sx2, sw2 = x.copy(), w.copy(), s_x.copy(), s_w.copy()
    x2[i, k - 1] = 0x7F
    w2[j, 130] = 0xFF
    y = host(run(qg, weights(qg, w2, s_w, tiled), e4(x2), dev(s_x)))
    hit = (np.arange(m) == i)[:, None] | (np.arange(n) == j)[None, :]
    assert np.all(np.isnan(y[hit])) and np.array_equal(y[~hit], clean[~hit])
    yb = run(qg, weights(qg, w2, s_w, tiled), e4(x2), dev(s_x), torch.bfloat16)
    assert np.array_equal(np.isnan(yb.float().cpu().numpy()), hit)
    sx2[0, i] = np.nan
    sw2[1, 1] = np.inf  # rows 128 .. 255 of the matrix
    y = host(run(qg, weights(qg, w, sw2, tiled), e4(x), dev(sx2)))
    assert np.all(np.isnan(y[i])) and not np.isfinite(y[:i, 128:256]).any()
    assert np.array_equal(y[:i, :128], clean[:i, :128]) and np.array_equal(y[:i, 256:], clean[:i, 256:])


def test_large_steps_and_small_ones(qg):
    note("steps")
    g = synth.rng(1)
    for m in (3, 200):
        x, s_x, w, s_w = operands(g, m, 130, 256)
        for a, b in ((1e20, 1e-20), (1e-30, 1e25), (1e-20, 1e-10)):
            sx, sw = (s_x * np.float32(a)).astype(np.float32), (s_w * np.float32(b)).astype(np.float32)
            ref, size, _ = fp8.product(x, sx, w, sw, cut=False)
            y = host(run(qg, weights(qg, w, sw, True), e4(x), dev(sx)))
            assert np.all(np.abs(y - ref) <= 265 * HALF * size)


def whole_codes(*shape):
    """Codes of -2, -1, 0, 1 and 2, made in slices."""
    table = torch.tensor([-2.0, -1.0, 0.0, 1.0, 2.0], device="cuda").to(E4).view(torch.uint8)
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for rows in out.view(-1, shape[-1]).split(8192):
        rows.copy_(table[torch.randint(0, 5, rows.shape, device="cuda")])
    return out.view(E4)


def rows_of(t, at):
    return t.view(torch.uint8)[at:].contiguous().view(E4)


def test_far_offsets(qg):
    """Matrices, activations and outputs past 4 GiB, against their last rows
    alone. Whole codes and steps of 1 and 1/2: sums below 2^18 in halves, so
    exact whichever kernel adds them."""
    note("far offsets")
    step = lambda *s: 0.5 + 0.5 * torch.randint(0, 2, s, device="cuda").float()
    k = 65536
    n = (1 << 32) // k + 300
    at = 65408  # 128 rows of step before 4 GiB
    w, s_w = whole_codes(n, k), step(-(-n // 128), k // 128)
    x, s_x = whole_codes(20, k), step(k // 128, 20)
    for tiled in (False, True):
        W = qg.QWeight(qg.QG_WFMT_FP8, n, k, w, s_w)
        part = qg.QWeight(qg.QG_WFMT_FP8, n - at, k, rows_of(w, at), s_w[at // 128:].contiguous())
        if tiled:
            W, part = qg.tiled16(W), qg.tiled16(part)
        for rows in (1, 20):
            xs, ss = rows_of(x, 20 - rows), s_x[:, 20 - rows:].contiguous()
            y = qg.qgemm_fp8(W, xs, ss, y_dtype=torch.float32)
            assert torch.equal(y[:, at:], qg.qgemm_fp8(part, xs, ss, y_dtype=torch.float32))
            ref = torch.zeros(rows, n - at, dtype=torch.float64, device="cuda")
            for b in range(k // 128):
                cols = slice(128 * b, 128 * b + 128)
                rows_step = s_w[at // 128:, b].double().repeat_interleave(128)[:n - at]
                ref += (xs[:, cols].double() @ part_cols(w, at, cols).t().contiguous()) * ss[b].double()[:, None] * rows_step
            assert torch.equal(y[:, at:], ref.float())
    # many tokens: the matrix as activations
    W = qg.QWeight(qg.QG_WFMT_FP8, 20, k, x, step(1, k // 128))
    sx = step(k // 128, n)
    for dt in (torch.float32, torch.bfloat16):
        y = qg.qgemm_fp8(W, w, sx, y_dtype=dt)
        assert torch.equal(y[at:], qg.qgemm_fp8(W, rows_of(w, at), sx[:, at:].contiguous(), y_dtype=dt))
    del w, W, y
    # outputs past 4 GiB
    m, n = 120000, 20000
    xs, sx = whole_codes(m, 128), step(1, m)
    W = qg.QWeight(qg.QG_WFMT_FP8, n, 128, whole_codes(n, 128), step(-(-n // 128), 1))
    for dt in (torch.float32, torch.bfloat16):
        y = qg.qgemm_fp8(W, xs, sx, y_dtype=dt)
        for at in (m - 700, 53600):  # 4 GiB of bf16 end in row 107374, of fp32 in row 53687
            assert torch.equal(y[at:at + 700], qg.qgemm_fp8(W, rows_of(xs, at)[:700], sx[:, at:at + 700].contiguous(), y_dtype=dt))
        del y


def part_cols(w, at, cols):
    return w.view(torch.uint8)[at:, cols].contiguous().view(E4).double()


def test_two_streams_and_graphs(qg):
    note("streams, graphs")
    g = synth.rng(2)
    launches, want = [], []
    for m, n, k in ((1, 1024, 2048), (61, 700, 1024), (300, 512, 1024)):
        x, s_x, w, s_w = operands(g, m, n, k)
        launches.append(qg.QgemmFp8Launch(weights(qg, w, s_w, m == 1), e4(x), dev(s_x), y_dtype=torch.float32))
        launches[-1].launch()
        want.append(launches[-1].y.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in launches]
    for a, st in zip(launches, streams):
        a.y.zero_()
    torch.cuda.synchronize()
    for a, st in zip(launches, streams):
        with torch.cuda.stream(st):
            a.launch()
    torch.cuda.synchronize()
    assert all(torch.equal(a.y, w) for a, w in zip(launches, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a in launches:
            a.launch()
    for _ in range(3):
        for a in launches:
            a.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.y, w) for a, w in zip(launches, want))


@pytest.mark.parametrize("t", [1, 16, 70, 300, 1500])
@pytest.mark.parametrize("tiled", [False, True])
def test_feed_forward(qg, t, tiled):
    """norm, gate and up, SwiGLU, down, as a layer runs them: each step against
    the oracle on what the step before it gave."""
    note("ffn t=%d tiled=%s" % (t, tiled))
    g = synth.rng(t)
    d, n, d2 = 512, 384, 520
    x = synth.to_bf16_bits(g.standard_normal((t, d)))
    r = synth.to_bf16_bits(3 * g.standard_normal((t, d)))
    nw = (1 + 0.1 * g.standard_normal(d)).astype(np.float32)
    xd, rd = dev(x).view(torch.bfloat16), dev(r).view(torch.bfloat16)
    gate_up = qg.quantize_fp8_weight(dev((g.standard_normal((2 * n, d)) / np.sqrt(d)).astype(np.float32)))
    down = qg.quantize_fp8_weight(dev((g.standard_normal((d2, n)) / np.sqrt(n)).astype(np.float32)))
    L = [qg.tiled16(w) if tiled else w for w in (gate_up, down)]
    y = qg.fp8_ffn(xd, rd, dev(nw), L[0], L[1])
    assert y.shape == (t, d2) and y.dtype == torch.bfloat16
    f32 = synth.bf16_bits_to_f32
    h = (f32(x) + f32(r)).astype(np.float32)
    assert np.array_equal(host(rd), f32_to_bf16_rne(h))
    q, s = qg.rms_norm(xd, dev(nw), 1e-6, dev(r).view(torch.bfloat16), out_dtype=E4)
    gu = qg.qgemm_fp8(L[0], q, s)
    codes = lambda W: host(W.codes.view(torch.uint8))
    ref, size, top = fp8.product(host(q.view(torch.uint8)), host(s), codes(gate_up), host(gate_up.scale))
    assert bf16_close(gu, ref, size, top, d)
    a, sa = qg.swiglu(gu, out_dtype=E4)
    ref, size, top = fp8.product(host(a.view(torch.uint8)), host(sa), codes(down), host(down.scale))
    assert bf16_close(y, ref, size, top, n)
    # the whole layer in fp64 on the quantized weights: the activations' codes are
    # off by up to half a step, 2^-4 of a value, twice; a sum of many averages them
    v, _ = fp8.rms_norm(f32(x), nw, 1e-6, f32(r))
    W = [fp8.decode(codes(w)) * np.repeat(np.repeat(host(w.scale).astype(np.float64), 128, 0)[:w.n], 128, 1)
         for w in (gate_up, down)]
    whole = fp8.swiglu(v @ W[0].T) @ W[1].T
    assert np.linalg.norm(y.float().cpu().numpy() - whole) <= 2 * (2.0 ** -4 + 2.0 ** -4) * np.linalg.norm(whole)


def test_int8_norm_feeds_the_w8a8_products(qg):
    note("norm -> W8A8")
    g = synth.rng(4)
    t, d, n = 37, 512, 300
    x = synth.to_bf16_bits(g.standard_normal((t, d)))
    nw = (1 + 0.1 * g.standard_normal(d)).astype(np.float32)
    q, s = qg.rms_norm(dev(x).view(torch.bfloat16), dev(nw), out_dtype=torch.int8)
    wq, s_w = qg.quantize_absmax(dev(g.standard_normal((n, d)).astype(np.float32)))
    y = host(qg.qgemm_w8a8(q, s, None, wq, s_w, None, 0))
    acc = host(q).astype(np.int64) @ host(wq).astype(np.int64).T
    ref = acc / (host(s).astype(np.float64)[:, None] * host(s_w).astype(np.float64)[None, :])
    # float(acc), two reciprocals of 1 ulp and two products
    assert np.all(np.abs(y - ref) <= 8 * HALF * np.abs(ref))
