"""GPU: the 8-bit path at the ends of what its calls allow."""
import sys

import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import dev, dev_bf16, f32_to_bf16_rne, host
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


def positive(g, *shape):
    """Codes of whole numbers 1 .. 8: every sum over a block is above zero."""
    return fp8.encode(g.integers(1, 9, shape))


# streams of one block and of two requested ahead, in workgroups of 8 and 16 waves, with and without waves that
# have no block left; tiles of every kind, in parts of k and whole
STEPS = [(1, 200, 384), (1, 130, 4096), (1, 300, 2176), (16, 4200, 384), (3, 9000, 384), (5, 257, 11008), (20, 200, 384),
         (31, 300, 2176), (30, 4200, 384), (61, 130, 384), (64, 1411, 2176), (130, 260, 1152), (300, 640, 1152),
         (298, 1024, 9984), (600, 1300, 1152), (801, 1000, 13696)]


@pytest.mark.parametrize("m,n,k", STEPS)
@pytest.mark.parametrize("tiled", [False, True])
def test_steps_without_an_end(qg, m, n, k, tiled):
    """An infinite step in the last block, and two finite ones whose product
    leaves fp32's range: infinite outputs, as the formula has it, whichever
    kernel runs; NaN where the infinite step meets a sum of zero."""
    note("steps m=%d n=%d k=%d tiled=%s" % (m, n, k, tiled))
    g = synth.rng(m + n + k)
    x, w = positive(g, m, k), positive(g, n, k)
    s_x = (2.0 ** g.integers(-2, 3, (k // 128, m))).astype(np.float32)
    s_w = (2.0 ** g.integers(-2, 3, (-(-n // 128), k // 128))).astype(np.float32)
    W = qg.QWeight(qg.QG_WFMT_FP8, n, k, dev(w).view(E4), dev(s_w))
    i, j = m - 1, (n - 1) // 128
    rows = np.arange(n) // 128 == j

    def y(s_x, s_w, dtype, x=x):
        L = qg.QWeight(W.fmt, n, k, W.codes, dev(s_w))
        return qg.qgemm_fp8(qg.tiled16(L) if tiled else L, dev(x).view(E4), dev(s_x), y_dtype=dtype).float().cpu().numpy()

    for dtype in (torch.float32, torch.bfloat16):
        clean = y(s_x, s_w, dtype)
        assert np.all(np.isfinite(clean)) and np.all(clean > 0)
        sx = s_x.copy()
        sx[-1, i] = np.inf
        got = y(sx, s_w, dtype)
        assert np.all(got[i] == np.inf) and np.array_equal(got[:i], clean[:i])
        sw = s_w.copy()
        sw[j, -1] = np.inf
        got = y(s_x, sw, dtype)
        assert np.all(got[:, rows] == np.inf) and np.array_equal(got[:, ~rows], clean[:, ~rows])
        sx, sw = s_x.copy(), s_w.copy()
        sx[-1, i] = sw[j, -1] = 1e25
        got = y(sx, sw, dtype)
        assert np.all(got[i, rows] == np.inf) and np.all(np.isfinite(got[i, ~rows])) and np.all(np.isfinite(got[:i]))
        assert np.array_equal(got[:i, ~rows], clean[:i, ~rows])
        zero = x.copy()
        zero[i, k - 128:] = 0
        sx = s_x.copy()
        sx[-1, i] = np.inf
        assert np.all(np.isnan(y(sx, s_w, dtype, zero)[i]))


def gates():
    """Gates over the whole range, densely where exp(-|g|) is a number."""
    near = np.concatenate([np.linspace(-110, 110, 40001), np.linspace(-88.9, -87.2, 4001),
                           2.0 ** np.linspace(-140, 6, 2001), -2.0 ** np.linspace(-140, 6, 2001)])
    far = np.array([0.0, -0.0, 1e4, -1e4, 1e10, -1e10, 1e30, 3e38, -1e30, -3e38, 126.5, -126.5, -149.0, -360.0, -362.0])
    g = np.concatenate([near, far]).astype(np.float32)
    return np.concatenate([g, np.zeros(-len(g) % 128, np.float32)])


@pytest.mark.parametrize("up", [1.0, -1.7, 3e30, 1e-30, 2.0 ** -120])
@pytest.mark.parametrize("bf16", [True, False])
def test_swiglu_over_the_range_of_fp32(qg, up, bf16):
    """fp32 outputs.  In half steps: exp(-g) from the square of the hardware's 2^t
    (one unit, 2, twice), the product that corrects it (1) and ln 2, whose fp32 value
    is off by 2^-28.4 (|g| 2^-28.4, |g| / 21 half steps), all of it times 1 / (1 + exp(g)) <= 1; the
    sum 1, the reciprocal 2 (one unit), two products 2: 10 + |g| / 21.  What is
    below 2^-126 keeps steps of 2^-149, half of one each: 1 / (1 + exp(-g)), which goes times |g u|
    (and where the scaled sum is above 2^126 its reciprocal, 2^-158, is 0), silu, which
    goes times |u|, and the result."""
    note("swiglu range up=%g bf16=%s" % (up, bf16))
    g = gates()
    n = len(g)
    u = (up * (1 + np.arange(n) % 7 / 8)).astype(np.float32)
    x = np.stack([np.concatenate([g, u]), np.concatenate([g, -u])])
    if bf16:
        bits = synth.to_bf16_bits(x)
        x, xd = synth.bf16_bits_to_f32(bits), dev_bf16(bits)
    else:
        xd = dev(x)
    gate, upv = x[:, :n].astype(np.float64), np.abs(x[:, n:].astype(np.float64))
    ref = fp8.swiglu(x)
    top = float(np.finfo(np.float32).max)
    y = host(qg.swiglu(xd, out_dtype=torch.float32))
    fits = np.abs(ref) <= top * (1 - 15 * HALF)  # gates from -88 on are below 15 half steps
    gu = np.abs(gate) * upv
    off = (10 + np.abs(gate) / 21) * HALF * np.abs(ref) + 2.0 ** -150 * ((1 + 2.0 ** -8) * gu + upv + 1)
    err = np.abs(y.astype(np.float64) - ref)
    worst = np.max(np.where(fits & (np.abs(ref) >= 2.0 ** -126) & (gate > -85) & (np.abs(gate) >= 2.0 ** -125), err / (HALF * np.maximum(np.abs(ref), 2.0 ** -126)), 0.0))
    print("half steps, at worst: %.2f" % worst, flush=True)
    assert np.all(err[fits] <= off[fits])
    over = np.abs(ref) > top * (1 + 15 * HALF)
    assert np.array_equal(y[over], np.copysign(np.inf, ref[over]).astype(np.float32))
    # the other outputs are the roundings of the same values
    assert np.array_equal(host(qg.swiglu(xd)), f32_to_bf16_rne(y))
    for dtype, most in ((E4, 40064), (torch.int8, 32768)):  # gates of -110 .. 110 and of -110 .. 70
        part = xd[:, torch.cat([torch.arange(most), n + torch.arange(most)]).cuda()].contiguous()
        q, s = qg.swiglu(part, out_dtype=dtype)
        if dtype == E4:
            ref_q, ref_s = fp8.quantize(y[:, :most])
            assert np.array_equal(host(s), ref_s) and np.array_equal(host(q.view(torch.uint8)), ref_q)
        else:
            ref_q, ref_s = oracle.quantize_absmax(y[:, :most], per_row=True)
            assert np.array_equal(host(s), ref_s) and np.array_equal(host(q), ref_q)


def test_swiglu_of_what_is_no_number(qg):
    """The formula's values: silu(inf) = inf, silu(-inf) = -inf / inf = NaN."""
    note("swiglu inf, nan")
    g = np.array([np.inf, -np.inf, np.nan, np.inf, 0.0, 2.0, -2.0, 0.0], np.float32)
    u = np.array([1.0, 1.0, 1.0, -2.0, np.inf, np.inf, np.inf, np.nan], np.float32)
    y = host(qg.swiglu(dev(np.concatenate([g, u])[None]), out_dtype=torch.float32))[0]
    assert np.array_equal(y, np.array([np.inf, np.nan, np.nan, -np.inf, np.nan, np.inf, -np.inf, np.nan], np.float32), equal_nan=True)


@pytest.mark.parametrize("k", [8, 128, 384, 4096, 32768])
@pytest.mark.parametrize("bf16", [True, False])
def test_rms_norm_with_a_large_eps(qg, k, bf16):
    """eps up to fp32's largest value beside rows whose squares leave the range,
    and beside rows whose squares do not but whose sum with eps does.  26 half
    steps as for every norm; scaling by powers of two adds none.  Results below
    2^-126 keep steps of 2^-149."""
    note("norm eps k=%d bf16=%s" % (k, bf16))
    g = synth.rng(k)
    scale = np.array([1.0, 1e15, 1e18, 4e18, 1.8e19, 3e19, 2e20, 1e22, 1e30, 0.0])[:, None]
    x = (g.uniform(0.5, 1.0, (10, k)) * np.where(g.random((10, k)) < 0.5, -1, 1) * scale).astype(np.float32)
    r = (g.uniform(-0.2, 0.2, (10, k)) * scale).astype(np.float32)
    w = (1 + g.random(k)).astype(np.float32)
    if bf16:
        xb, rb = synth.to_bf16_bits(x), synth.to_bf16_bits(r)
        x, r = synth.bf16_bits_to_f32(xb), synth.bf16_bits_to_f32(rb)
        xd, rd = dev_bf16(xb), dev_bf16(rb)
    else:
        xd, rd = dev(x), dev(r)
    for eps in (1e-6, 1.0, 1e30, 1e36, 1e38, 3.3e38, float(np.finfo(np.float32).max)):
        for res in (None, r):
            v, _ = fp8.rms_norm(x, w, float(np.float32(eps)), res)
            y = host(qg.rms_norm(xd, dev(w), eps, None if res is None else rd, None if res is None else torch.empty_like(rd),
                                 out_dtype=torch.float32))
            assert np.all(np.abs(y - v) <= 26 * HALF * np.abs(v) + 2.0 ** -149), (eps, res is None)


@pytest.mark.parametrize("m,n,k", [(1, 200, 384), (30, 4200, 384), (600, 1300, 1152), (298, 1024, 9984)])
def test_steps_whose_product_is_below_the_normal_numbers(qg, m, n, k):
    """s_x s_w of 2^-148: kept as fp32 keeps it, so whole sums come out exactly."""
    note("small steps m=%d n=%d k=%d" % (m, n, k))
    g = synth.rng(m + k)
    x, w = positive(g, m, k), positive(g, n, k)
    s_x, s_w = np.full((k // 128, m), 2.0 ** -126, np.float32), np.full((-(-n // 128), k // 128), 2.0 ** -22, np.float32)
    ref = (fp8.decode(x) @ fp8.decode(w).T) * 2.0 ** -148  # sums up to 64 k, below 2^24
    W = qg.QWeight(qg.QG_WFMT_FP8, n, k, dev(w).view(E4), dev(s_w))
    y = host(qg.qgemm_fp8(W, dev(x).view(E4), dev(s_x), y_dtype=torch.float32))
    assert np.array_equal(y.astype(np.float64), ref)
