"""GPU: the 8-bit path at the ends of what its calls allow."""
import sys

import numpy as np
import pytest
import torch

import synth
from gpu_util import dev
from oracle import fp8

pytestmark = pytest.mark.gpu
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
