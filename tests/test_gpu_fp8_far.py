"""GPU row operators of the 8-bit path where offsets pass 32 bits: more rows than
a launch has workgroups for, values past element 2^32, chunks past 2^32.
Inputs repeat a block of rows, so outputs repeat the block's own, which a small call
gives; its length is a prime (times 128 for weights), so no wrong offset by a
power of two meets the same row."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
PERIOD = 1000003  # rows
K = 128


def note(msg):
    print("[case] " + msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantized_gemv_amd as q
    q.lib()
    return q


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def room(gib):
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < (gib + 4) << 30:
        pytest.skip("%d GiB of GPU memory are free, %d needed" % (free >> 30, gib + 4))


def repeated(block, rows):
    out = torch.empty(rows, block.shape[1], dtype=block.dtype, device="cuda")
    for at in range(0, rows, len(block)):
        out[at:at + len(block)].copy_(block[:rows - at])
    return out


def same(a, b):
    as_bits = lambda t: t.view(torch.uint8) if t.dtype == E4 else t
    return torch.equal(as_bits(a), as_bits(b))


def check(got, block, dim=0):
    """Every repetition of the block along dim, and the part of one at the end."""
    rows, period = got.shape[dim], block.shape[dim]
    for at in range(0, rows, period):
        n = min(period, rows - at)
        assert same(got.narrow(dim, at, n), block.narrow(dim, 0, n)), at


FAR = 34000001  # rows of 128: 4.35e9 values, 2125001 workgroups of 16 rows


def test_norm_with_residual(qg):
    note("far norm")
    room(40)
    x, r = (torch.randn(PERIOD, K, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = torch.rand(K, device="cuda") + 0.5
    for dtype in (E4, torch.int8, torch.bfloat16):
        ro = torch.empty_like(r)
        y = qg.rms_norm(x, w, residual=r, residual_out=ro, out_dtype=dtype)
        xf, rf = repeated(x, FAR), repeated(r, FAR)
        a = qg.RmsNormLaunch(xf, w, residual=rf, residual_out=torch.empty_like(rf) if dtype == E4 else rf, out_dtype=dtype)
        a.launch()
        check(a.y, y if a.s is None else y[0])
        check(a.residual_out, ro)
        if a.s is not None:
            check(a.s, y[1], a.s.dim() - 1)
        del a, xf, rf
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [E4, torch.int8, torch.float32])
def test_swiglu(qg, dtype):
    note("far swiglu %s" % dtype)
    room(40)
    x = torch.randn(PERIOD, 2 * K, device="cuda", dtype=torch.bfloat16)
    y = qg.swiglu(x, out_dtype=dtype)
    a = qg.SwigluLaunch(repeated(x, FAR), out_dtype=dtype)
    a.launch()
    check(a.y, y if a.s is None else y[0])
    if a.s is not None:
        check(a.s, y[1], a.s.dim() - 1)


@pytest.mark.parametrize("rows", [FAR, (1 << 28) + 1000])
def test_quantize(qg, rows):
    """Workgroups that walk on, and more than 2^32 chunks of 8 values."""
    note("far quantize rows=%d" % rows)
    room(rows * (3 * K + 4) >> 30)
    x = torch.randn(PERIOD, K, device="cuda", dtype=torch.bfloat16)
    q, s = qg.quantize_fp8(x)
    qf, sf = qg.quantize_fp8(repeated(x, rows))
    check(qf, q)
    check(sf, s, 1)


def test_quantize_weight(qg):
    """More blocks of 128 x 128 than workgroups; the last has fewer rows."""
    note("far weights")
    n = (1 << 27) + 128 * 1000 + 5
    room(n * 3 * K >> 30)
    period = 128 * 7919
    w = torch.randn(period, K, device="cuda", dtype=torch.bfloat16)
    W = qg.quantize_fp8_weight(w)
    F = qg.quantize_fp8_weight(repeated(w, n))
    whole = n // 128 * 128
    check(F.codes[:whole], W.codes)
    check(F.scale[:whole // 128], W.scale)
    at = whole % period
    last = qg.quantize_fp8_weight(w[at:at + n - whole].clone())
    assert same(F.codes[whole:], last.codes) and same(F.scale[whole // 128:], last.scale)
