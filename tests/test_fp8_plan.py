"""Which kernel an e4m3 product of given sizes reaches (CPU): every one that any
size reaches is reached by the sizes of the GPU tests, and no launch goes past
what a grid may have."""
import os
import random
import subprocess

import pytest

import test_gpu_fp8_paths as paths
import test_gpu_fp8gemm as gemm

HERE = os.path.dirname(os.path.abspath(__file__))
HEADER = os.path.join(HERE, "..", "quantized_gemv_amd", "csrc", "qg_fp8_plan.h")
S, M, H, L, XL = range(5)
BM, BN = (64, 128, 192, 256, 256), (64, 128, 128, 128, 256)
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def plans():
    exe, src = os.path.join(HERE, "host", "_fp8_plan_driver"), os.path.join(HERE, "host", "fp8_plan_driver.cpp")
    if not os.path.exists(exe) or os.path.getmtime(exe) < max(os.path.getmtime(src), os.path.getmtime(HEADER)):
        made = "%s.%d" % (exe, os.getpid())
        subprocess.run(["g++", "-O2", "-std=c++17", src, "-o", made], check=True)
        os.replace(made, exe)

    def run(sizes):
        text = "".join("%d %d %d %d\n" % s for s in sizes)
        out = subprocess.run([exe], input=text, capture_output=True, check=True, text=True).stdout.splitlines()
        return [tuple(int(v) for v in line.split()) for line in out]
    return run


def kernel(size, plan):
    """What tells one launch of the library from another: a stream by its tokens,
    rows and waves; tiles by kind and outputs, whole, in parts of k, or two kinds."""
    (m, n, k, yt), (stream, kind, parts, cols, rest) = size, plan
    if stream:
        return "stream", 1 if m <= 16 else 2 if m <= 32 else 3, kind, m <= 16 and kind == 1 and k > 4096
    if kind == XL and cols < -(-n // 256):
        return "two", rest, yt
    return "tiles", kind, yt, parts > 1


# every kernel that 20000 sizes of a projection reach (test_no_other_kernel): streams of 16 tokens x 16 (8 or 16
# waves), 32, 64 rows, of 32 tokens x 16, 32 rows in one pass and in several; tiles; two kinds
ALL = {("stream", 1, 1, False), ("stream", 1, 1, True), ("stream", 1, 2, False), ("stream", 1, 4, False),
       ("stream", 2, 1, False), ("stream", 2, 2, False), ("stream", 3, 1, False), ("stream", 3, 2, False)}
ALL |= {("tiles", kind, yt, parts) for kind in (S, M, H, L) for yt in (F32, BF16) for parts in (False, True)}
ALL |= {("tiles", XL, BF16, False), ("tiles", XL, BF16, True), ("two", H, BF16), ("two", L, BF16)}


def test_gpu_tests_reach_every_kernel(plans):
    sizes = [(*s, yt) for s in gemm.SHAPES + gemm.LARGE + paths.PATHS for yt in (F32, BF16)]
    got = {kernel(s, p) for s, p in zip(sizes, plans(sizes))}
    assert ALL <= got, sorted(ALL - got, key=str)


def test_captured_and_concurrent_products_use_a_workspace(plans):
    for yt in (F32, BF16):
        sizes = [(*s, yt) for s in paths.JOINED]
        assert all(p[2] > 1 for p in plans(sizes))


def test_no_other_kernel_and_no_launch_too_large(plans):
    """Random sizes over the whole range: grids, parts of k and columns of tiles."""
    rng = random.Random(5)
    log = lambda hi: int(2 ** rng.uniform(0, hi))
    sizes = []
    while len(sizes) < 60000:
        m, n, k = (log(28), log(26), 128 * log(11.01)) if len(sizes) % 2 else (log(13), log(15.5), 128 * log(7.5))
        if m < 1 << 28 and n < 1 << 26 and k <= 262144 and m * k <= 1 << 40 and n * k <= 1 << 40 and m * n <= 1 << 36:
            sizes.append((m, n, k, rng.randint(0, 1)))
    sizes += [(1 << 20, 1 << 16, 128, 1), ((1 << 28) - 1, 255, 128, 0), (1, (1 << 26) - 1, 16384, 1), (16, (1 << 26) - 1, 128, 0),
              (17, (1 << 26) - 1, 128, 0), (1 << 20, 16, 262144, 1), ((1 << 20) + 1, 16, 128, 1), (1023, (1 << 26) - 1, 128, 1)]
    up = lambda a, b: -(-a // b)
    seen = set()
    for (m, n, k, yt), p in zip(sizes, plans(sizes)):
        stream, kind, parts, cols, rest = p
        what = (m, n, k, yt, p)
        seen.add(kernel((m, n, k, yt), p))
        if stream:
            threads = 1024 if m <= 16 and kind == 1 and k > 4096 else 512
            gx, gy = up(n, 16 * kind), up(m, 16 if m <= 16 else 32)
            assert parts == 1 and gy < 1 << 16 and gx * gy * threads <= 1 << 32, what
            assert kind in ((1, 2, 4) if m <= 16 else (1, 2)), what
            continue
        assert 1 <= parts <= min(8, k // 128) and kind <= (L if yt == F32 else XL), what
        tm, tn = up(m, BM[kind]), up(n, BN[kind])
        grid = tm * tn * parts
        if kind == XL and cols < tn:
            assert cols >= 1 and parts == 1 and rest in (H, L), what
            grid = tm * cols + up(m, BM[rest]) * up(n - 256 * cols, BN[rest])
        else:
            assert cols >= tn, what
        assert grid * 512 < 1 << 32 and tm < 1 << 31, what
    assert seen == ALL, (sorted(seen - ALL, key=str), sorted(ALL - seen, key=str))
