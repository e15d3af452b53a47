"""GPU low-rank adapters (qg_lora_add) against the fp64 oracle.

Tolerance per row: A x is exact products in fp32 sums (1e-5 of the row's
largest component, as for the W8A16 products), its part in y at most
|scale| sum_j |B[n][j]| times that; the second product adds r + 8 roundings of
its absolute sum; y is rounded once (fp32 2^-24, bf16 2^-8)."""
import sys

import numpy as np
import pytest
import torch

from gpu_util import TOL_F32, bf16_to_f64, dev, dev_bf16, host
from oracle import rows as R
import synth

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24


def note(msg):
    print("[case] " + msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantized_gemv_amd as q
    q.lib()
    return q


def bf16(g, shape, sd):
    bits = synth.to_bf16_bits(synth.gaussian(g, shape, sd))
    return dev_bf16(bits), synth.bf16_bits_to_f32(bits).astype(np.float64)


class Case:
    def __init__(self, qg, m, groups, k, mats, ybf16, seed, drop=0.0, runs=False, scaled=True):
        """mats: list of (r, n)."""
        g = synth.rng(seed)
        self.xd, self.x = bf16(g, (m, k), 1.0)
        ids = np.repeat(g.integers(0, groups, m // 7 + 1), 7)[:m] if runs else g.integers(0, groups, m)
        self.ids = np.where(g.random(m) < drop, -1, ids).astype(np.int32)
        self.groups = qg.group_rows(dev(self.ids), groups)
        self.ad, self.np, self.ys, self.y0, self.full = [], [], [], [], []
        for r, n in mats:
            ad, a = bf16(g, (groups, r, k), 1.0 / np.sqrt(k))
            bd, b = bf16(g, (groups, n, r), 0.7)
            s = (0.5 + g.random(groups)).astype(np.float32) if scaled else None
            self.ad.append(qg.LoraAdapters(ad, bd, None if s is None else dev(s)))
            self.np.append((a, b, s))
            full = torch.empty(m * n + 128, dtype=torch.bfloat16 if ybf16 else torch.float32, device="cuda")
            full.view(torch.uint8).fill_(0x5A)
            y = full[64:64 + m * n].view(m, n)
            yd, yv = bf16(g, (m, n), 1.0)
            y.copy_(yd)
            self.ys.append(y)
            self.y0.append(yv)
            self.full.append(full)
        self.ybf16 = ybf16

    def want(self, j):
        a, b, s = self.np[j]
        d = R.lora_delta(self.x, self.ids, a, b, s)
        tol = np.zeros_like(d)
        for t, g in enumerate(self.ids):
            if g >= 0:
                v = a[g] @ self.x[t]
                sc = 1.0 if s is None else float(s[g])
                tol[t] = sc * (np.abs(b[g]).sum(1) * TOL_F32 * np.abs(v).max()
                               + (b.shape[2] + 8) * 2 * HALF * (np.abs(b[g]) @ np.abs(v)))
        y = self.y0[j] + d
        return y, tol + (2.0 ** -8 if self.ybf16 else HALF) * (np.abs(y) + tol)

    def check(self):
        for j, y in enumerate(self.ys):
            want, tol = self.want(j)
            got = bf16_to_f64(host(y)) if self.ybf16 else host(y).astype(np.float64)
            none = self.ids < 0
            assert np.array_equal(got[none], self.y0[j][none]), "rows without an adapter changed"
            bad = np.abs(got - want) - tol
            bad[none] = 0
            assert np.all(bad <= 0), "matrix %d off by up to %g" % (j, bad.max())
            raw = self.full[j].view(torch.uint8).cpu().numpy()
            isz = self.full[j].dtype.itemsize
            assert np.all(raw[:64 * isz] == 0x5A) and np.all(raw[-64 * isz:] == 0x5A), "written outside"


@pytest.mark.parametrize("ybf16", [False, True])
@pytest.mark.parametrize("m,groups,k,mats,drop,runs", [
    (1, 1, 128, [(8, 4)], 0.0, False),
    (40, 2, 128, [(8, 5), (16, 6), (8, 7), (8, 66), (8, 67), (8, 129), (8, 259)], 0.1, True),
    (1, 64, 4096, [(16, 4096)], 0.0, False),
    (2, 3, 256, [(24, 33)], 0.0, False),
    (16, 64, 1024, [(16, 300), (8, 40), (64, 17)], 0.0, False),
    (17, 2, 384, [(32, 255)], 0.3, False),
    (40, 5, 640, [(40, 129)], 0.5, True),
    (64, 1, 512, [(128, 100)], 0.0, False),
    (61, 1000, 256, [(16, 64), (16, 64)], 0.25, False),
    (100, 7, 2176, [(256, 70)], 0.1, True),
    (300, 4, 256, [(8, 514), (48, 257)], 0.1, True),
    (1000, 3, 512, [(64, 200)], 0.0, True),
    (130, 2, 128, [(8, 16), (16, 16), (24, 16), (32, 16), (64, 16), (72, 16), (128, 16), (136, 16)], 0.0, True),
])
def test_lora(qg, m, groups, k, mats, ybf16, drop, runs):
    note("lora m=%d groups=%d k=%d mats=%s ybf16=%s" % (m, groups, k, mats, ybf16))
    c = Case(qg, m, groups, k, mats, ybf16, 3 * m + k, drop, runs, scaled=m % 2 == 0)
    qg.lora_add(c.xd, c.groups, c.ad, c.ys)
    c.check()


def test_lora_no_rows_have_adapters(qg):
    note("lora with every row without an adapter")
    c = Case(qg, 40, 3, 256, [(16, 64)], False, 4, drop=1.1)
    qg.lora_add(c.xd, c.groups, c.ad, c.ys)
    c.check()


def test_lora_long_k(qg):
    note("lora with the largest k")
    for m in (3, 200):
        c = Case(qg, m, 2, qg.QG_BATCH_MAX_K, [(8, 48)], False, 6)
        qg.lora_add(c.xd, c.groups, c.ad, c.ys)
        c.check()


@pytest.mark.parametrize("m,groups,used,mats", [
    (1000, 256, 12, [(64, 300), (16, 64)]),  # a prompt of a few requests, many adapters loaded
    (1000, 1024, 1, [(16, 200)]),
    (70, 1024, 2, [(128, 130)]),
])
def test_lora_few_of_many_adapters(qg, m, groups, used, mats):
    note("lora m=%d, %d of %d adapters in use" % (m, used, groups))
    c = Case(qg, m, groups, 256, mats, False, 8, drop=0.1, runs=True)
    g = synth.rng(9)
    of = g.choice(groups, size=used, replace=False)
    c.ids = np.where(c.ids < 0, -1, np.sort(of[g.integers(0, used, m)])).astype(np.int32)
    c.groups = qg.group_rows(dev(c.ids), groups)
    qg.lora_add(c.xd, c.groups, c.ad, c.ys)
    c.check()


def test_lora_repeats_bit_for_bit(qg):
    note("lora twice on the same inputs")
    c = Case(qg, 90, 5, 1024, [(32, 200)], False, 7, runs=True)
    y = [t.clone() for t in c.ys]
    ws = torch.empty(qg.LoraLaunch(c.xd, c.groups, c.ad, y).nws, dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # its contents on entry do not matter
    qg.lora_add(c.xd, c.groups, c.ad, y, ws=ws)
    qg.lora_add(c.xd, c.groups, c.ad, c.ys)
    assert torch.equal(y[0], c.ys[0])
    c.check()


def test_lora_past_4_gib(qg):
    note("lora whose y and b pass 32-bit offsets")
    m, groups, k, r, n = 300, 9, 128, 256, 1000000
    x = torch.randn((m, k), device="cuda").bfloat16()
    a = torch.randn((groups, r, k), device="cuda").bfloat16()
    b = torch.zeros((groups, n, r), dtype=torch.bfloat16, device="cuda")
    cols = torch.tensor([0, 1, n // 2, n - 1], device="cuda")
    b[groups - 1, cols] = torch.randn((4, r), device="cuda").bfloat16()
    y = torch.zeros((m, n), dtype=torch.float32, device="cuda")
    plan = qg.group_rows(torch.full((m,), groups - 1, dtype=torch.int32, device="cuda"), groups)
    qg.lora_add(x, plan, [qg.LoraAdapters(a, b)], [y])
    v = x.double().cpu() @ a[groups - 1].double().cpu().t()
    bb = b[groups - 1, cols].double().cpu()
    want = (v @ bb.t()).numpy()
    tol = (bb.abs().sum(1) * TOL_F32 * v.abs().max()).numpy() + (r + 8) * 2 * HALF * (v.abs() @ bb.abs().t()).numpy()
    assert np.all(np.abs(host(y[:, cols]) - want) <= tol)
    assert int((y != 0).sum()) <= m * 4


def test_beside_a_shared_projection(qg):
    """A decode step's q, k, v: the shared W8A16 projections, then the
    adapters of all three in one call."""
    note("qgemv_batch_grouped then lora_add")
    g = synth.rng(12)
    m, k, ns = 11, 512, (512, 128, 128)
    ws = []
    for n in ns:
        q, s = qg.quantize_absmax(dev(synth.gaussian(g, (n, k), 0.02)), per_row=True)
        ws.append(qg.QWeight(qg.QG_WFMT_INT8, n, k, q, s))
    c = Case(qg, m, 6, k, [(16, n) for n in ns], False, 13, drop=0.3)
    base = qg.qgemv_batch_grouped(ws, c.xd)
    for j in range(3):
        c.y0[j] = host(base[j]).astype(np.float64)
        c.ys[j].copy_(base[j])
    qg.lora_add(c.xd, c.groups, c.ad, c.ys)
    c.check()


def test_stream_and_graph(qg):
    note("lora on another stream, captured and replayed")
    c = Case(qg, 48, 6, 512, [(16, 192), (32, 64)], False, 14, drop=0.2)
    y0 = [y.clone() for y in c.ys]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        qg.lora_add(c.xd, c.groups, c.ad, c.ys)
    st.synchronize()
    c.check()
    ys = [y.clone() for y in y0]
    launch = qg.LoraLaunch(c.xd, c.groups, c.ad, ys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        launch.launch()
    for seed in (1, 2, 3):
        c.xd.copy_(bf16(synth.rng(seed), (48, 512), 1.0)[0])
        for y, z in zip(ys, y0):
            y.copy_(z)
        graph.replay()
        torch.cuda.synchronize()
        want = [y.clone() for y in y0]
        qg.lora_add(c.xd, c.groups, c.ad, want)
        assert all(torch.equal(a, b) for a, b in zip(ys, want))


def test_launch_keeps_its_tensors(qg):
    note("an adapter's fields set anew after the launch object was made")
    c = Case(qg, 24, 3, 256, [(16, 96)], False, 15)
    launch = qg.LoraLaunch(c.xd, c.groups, c.ad, c.ys)
    ad = c.ad[0]
    shapes = [(ad.a.shape, ad.a.dtype), (ad.b.shape, ad.b.dtype), (ad.scale.shape, ad.scale.dtype)] \
        if ad.scale is not None else [(ad.a.shape, ad.a.dtype), (ad.b.shape, ad.b.dtype)]
    ad.a = ad.b = ad.scale = None
    others = [torch.full(s, 7.0, dtype=d, device="cuda") for s, d in shapes for _ in range(4)]
    launch.launch()
    torch.cuda.synchronize()
    c.check()
    del others


def test_launch_on_another_stream_and_dropped(qg):
    note("a launch object used on another stream than its own, dropped while its kernels wait")
    c = Case(qg, 300, 4, 1024, [(32, 260), (16, 96)], False, 18, runs=True)
    launch = qg.LoraLaunch(c.xd, c.groups, c.ad, c.ys)
    size = launch.nws
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    m = torch.zeros((4096, 4096), device="cuda")
    with torch.cuda.stream(st):
        for _ in range(20):  # the launch waits behind these
            torch.mm(m, m)
        launch.launch()
    del launch
    # the first stream's next tensors of that size: none may be the workspace
    others = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((t == 0x5A).all()) for t in others)
    c.check()


def test_values_that_are_not_finite_stay_in_their_rows(qg):
    note("NaN and infinities in x and B")
    m, k, n = 40, 256, 70
    c = Case(qg, m, 3, k, [(24, n)], False, 16, drop=0.3)
    with_a = np.flatnonzero(c.ids >= 0)
    without = np.flatnonzero(c.ids < 0)
    c.xd[int(with_a[0]), 5] = float("nan")
    c.xd[int(with_a[1]), 6] = float("inf")
    c.xd[int(without[0]), 7] = float("nan")
    g = int(c.ids[with_a[2]])
    c.ad[0].b[g, 11, 3] = float("inf")
    qg.lora_add(c.xd, c.groups, c.ad, c.ys)
    got = host(c.ys[0])
    want, tol = c.want(0)
    odd = np.zeros((m, n), bool)
    odd[with_a[:2]] = True
    odd[c.ids == g, 11] = True
    assert np.all(np.isnan(got[odd]))
    assert np.all(np.abs(got[~odd] - want[~odd]) <= tol[~odd])


@pytest.mark.parametrize("ybf16", [False, True])
def test_nan_scales_reach_y(qg, ybf16):
    """Also those whose upper half a rounding by adding to the bits carries
    over into a zero."""
    note("NaN of every payload in the adapters' scales, ybf16=%s" % ybf16)
    nans = np.array([0x7FFFFFFF, 0xFFFFFFFF, 0x7FFF8000, 0x7FC00000], np.uint32).view(np.float32)
    for m in (40, 600):
        c = Case(qg, m, 6, 256, [(24, 70)], ybf16, 20, drop=0.2)
        c.ad[0].scale[1:5] = dev(nans)
        qg.lora_add(c.xd, c.groups, c.ad, c.ys)
        assert np.array_equal(np.isnan(bf16_to_f64(host(c.ys[0])) if ybf16 else host(c.ys[0])),
                              np.repeat(((c.ids >= 1) & (c.ids < 5))[:, None], 70, axis=1))


def test_refusals(qg):
    c = Case(qg, 8, 4, 256, [(16, 32)], False, 1)
    x, gr, ad, ys = c.xd, c.groups, c.ad, c.ys
    for bad in (x.float(), x[:, :128], x[:7]):
        with pytest.raises(ValueError):
            qg.lora_add(bad, gr, ad, ys)
    with pytest.raises(ValueError):
        qg.lora_add(x, gr, ad, [ys[0][:, :16].contiguous()])
    with pytest.raises(ValueError):
        qg.lora_add(x, gr, ad * 9, ys * 9)
    with pytest.raises(ValueError):
        qg.lora_add(x, gr, ad, [ys[0].half()])
    with pytest.raises(ValueError):
        qg.LoraAdapters(ad[0].a, ad[0].b[:, :, :8].contiguous())
    with pytest.raises(qg.QgError):
        qg.lora_add(x, gr, [qg.LoraAdapters(ad[0].a[:, :12].contiguous(), ad[0].b[:, :, :12].contiguous())], ys)
    with pytest.raises(qg.QgError):
        qg.lora_add(x, gr, ad * 2, ys * 2)
    with pytest.raises(qg.QgError):
        qg.lora_add(x, gr, ad, ys, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qg.QgError):
        qg.lora_add(x, qg.RowGroups(gr.offsets, gr.order, gr.pos, 2), ad, ys)
