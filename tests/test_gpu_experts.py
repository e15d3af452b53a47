"""GPU expert products (qg_qgemm_experts, _swiglu, _combine) and the expert
feed-forward against the fp64 oracle on the same codes, scales and inputs.

Tolerances.  W8A16: exact products, fp32 sums of K terms; as for the other
W8A16 products, 1e-5 of the row's largest output (TOL_F32).  W8A8: int32 sums
are exact, so y carries the roundings of float(acc), the scales' product or
reciprocals, and the quotient: at most 8 half steps of 2^-24, elementwise.
SwiGLU: |silu'| <= 1.1, so its error is 1.1 |dg| |u| + |silu(g)| |du| plus 8
half steps for exp, sum, quotient and product.  Combine: the products' errors
times |w|, plus one rounding per slot.  bf16 outputs add half a step, 2^-8."""
import sys

import numpy as np
import pytest
import torch

from gpu_util import TOL_F32, bf16_to_f64, dev, dev_bf16, f32_to_bf16_rne, host
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


class Case:
    """Codes, scales, activations and a plan on both sides."""

    def __init__(self, qg, t, e, top, k, n, act8, tiled, seed, mats=1, spread="even", drop=0.0, gather=True):
        g = synth.rng(seed)
        self.t, self.e, self.top, self.k, self.n, self.act8, self.gather = t, e, top, k, n, act8, gather
        if spread == "even":
            ids = np.stack([g.permutation(e)[:top] for _ in range(t)])
        elif spread == "one":            # every token's first slot the same expert
            ids = np.stack([np.roll(np.arange(e), -(e // 2))[:top] for _ in range(t)])
        else:                            # skewed: expert j with weight 1 / (1 + j)^2
            p = 1.0 / (1 + np.arange(e)) ** 2
            ids = np.stack([g.choice(e, size=top, replace=False, p=p / p.sum()) for _ in range(t)])
        ids = np.where(g.random(ids.shape) < drop, -1, ids).astype(np.int32)
        self.offsets, self.order, self.pos = R.group_rows(ids, e)
        self.live = int(self.offsets[-1])
        self.weights = g.random((t, top)).astype(np.float32)
        rows = t if gather else t * top
        if act8:
            self.x = g.integers(-127, 128, (rows, k)).astype(np.int8)
            self.s_x = (20 + 40 * g.random(rows)).astype(np.float32)
            self.xd, self.sxd = dev(self.x), dev(self.s_x)
        else:
            bits = synth.to_bf16_bits(synth.gaussian(g, (rows, k), 1.0))
            self.x, self.s_x = synth.bf16_bits_to_f32(bits), None
            self.xd, self.sxd = dev_bf16(bits), None
        self.codes = [g.integers(-127, 128, (e, n, k)).astype(np.int8) for _ in range(mats)]
        # products of about unit size
        unit = 73.0 * np.sqrt(k)
        self.scale = [(unit * (0.5 + g.random((e, n)))).astype(np.float32) for _ in range(mats)]
        self.w = []
        for c, s in zip(self.codes, self.scale):
            w = qg.QExperts(qg.QG_WFMT_INT8, e, n, k, dev(c), dev(s))
            self.w.append(qg.tiled16_experts(w) if tiled else w)
        self.groups = qg.RowGroups(dev(self.offsets), dev(self.order), dev(self.pos), top)

    def products(self, j=0):
        """(y, tolerance) of matrix j, live rows only."""
        y = R.y_experts(self.codes[j], self.scale[j], self.x, self.offsets, self.order if self.gather else None,
                        self.top, self.s_x)[:self.live]
        if self.act8:
            return y, 8 * HALF * np.abs(y)
        return y, np.repeat(TOL_F32 * np.abs(y).max(axis=1, keepdims=True), self.n, axis=1) if self.live else y

    def swiglu(self):
        (g, dg), (u, du) = self.products(0), self.products(1)
        y = R.y_swiglu(g, u)
        silu = R.y_swiglu(g, np.ones_like(g))
        return y, 1.1 * dg * np.abs(u) + np.abs(silu) * du + 8 * HALF * np.abs(y)

    def combine(self):
        y, dy = self.products()
        out = R.y_combine(y, self.pos, self.weights)
        tol = R.y_combine(dy, self.pos, self.weights) + self.top * HALF * R.y_combine(np.abs(y), self.pos, self.weights)
        return out, tol


def out_buffer(rows, n, bf16, guard=64):
    full = torch.empty(rows * n + 2 * guard, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    full.view(torch.uint8).fill_(0x5A)
    return full, full[guard:guard + rows * n].view(rows, n)


def check(full, y, live, want, tol, bf16, guard=64):
    """Rows below `live` within tolerance; the rest and the guards untouched."""
    raw = full.view(torch.uint8).cpu().numpy()
    isz = full.dtype.itemsize
    n = y.shape[1]
    assert np.all(raw[:guard * isz] == 0x5A) and np.all(raw[(guard + live * n) * isz:] == 0x5A), "written outside"
    got = host(y)[:live]
    got = bf16_to_f64(got) if bf16 else got.astype(np.float64)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    bad = np.abs(got - want) - (tol + 1e-37)
    assert np.all(bad <= 0), "off by up to %g at %s" % (bad.max(), np.unravel_index(np.argmax(bad), bad.shape))


SIZES = [  # t, e, top, k, n, spread, drop
    (1, 1, 1, 128, 1, "even", 0.0),
    (9, 2, 2, 128, 3, "even", 0.2),
    (9, 5, 3, 1152, 6, "skew", 0.2),
    (1, 8, 2, 256, 40, "even", 0.0),
    (2, 3, 1, 128, 16, "even", 0.5),
    (5, 4, 4, 384, 33, "even", 0.2),
    (16, 64, 8, 256, 96, "even", 0.0),
    (15, 2, 1, 512, 130, "one", 0.0),
    (16, 2, 1, 512, 128, "one", 0.0),
    (17, 5, 2, 640, 129, "one", 0.0),
    (33, 9, 3, 1024, 257, "skew", 0.1),
    (64, 8, 2, 512, 200, "skew", 0.0),
    (100, 16, 4, 384, 511, "skew", 0.1),
    (130, 4, 2, 2176, 300, "even", 0.0),
    (257, 3, 2, 256, 384, "one", 0.0),
    (300, 70, 1, 128, 64, "skew", 0.0),
    (600, 6, 2, 512, 520, "skew", 0.05),
    (1100, 4, 1, 256, 272, "one", 0.0),
    # enough tiles to fill the card with few rows per expert
    (80, 64, 8, 256, 1030, "skew", 0.0),
    (200, 33, 4, 384, 2050, "skew", 0.1),
    (150, 40, 6, 128, 1537, "even", 0.02),
    # many rows, too few 128-row tiles to fill the card
    (500, 5, 3, 640, 440, "skew", 0.0),
    (333, 30, 5, 256, 391, "skew", 0.1),
    # the most slots per token; more experts than a wave has lanes, many empty
    (21, 20, 16, 128, 70, "even", 0.1),
    (300, 1024, 3, 128, 18, "even", 0.0),
]


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_experts(qg, size, act8, tiled):
    t, e, top, k, n, spread, drop = size
    bf16 = (t + n) % 2 == 1
    note("experts %s act8=%s tiled=%s bf16=%s" % (size, act8, tiled, bf16))
    c = Case(qg, t, e, top, k, n, act8, tiled, 31 * t + n, spread=spread, drop=drop)
    full, y = out_buffer(t * top, n, bf16)
    qg.qgemm_experts(c.w[0], c.xd, c.groups, s_x=c.sxd, y=y)
    check(full, y, c.live, *c.products(), bf16)
    # the same call again gives the same bits
    z = torch.full_like(y, 7.0)
    qg.qgemm_experts(c.w[0], c.xd, c.groups, s_x=c.sxd, y=z)
    assert torch.equal(y[:c.live], z[:c.live]) and bool((z[c.live:] == 7.0).all())


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_swiglu(qg, size, act8, tiled):
    t, e, top, k, n, spread, drop = size
    bf16 = (t + n) % 2 == 0
    note("swiglu %s act8=%s tiled=%s bf16=%s" % (size, act8, tiled, bf16))
    c = Case(qg, t, e, top, k, n, act8, tiled, 37 * t + n, mats=2, spread=spread, drop=drop)
    full, y = out_buffer(t * top, n, bf16)
    qg.qgemm_experts_swiglu(c.w[0], c.w[1], c.xd, c.groups, s_x=c.sxd, y=y)
    check(full, y, c.live, *c.swiglu(), bf16)


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_combine(qg, size, act8, gather):
    t, e, top, k, n, spread, drop = size
    bf16, tiled = (t + n) % 2 == 0, t % 2 == 0
    note("combine %s act8=%s gather=%s tiled=%s bf16=%s" % (size, act8, gather, tiled, bf16))
    c = Case(qg, t, e, top, k, n, act8, tiled, 41 * t + n, spread=spread, drop=drop, gather=gather)
    full, y = out_buffer(t, n, bf16)
    qg.qgemm_experts_combine(c.w[0], c.xd, c.groups, dev(c.weights), s_x=c.sxd, gather=gather, y=y)
    check(full, y, t, *c.combine(), bf16)


def test_all_rows_dropped(qg):
    note("experts with every row dropped")
    for act8 in (False, True):
        c = Case(qg, 20, 4, 2, 256, 70, act8, True, 3, drop=1.1)
        assert c.live == 0
        full, y = out_buffer(40, 70, False)
        qg.qgemm_experts(c.w[0], c.xd, c.groups, s_x=c.sxd, y=y)
        torch.cuda.synchronize()
        assert bool((full.view(torch.uint8) == 0x5A).all())
        out = qg.qgemm_experts_combine(c.w[0], c.xd, c.groups, dev(c.weights), s_x=c.sxd, gather=True)
        assert not host(out).any()


def test_large_gates(qg):
    note("swiglu with gates far from zero")
    c = Case(qg, 40, 3, 1, 256, 64, False, True, 5, mats=2)
    c.scale[0][:] = 1.0  # gates of several thousand, both signs
    c.w[0].scale.copy_(dev(c.scale[0]))
    full, y = out_buffer(40, 64, False)
    qg.qgemm_experts_swiglu(c.w[0], c.w[1], c.xd, c.groups, y=y)
    check(full, y, c.live, *c.swiglu(), False)


def test_non_finite_rows_stay_alone(qg):
    note("a row of infinities and NaN spoils no other row")
    for t, e in ((16, 2), (600, 2)):
        c = Case(qg, t, e, 1, 256, 96, False, True, 8, spread="one")
        y0 = host(qg.qgemm_experts(c.w[0], c.xd, c.groups))
        c.xd[3] = float("nan")
        c.xd[7, 5] = float("inf")
        y1 = host(qg.qgemm_experts(c.w[0], c.xd, c.groups))
        rows = np.isin(c.order, [3, 7])
        assert np.array_equal(y0[~rows], y1[~rows]) and not np.isfinite(y1[c.order == 3]).any()


# fp32 NaN whose upper half a rounding by adding to the bits carries over into
# a zero of either sign
NANS = np.array([0x7FFFFFFF, 0xFFFFFFFF, 0x7FFF8000, 0x7FC00000], np.uint32).view(np.float32)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("act8", [False, True])
def test_nan_scales_and_weights_reach_y(qg, act8, bf16):
    note("NaN of every payload in scales and weights, act8=%s bf16=%s" % (act8, bf16))
    dt = torch.bfloat16 if bf16 else torch.float32
    for t, e, n in ((16, 2, 96), (600, 2, 520)):  # streams, tiles
        c = Case(qg, t, e, 1, 256, n, act8, True, 8, mats=2, gather=True)
        c.scale[0][:, 5:9] = NANS
        c.w[0].scale.copy_(dev(c.scale[0]))
        for y in (qg.qgemm_experts(c.w[0], c.xd, c.groups, s_x=c.sxd, y_dtype=dt),
                  qg.qgemm_experts_swiglu(c.w[0], c.w[1], c.xd, c.groups, s_x=c.sxd, y_dtype=dt)):
            odd = torch.isnan(y).cpu().numpy()
            assert odd[:, 5:9].all() and not odd[:, :5].any() and not odd[:, 9:].any()
        c.weights[3:7, 0] = NANS
        y = qg.qgemm_experts_combine(c.w[1], c.xd, c.groups, dev(c.weights), s_x=c.sxd, gather=True, y_dtype=dt)
        odd = torch.isnan(y).cpu().numpy()
        assert odd[3:7].all() and not odd[:3].any() and not odd[7:].any()


def test_bf16_outputs_are_rounded_to_nearest_even(qg):
    """Any fp32 value through a combine of products that are exactly 1."""
    note("bf16 rounding of many fp32 values")
    t = 1 << 16
    bits = synth.rng(19).integers(0, 1 << 32, t, dtype=np.uint64).astype(np.uint32)
    # halves (to even, both ways), their neighbours, the least and the largest values
    edge = [h + d for h in (0x3F808000, 0x3F818000, 0x00008000, 0x00018000, 0x7F7F8000, 0x007F8000) for d in (-1, 0, 1)]
    edge += [0, 1, 0x007FFFFF, 0x00800000, 0x7F7FFFFF, 0x7F800000]
    edge = np.array(edge + [e | 0x80000000 for e in edge], np.uint32)
    bits[:len(edge)] = edge
    w = bits.view(np.float32)
    x = torch.zeros((t, 128), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    codes = torch.zeros((1, 4, 128), dtype=torch.int8, device="cuda")
    codes[:, :, 0] = 1
    one = qg.QExperts(qg.QG_WFMT_INT8, 1, 4, 128, codes, torch.ones((1, 4), device="cuda"))
    plan = qg.group_rows(torch.zeros((t, 1), dtype=torch.int32, device="cuda"), 1)
    y = host(qg.qgemm_experts_combine(one, x, plan, dev(w.reshape(t, 1)), gather=True, y_dtype=torch.bfloat16))
    nan = np.isnan(w)
    with np.errstate(invalid="ignore"):
        want = f32_to_bf16_rne(w + np.float32(0))  # a sum that starts at +0: no -0
    assert np.array_equal(y[~nan], np.repeat(want[~nan, None], 4, axis=1))
    assert np.isnan(bf16_to_f64(y[nan])).all() and nan.sum() > 100


def test_long_k(qg):
    note("experts with the largest k of each mode")
    for k, act8 in ((qg.QG_BATCH_MAX_K, False), (qg.QG_QGEMM_MAX_K, True)):
        for t in (3, 200):
            c = Case(qg, t, 2, 1, k, 40, act8, t == 3, 9)
            full, y = out_buffer(t, 40, False)
            qg.qgemm_experts(c.w[0], c.xd, c.groups, s_x=c.sxd, y=y)
            check(full, y, c.live, *c.products(), False)


def test_weights_past_4_gib(qg):
    note("experts whose codes and outputs pass 32-bit offsets")
    # 5 experts of 1.07e9 codes: only the last ones are written, the rest stays zero
    e, n, k = 5, 262144, 4096
    codes = torch.zeros((e, n, k), dtype=torch.int8, device="cuda")
    g = synth.rng(10)
    rows = np.array([0, 1, n // 2, n - 1])
    vals = g.integers(-127, 128, (len(rows), k)).astype(np.int8)
    codes[e - 1, torch.from_numpy(rows).cuda()] = dev(vals)
    scale = torch.full((e, n), 2000.0, device="cuda")
    w = qg.QExperts(qg.QG_WFMT_INT8, e, n, k, codes, scale)
    for t in (3, 200):
        bits = synth.to_bf16_bits(synth.gaussian(g, (t, k), 1.0))
        plan = qg.group_rows(torch.full((t,), e - 1, dtype=torch.int32, device="cuda"), e)
        y = qg.qgemm_experts(w, dev_bf16(bits), plan)
        got = y[:, torch.from_numpy(rows).cuda()]
        want = synth.bf16_bits_to_f32(bits).astype(np.float64) @ vals.astype(np.float64).T / 2000.0
        assert np.abs(host(got) - want).max() <= TOL_F32 * np.abs(want).max()
        assert int((y != 0).sum()) <= t * len(rows)
        del y, got


def test_x_past_4_gib(qg):
    note("an x that passes 32-bit offsets")
    k, rows = 262144, 8500
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    g = synth.rng(11)
    at = [0, 17, 8191, 8192, rows - 1]
    bits = synth.to_bf16_bits(synth.gaussian(g, (len(at), k), 1.0))
    x[torch.tensor(at, device="cuda")] = dev_bf16(bits)
    codes = g.integers(-127, 128, (1, 16, k)).astype(np.int8)
    w = qg.QExperts(qg.QG_WFMT_INT8, 1, 16, k, dev(codes), torch.full((1, 16), 30000.0, device="cuda"))
    plan = qg.group_rows(torch.zeros(rows, dtype=torch.int32, device="cuda"), 1)
    y = host(qg.qgemm_experts(w, x, plan))
    want = synth.bf16_bits_to_f32(bits).astype(np.float64) @ codes[0].astype(np.float64).T / 30000.0
    assert np.abs(y[at] - want).max() <= TOL_F32 * np.abs(want).max()
    rest = np.ones(rows, bool)
    rest[at] = False
    assert not y[rest].any()


@pytest.mark.parametrize("n", [32, 600])  # 32-row and 128-row tiles
@pytest.mark.parametrize("act8", [False, True])
def test_tiles_read_x_just_below_4_gib(qg, act8, n):
    note("tiles over an x of almost 4 GiB, act8=%s n=%d" % (act8, n))
    k, rows, e = 131072, 32000 if act8 else 16000, 2
    x = torch.zeros((rows, k), dtype=torch.int8 if act8 else torch.bfloat16, device="cuda")
    g = synth.rng(13)
    at = np.array([0, rows // 4, rows // 2 - 1, rows // 2, 3 * rows // 4, rows - 2, rows - 1])
    if act8:
        vals = g.integers(-127, 128, (len(at), k)).astype(np.int8)
        x[torch.from_numpy(at).cuda()] = dev(vals)
    else:
        bits = synth.to_bf16_bits(synth.gaussian(g, (len(at), k), 1.0))
        vals = synth.bf16_bits_to_f32(bits)
        x[torch.from_numpy(at).cuda()] = dev_bf16(bits)
    codes = g.integers(-127, 128, (e, n, k)).astype(np.int8)
    w = qg.QExperts(qg.QG_WFMT_INT8, e, n, k, dev(codes), torch.full((e, n), 30000.0, device="cuda"))
    ids = g.integers(0, e, rows).astype(np.int32)
    plan = qg.group_rows(dev(ids), e)
    y = qg.qgemm_experts(w, x, plan, s_x=torch.ones(rows, device="cuda") if act8 else None)
    pos = host(plan.pos)
    got = host(y[torch.from_numpy(pos[at].astype(np.int64)).cuda()])
    for j, r in enumerate(at):
        want = vals[j].astype(np.float64) @ codes[ids[r]].astype(np.float64).T / 30000.0
        tol = 8 * HALF * np.abs(want) if act8 else TOL_F32 * np.abs(want).max()
        assert np.all(np.abs(got[j] - want) <= tol), "row %d" % r
    assert int((y != 0).any(1).sum()) == len(at)


def test_outputs_past_4_gib(qg):
    note("tiles and combine whose products pass 4 GiB")
    t, top, e, k, n = 20000, 2, 4, 128, 32768
    g = synth.rng(14)
    bits = synth.to_bf16_bits(synth.gaussian(g, (t, k), 1.0))
    x = synth.bf16_bits_to_f32(bits).astype(np.float64)
    codes = g.integers(-127, 128, (e, n, k)).astype(np.int8)
    w = qg.QExperts(qg.QG_WFMT_INT8, e, n, k, dev(codes), torch.full((e, n), 800.0, device="cuda"))
    ids = np.stack([g.permutation(e)[:top] for _ in range(t)]).astype(np.int32)
    wt = g.random((t, top)).astype(np.float32)
    plan = qg.group_rows(dev(ids), e)
    y = qg.qgemm_experts(w, dev_bf16(bits), plan)
    out = qg.qgemm_experts_combine(w, dev_bf16(bits), plan, dev(wt), gather=True)
    pos = host(plan.pos).reshape(t, top)
    for r in (0, 1, t // 2, t - 2, t - 1, int(np.argmax(pos.max(1)))):
        rows = [x[r] @ codes[ids[r, j]].astype(np.float64).T / 800.0 for j in range(top)]
        for j in range(top):
            assert np.abs(host(y[int(pos[r, j])]) - rows[j]).max() <= TOL_F32 * np.abs(rows[j]).max()
        want = wt[r].astype(np.float64) @ np.array(rows)
        tol = wt[r].astype(np.float64) @ np.array([TOL_F32 * np.abs(v).max() + top * HALF * np.abs(v) for v in rows])
        assert np.all(np.abs(host(out[r]) - want) <= tol)


@pytest.mark.parametrize("t", [5, 400])
def test_the_same_expert_twice(qg, t):
    """A choice that names an expert twice for a token (another router's) adds
    both of its products."""
    note("the same expert in two slots, t=%d" % t)
    c = Case(qg, t, 4, 3, 256, 130, False, True, 17)
    ids = synth.rng(18).integers(0, 4, (t, 3)).astype(np.int32)
    ids[:, 1] = ids[:, 0]
    c.offsets, c.order, c.pos = R.group_rows(ids, 4)
    c.live = int(c.offsets[-1])
    c.groups = qg.group_rows(dev(ids), 4)
    full, y = out_buffer(t, 130, False)
    qg.qgemm_experts_combine(c.w[0], c.xd, c.groups, dev(c.weights), gather=True, y=y)
    check(full, y, t, *c.combine(), False)


def test_very_wide_matrix(qg):
    note("a matrix of more than 2^21 rows")
    n, k, t = 2100003, 128, 200
    g = synth.rng(12)
    at = [0, 1, n // 2, n - 17, n - 1]
    vals = g.integers(-127, 128, (len(at), k)).astype(np.int8)
    codes = torch.zeros((1, n, k), dtype=torch.int8, device="cuda")
    codes[0, torch.tensor(at, device="cuda")] = dev(vals)
    w = qg.QExperts(qg.QG_WFMT_INT8, 1, n, k, codes, torch.full((1, n), 700.0, device="cuda"))
    bits = synth.to_bf16_bits(synth.gaussian(g, (t, k), 1.0))
    plan = qg.group_rows(torch.zeros(t, dtype=torch.int32, device="cuda"), 1)
    y = qg.qgemm_experts(w, dev_bf16(bits), plan)
    want = synth.bf16_bits_to_f32(bits).astype(np.float64) @ vals.astype(np.float64).T / 700.0
    assert np.abs(host(y[:, torch.tensor(at, device="cuda")]) - want).max() <= TOL_F32 * np.abs(want).max()
    assert int((y != 0).sum()) <= t * len(at)


def test_two_streams_at_once(qg):
    note("two combine calls on two streams")
    c = [Case(qg, 64, 8, 2, 512, 200, act8, True, 60, spread="skew", gather=False) for act8 in (False, True)]
    st = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for j in (0, 1):
            with torch.cuda.stream(st[j]):
                outs.append((j, qg.qgemm_experts_combine(c[j].w[0], c[j].xd, c[j].groups, dev(c[j].weights), s_x=c[j].sxd)))
    torch.cuda.synchronize()
    for j, y in outs:
        want, tol = c[j].combine()
        assert np.all(np.abs(host(y) - want) <= tol + 1e-37)


def test_stream_and_graph(qg):
    note("expert feed-forward on another stream, captured and replayed")
    for t, act8, f in ((4, False, 384), (300, True, 384), (1200, False, 2048), (1200, True, 2048)):
        g = synth.rng(t)
        e, top, k = 8, 2, 256
        gate, up, down = (qg.tiled16_experts(qg.quantize_experts(dev(synth.gaussian(g, s, 0.05))))
                          for s in ((e, f, k), (e, f, k), (e, k, f)))
        x = dev_bf16(synth.to_bf16_bits(synth.gaussian(g, (t, k), 1.0)))
        logits = dev(synth.gaussian(g, (t, e), 1.0))

        def step():
            return qg.moe_ffn(x, logits, gate, up, down, top, act_int8=act8, y_dtype=torch.float32)

        want = step().clone()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            other = step()
        st.synchronize()
        assert torch.equal(other, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step()
        for seed in (1, 2, 3):
            x.copy_(dev_bf16(synth.to_bf16_bits(synth.gaussian(synth.rng(seed), (t, k), 1.0))))
            logits.copy_(dev(synth.gaussian(synth.rng(seed + 9), (t, e), 1.0)))
            graph.replay()
            torch.cuda.synchronize()
            got = y.clone()
            assert torch.equal(got, step())


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("t", [1, 13, 200])
def test_ffn(qg, t, act8):
    """The whole feed-forward against the oracle's stages, each stage checked
    on the tensors the stage before it gave (so its own tolerance applies)."""
    note("moe_ffn t=%d act8=%s" % (t, act8))
    g = synth.rng(50 + t)
    e, top, k, f = 12, 3, 512, 640
    ws = [qg.quantize_experts(dev(synth.gaussian(g, s, 0.05))) for s in ((e, f, k), (e, f, k), (e, k, f))]
    bits = synth.to_bf16_bits(synth.gaussian(g, (t, k), 1.0))
    l = synth.gaussian(g, (t, e), 1.0)
    l[0, : e - 1] = -np.inf  # one expert left for the first token
    y = host(qg.moe_ffn(dev_bf16(bits), dev(l), *ws, top, act_int8=act8, y_dtype=torch.float32))
    r = qg.moe_route(dev(l), top)
    ids, w = R.moe_route(l, top, True)
    assert np.array_equal(host(r.ids), ids)
    plan = R.group_rows(ids, e)
    xd, s_x, s_h = dev_bf16(bits), None, None
    if act8:
        xd, s_x = qg.quantize_absmax(xd, per_row=True)
    h = qg.qgemm_experts_swiglu(ws[0], ws[1], xd, r.groups, s_x=s_x)
    hd = h
    if act8:
        hd, s_h = qg.quantize_absmax(h, per_row=True)
    hh = host(hd).astype(np.float64) if act8 else bf16_to_f64(host(hd))
    prod = R.y_experts(host(ws[2].codes), host(ws[2].scale), hh, plan[0], None, 1, None if s_h is None else host(s_h))
    want = R.y_combine(prod, plan[2], host(r.weights))
    assert np.abs(y - want).max() <= 2 * TOL_F32 * np.abs(prod[: plan[0][-1]]).max()


def test_refusals(qg):
    c = Case(qg, 8, 4, 2, 256, 32, False, False, 1, mats=2)
    x, gr, w = c.xd, c.groups, c.w[0]
    for bad in (x.float(), x[:, :128], x[:7], x.to(torch.int8), x.t()):
        with pytest.raises(ValueError):
            qg.qgemm_experts(w, bad, gr)
    with pytest.raises(ValueError):
        qg.qgemm_experts(w, x, gr, s_x=torch.ones(8, device="cuda"))
    with pytest.raises(ValueError):
        qg.qgemm_experts(w, x, gr, gather=False)
    with pytest.raises(ValueError):
        qg.qgemm_experts(w, x, qg.RowGroups(gr.offsets, gr.order, gr.pos, 0))
    with pytest.raises(ValueError):
        qg.qgemm_experts(w, x, gr, y_dtype=torch.float16)
    with pytest.raises(ValueError):
        qg.qgemm_experts(w, x, gr, y=torch.empty((15, 32), device="cuda"))
    with pytest.raises(ValueError):
        qg.qgemm_experts(w, x, qg.group_rows(torch.zeros(8, dtype=torch.int32, device="cuda"), 3))
    with pytest.raises(ValueError):
        qg.QExperts(qg.QG_WFMT_INT8_T16, 4, 33, 256, w.codes, w.scale)
    with pytest.raises(ValueError):
        qg.qgemm_experts_combine(w, x, gr, torch.ones(15, device="cuda"), gather=True)
    with pytest.raises(qg.QgError):
        qg.qgemm_experts_swiglu(w, qg.tiled16_experts(c.w[1]), x, gr)
    with pytest.raises(qg.QgError):
        qg.qgemm_experts_combine(w, x, gr, dev(c.weights), gather=True,
                                 ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
