"""GPU row plans and router (qg_group_rows, qg_moe_route) against the oracle.

ids, offsets, order and pos must match exactly.  Weights: d = l - max is one
fp32 rounding (relative error of exp: |d| 2^-24, of the sum the same at
most), exp and the division add a few ulp, a sum of E terms at most
log2(64) + E / 64 roundings: with |d| <= 40 where it matters
(exp(-40) = 4e-18 times the largest), 160 half steps of 2^-24 bound the
relative error; smaller weights are held to an absolute 1e-17."""
import sys

import numpy as np
import pytest
import torch

from gpu_util import dev, dev_bf16, host
from oracle import rows as R
import synth

pytestmark = pytest.mark.gpu
RTOL_W, ATOL_W = 160 * 2.0 ** -24, 1e-17


def note(msg):
    print("[case] " + msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantized_gemv_amd as q
    q.lib()
    return q


def plan_fast(ids, groups):
    """The oracle's plan by a stable numpy sort (for long inputs)."""
    key = np.where((ids >= 0) & (ids < groups), ids, groups)
    order = np.argsort(key, kind="stable").astype(np.int32)
    offsets = np.concatenate(([0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups]))).astype(np.int32)
    pos = np.empty(len(ids), np.int32)
    pos[order] = np.arange(len(ids))
    pos[key == groups] = -1
    order[offsets[-1]:] = -1
    return offsets, order, pos


def check_plan(plan, offsets, order, pos):
    assert np.array_equal(host(plan.offsets), offsets)
    assert np.array_equal(host(plan.order), order)
    assert np.array_equal(host(plan.pos), pos)


@pytest.mark.parametrize("rows,groups", [(1, 1), (1, 1024), (2, 3), (63, 5), (64, 64), (65, 2), (511, 129), (2047, 1000),
                                         (2048, 8), (2049, 8), (4096, 1024), (5000, 1), (70001, 77), (131072 + 5, 128),
                                         (300001, 1024), (5000003, 1000)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_group_rows(qg, rows, groups, drop):
    note("group_rows %d rows, %d groups, drop %g" % (rows, groups, drop))
    g = synth.rng(rows + groups)
    ids = g.integers(0, groups, rows).astype(np.int32)
    # ids without a group: -1, the first one past the end, extremes
    bad = np.array([-1, groups, 2**31 - 1, -2**31], np.int32)
    ids = np.where(g.random(rows) < drop, bad[g.integers(0, 4, rows)], ids).astype(np.int32)
    want = R.group_rows(ids, groups) if rows * groups < 200000 else plan_fast(ids, groups)
    assert all(np.array_equal(a, b) for a, b in zip(want, plan_fast(ids, groups)))
    check_plan(qg.group_rows(dev(ids), groups), *want)


def test_group_rows_most(qg):
    """The longest plan there can be, checked on the device: places and rows
    are each other's inverse, sorted by id, equal ids in row order."""
    rows, groups = qg.QG_MAX_PLAN_ROWS, 1000
    note("group_rows of %d rows" % rows)
    ids = torch.randint(-3, groups + 3, (rows,), dtype=torch.int32, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(4))
    plan = qg.group_rows(ids, groups)
    count = torch.zeros(groups, dtype=torch.int64, device="cuda")
    piece = 1 << 27
    for lo in range(0, rows, piece):
        part = ids[lo:lo + piece]
        inside = (part >= 0) & (part < groups)
        count += torch.bincount(part[inside], minlength=groups)
        pos = plan.pos[lo:lo + piece]
        assert torch.equal(pos >= 0, inside)
        back = plan.order[pos.clamp(min=0).long()]
        assert bool((back == torch.arange(lo, lo + part.numel(), dtype=torch.int32, device="cuda"))[inside].all())
    assert torch.equal(plan.offsets[1:].long(), torch.cumsum(count, 0)) and int(plan.offsets[0]) == 0
    live = int(plan.offsets[-1])
    assert bool((plan.order[live:] == -1).all())
    for lo in range(0, live - 1, piece):
        order = plan.order[lo:min(lo + piece + 1, live)]
        of = ids[order.long()]
        assert bool(((of[1:] > of[:-1]) | ((of[1:] == of[:-1]) & (order[1:] > order[:-1]))).all())


def test_group_rows_one_group_holds_all_and_none(qg):
    note("group_rows all equal / all dropped")
    for v in (3, -1):
        ids = np.full(9000, v, np.int32)
        check_plan(qg.group_rows(dev(ids), 7), *plan_fast(ids, 7))


def test_group_rows_of_another_router(qg):
    note("group_rows of ids [tokens][top_k]")
    ids = synth.rng(6).integers(-1, 9, (50, 3)).astype(np.int32)
    plan = qg.group_rows(dev(ids), 9)
    check_plan(plan, *plan_fast(ids.reshape(-1), 9))
    assert plan.per_row == 3
    with pytest.raises(ValueError):
        qg.group_rows(dev(ids.reshape(5, 10, 3)), 9)


def test_group_rows_reused_buffers(qg):
    note("group_rows into given buffers and workspace, a smaller input after a larger one")
    g = synth.rng(5)
    ws = torch.empty(qg.lib().qg_group_rows_workspace_bytes(10000, 33), dtype=torch.uint8, device="cuda")
    for rows in (10000, 10000, 4097):
        ids = g.integers(-1, 33, rows).astype(np.int32)
        out = qg.group_rows(dev(np.zeros(rows, np.int32)), 33)
        check_plan(qg.group_rows(dev(ids), 33, out=out, ws=ws), *plan_fast(ids, 33))
    with pytest.raises(ValueError):
        qg.group_rows(dev(ids), 32, out=out)
    with pytest.raises(ValueError):
        qg.group_rows(dev(ids[:100]), 33, out=out)


def logits_case(t, e, bf16, seed, masked=0.0):
    g = synth.rng(seed)
    l = synth.gaussian(g, (t, e), 3.0)
    # ties: a quarter of the values from a coarse grid, +0 and -0 among them
    grid = np.array([-1.0, -0.0, 0.0, 1.0, 2.0], np.float32)
    l = np.where(g.random((t, e)) < 0.25, grid[g.integers(0, 5, (t, e))], l)
    l = np.where(g.random((t, e)) < masked, np.float32(-np.inf), l).astype(np.float32)
    if bf16:
        bits = synth.to_bf16_bits(l)
        return dev_bf16(bits), synth.bf16_bits_to_f32(bits)
    return dev(l), l


def route_fast(l, top_k, renorm):
    """The oracle's router by a stable numpy sort (for many finite tokens)."""
    l = l.astype(np.float64)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :top_k].astype(np.int32)
    p = np.exp(l - l.max(1, keepdims=True))
    w = np.take_along_axis(p, ids.astype(np.int64), 1)
    return ids, w / (w if renorm else p).sum(1, keepdims=True)


def check_route(qg, x, l, top_k, renorm, out=None):
    ids, w = R.moe_route(l, top_k, renorm) if l.shape[0] <= 3000 else route_fast(l, top_k, renorm)
    r = qg.moe_route(x, top_k, renorm, out=out)
    assert np.array_equal(host(r.ids), ids)
    assert np.allclose(host(r.weights), w, rtol=RTOL_W, atol=ATOL_W)
    check_plan(r.groups, *plan_fast(ids.reshape(-1), l.shape[1]))
    return r


@pytest.mark.parametrize("t,e,top_k", [(1, 1, 1), (1, 8, 2), (3, 64, 8), (16, 64, 8), (5, 65, 16), (33, 128, 6),
                                       (64, 129, 8), (100, 256, 1), (7, 257, 5), (20, 1024, 16), (257, 60, 4),
                                       (700, 96, 8), (70001, 8, 2), (2048, 16, 1), (2049, 16, 1), (65, 40, 16)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route(qg, t, e, top_k, bf16, renorm):
    note("route t=%d e=%d top=%d bf16=%s renorm=%s" % (t, e, top_k, bf16, renorm))
    x, l = logits_case(t, e, bf16, 7 * t + e)
    check_route(qg, x, l, top_k, renorm)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_masked(qg, renorm):
    note("route with masked experts")
    for t, e, top_k, masked in ((40, 16, 8, 0.6), (3000, 24, 4, 0.9), (9, 300, 16, 0.99)):
        x, l = logits_case(t, e, False, e, masked)
        l[0] = -np.inf                                   # nothing left
        if t > 3:
            l[1] = np.nan
            l[2, :] = -np.finfo(np.float32).max           # the lowest value masks nothing by itself
            l[3] = -np.inf
            l[3, e - 1] = 5.0
        l[-1, 0] = np.inf
        l[-1, 1:3] = np.nan
        check_route(qg, dev(l), l, top_k, renorm)


def test_route_large_range(qg):
    note("route with a large range of logits")
    l = np.array([[-3e38, 3e38, 0.0, 1e-40, -1e-40, 80.0, -80.0, 3e38]], np.float32)
    for renorm in (False, True):
        check_route(qg, dev(l), l, 8, renorm)


def test_route_reuse_stream_and_graph(qg):
    note("route into given buffers on another stream, captured and replayed")
    for t, e, top_k in ((16, 64, 8), (1000, 64, 8)):
        x, l = logits_case(t, e, False, 3)
        out = check_route(qg, x, l, top_k, True)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            qg.moe_route(x, top_k, True, out=out)
        st.synchronize()
        ws = torch.empty(max(1, qg.lib().qg_group_rows_workspace_bytes(t * top_k, e)), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qg.moe_route(x, top_k, True, out=out, ws=ws)
        for seed in (11, 12, 13):
            y, l = logits_case(t, e, False, seed)
            x.copy_(y)
            graph.replay()
            ids, w = R.moe_route(l, top_k, True)
            assert np.array_equal(host(out.ids), ids)
            assert np.allclose(host(out.weights), w, rtol=RTOL_W, atol=ATOL_W)
            check_plan(out.groups, *plan_fast(ids.reshape(-1), e))
            check_route(qg, x, l, top_k, True)


def test_route_refusals(qg):
    x = torch.zeros((4, 8), device="cuda")
    with pytest.raises(qg.QgError):
        qg.moe_route(x, 9)
    with pytest.raises(qg.QgError):
        qg.moe_route(torch.zeros((1, 64), device="cuda"), 17)
    with pytest.raises(ValueError):
        qg.moe_route(x.half(), 2)
    with pytest.raises(ValueError):
        qg.moe_route(x[:, ::2], 2)
    with pytest.raises(ValueError):
        qg.moe_route(x[0], 2)
    with pytest.raises(ValueError):
        qg.group_rows(torch.zeros(4, dtype=torch.int64, device="cuda"), 2)
