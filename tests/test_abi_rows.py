"""Host-side checks of the row-dependent products' entry points (CPU only):
argument validation returns the documented status codes and launches
nothing, and the binding refuses tensors that do not fit."""
import ctypes

import pytest
import torch

A, U = 4096, 4097  # a 16-B aligned fake address, and a misaligned one
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                  reason="passes fake device addresses; runs where no GPU is visible")
NULLPTR, SHAPE, ALIGN, ARG, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def qg():
    import os

    import quantized_gemv_amd as q
    if not os.path.exists(q.LIB_PATH):
        from quantized_gemv_amd.build import build
        build()
    return q


def groups(qg, **kw):
    a = dict(offsets=A, order=A, rows=32, groups=4, per_row=2)
    a.update(kw)
    return ctypes.byref(qg.CRowGroups(a["offsets"], a["order"], a["rows"], a["groups"], a["per_row"]))


def experts(qg, **kw):
    a = dict(fmt=qg.QG_WFMT_INT8, e=4, n=64, k=256, codes=A, scale=A)
    a.update(kw)
    return ctypes.byref(qg.CExperts(a["fmt"], 0, a["e"], a["n"], a["k"], a["codes"], a["scale"]))


def test_workspace_sizes(qg):
    f = qg.lib().qg_group_rows_workspace_bytes
    assert f(1, 1) == 0 and f(2048, 1024) == 0
    assert f(2049, 16) >= 2 * 16 * 4
    assert f(0, 16) == 0 and f(qg.QG_MAX_PLAN_ROWS + 1, 16) == 0 and f(5000, 0) == 0 and f(5000, 1025) == 0
    assert f(qg.QG_MAX_PLAN_ROWS, 1024) <= 64 * 1024 * 4
    f = qg.lib().qg_experts_combine_workspace_bytes
    assert f(10, 33) >= 10 * 33 * 4
    assert f(0, 33) == 0 and f(10, 0) == 0 and f(qg.QG_MAX_PLAN_ROWS, 1 << 29) == 0
    f = qg.lib().qg_lora_workspace_bytes
    m = (qg.CLora * 2)(qg.CLora(A, A, None, 64, 8, 0, A), qg.CLora(A, A, None, 64, 40, 0, A))
    assert f(m, 2, 100, 4, 256) >= 100 * (16 + 48) * 4
    assert f(m, 0, 100, 4, 256) == 0 and f(m, 9, 100, 4, 256) == 0 and f(m, 2, 0, 4, 256) == 0
    assert f(m, 2, 100, 0, 256) == 0 and f(m, 2, 100, 4, 100) == 0
    m[1].r = 12
    assert f(m, 2, 100, 4, 256) == 0


@needs_no_gpu
def test_validation_group_rows(qg):
    f = qg.lib().qg_group_rows
    assert f(None, 8, 4, A, A, A, None, 0, None) == NULLPTR
    assert f(A, 8, 4, A, A, None, None, 0, None) == NULLPTR
    assert f(A, 0, 4, A, A, A, None, 0, None) == SHAPE
    assert f(A, qg.QG_MAX_PLAN_ROWS + 1, 4, A, A, A, A, 1 << 30, None) == SHAPE
    assert f(A, 8, 0, A, A, A, None, 0, None) == SHAPE
    assert f(A, 8, 1025, A, A, A, None, 0, None) == SHAPE
    assert f(A, 8, 4, U, A, A, None, 0, None) == ALIGN
    need = qg.lib().qg_group_rows_workspace_bytes(5000, 4)
    assert need and f(A, 5000, 4, A, A, A, None, need, None) == WORKSPACE
    assert f(A, 5000, 4, A, A, A, A, need - 1, None) == WORKSPACE
    assert f(A, 5000, 4, A, A, A, U, need, None) == ALIGN


@needs_no_gpu
def test_validation_moe_route(qg):
    f = qg.lib().qg_moe_route
    assert f(None, 0, 4, 8, 2, 1, A, A, A, A, A, None, 0, None) == NULLPTR
    assert f(A, 0, 4, 8, 2, 1, A, None, A, A, A, None, 0, None) == NULLPTR
    assert f(A, 2, 4, 8, 2, 1, A, A, A, A, A, None, 0, None) == ARG
    assert f(A, 0, 4, 8, 9, 1, A, A, A, A, A, None, 0, None) == SHAPE
    assert f(A, 0, 4, 64, 17, 1, A, A, A, A, A, None, 0, None) == SHAPE
    assert f(A, 0, 4, 8, 0, 1, A, A, A, A, A, None, 0, None) == SHAPE
    assert f(A, 0, 0, 8, 2, 1, A, A, A, A, A, None, 0, None) == SHAPE
    assert f(A, 0, 4, 1025, 2, 1, A, A, A, A, A, None, 0, None) == SHAPE
    assert f(A, 0, qg.QG_MAX_PLAN_ROWS, 8, 2, 1, A, A, A, A, A, None, 0, None) == SHAPE
    assert f(A + 2, 0, 4, 8, 2, 1, A, A, A, A, A, None, 0, None) == ALIGN
    assert f(A, 0, 4096, 8, 2, 1, A, A, A, A, A, None, 0, None) == WORKSPACE


@needs_no_gpu
def test_validation_experts(qg):
    f = qg.lib().qg_qgemm_experts

    def call(w=None, g=None, amode=qg.QG_ACT_FLOAT, x=A, s_x=None, x_rows=16, y=A, yt=0):
        return f(w or experts(qg), g or groups(qg), amode, x, s_x, x_rows, y, yt, None)

    assert f(None, groups(qg), 1, A, None, 16, A, 0, None) == NULLPTR
    assert f(experts(qg), None, 1, A, None, 16, A, 0, None) == NULLPTR
    assert call(x=None) == NULLPTR and call(y=None) == NULLPTR
    assert call(experts(qg, codes=None)) == NULLPTR and call(experts(qg, scale=None)) == NULLPTR
    assert call(g=groups(qg, offsets=None)) == NULLPTR
    assert call(amode=qg.QG_ACT_INT8) == NULLPTR  # no s_x
    assert call(amode=3) == ARG and call(yt=2) == ARG and call(experts(qg, fmt=1)) == ARG
    assert call(g=groups(qg, rows=0)) == SHAPE and call(g=groups(qg, groups=5)) == SHAPE
    assert call(g=groups(qg, per_row=0)) == SHAPE and call(g=groups(qg, per_row=17)) == SHAPE
    assert call(g=groups(qg, rows=qg.QG_MAX_PLAN_ROWS + 1)) == SHAPE
    assert call(experts(qg, k=192)) == SHAPE and call(experts(qg, n=0)) == SHAPE
    assert call(experts(qg, e=1025), groups(qg, groups=1025)) == SHAPE
    assert call(experts(qg, k=qg.QG_BATCH_MAX_K + 128)) == SHAPE
    assert call(experts(qg, k=qg.QG_QGEMM_MAX_K + 128), amode=qg.QG_ACT_INT8, s_x=A) == SHAPE
    assert call(experts(qg, n=1 << 29, k=qg.QG_BATCH_MAX_K)) == SHAPE
    assert call(x_rows=0) == SHAPE and call(x_rows=1 << 31) == SHAPE
    assert call(g=groups(qg, order=None), x_rows=31) == SHAPE
    assert call(experts(qg, codes=U)) == ALIGN and call(x=U) == ALIGN and call(y=U) == ALIGN
    assert call(experts(qg, scale=U)) == ALIGN and call(g=groups(qg, order=U)) == ALIGN


@needs_no_gpu
def test_validation_experts_swiglu(qg):
    f = qg.lib().qg_qgemm_experts_swiglu

    def call(gate, up):
        return f(gate, up, groups(qg), 1, A, None, 16, A, 0, None)

    assert call(None, experts(qg)) == NULLPTR and call(experts(qg), None) == NULLPTR
    assert call(experts(qg, codes=None), experts(qg)) == NULLPTR
    assert call(experts(qg, fmt=qg.QG_WFMT_INT8_T16), experts(qg)) == ARG
    assert call(experts(qg, n=65), experts(qg)) == SHAPE and call(experts(qg, k=384), experts(qg)) == SHAPE
    assert call(experts(qg, codes=U), experts(qg)) == ALIGN


@needs_no_gpu
def test_validation_experts_combine(qg):
    f = qg.lib().qg_qgemm_experts_combine
    need = qg.lib().qg_experts_combine_workspace_bytes(32, 64)

    def call(pos=A, weights=A, tokens=16, ws=A, nws=need):
        return f(experts(qg), groups(qg, order=None), 1, A, None, 32, pos, weights, tokens, A, 0, ws, nws, None)

    assert call(pos=None) == NULLPTR and call(weights=None) == NULLPTR
    assert call(tokens=15) == SHAPE and call(tokens=0) == SHAPE
    assert call(pos=U) == ALIGN and call(ws=U) == ALIGN
    assert call(ws=None) == WORKSPACE and call(nws=need - 1) == WORKSPACE


@needs_no_gpu
def test_validation_lora(qg):
    f = qg.lib().qg_lora_add

    def call(r=16, n=64, a=A, b=A, y=A, scale=None, count=1, g=None, x=A, x_rows=32, k=256, yt=0, ws=A, nws=1 << 40):
        m = (qg.CLora * 1)(qg.CLora(a, b, scale, n, r, 0, y))
        return f(m, count, g or groups(qg, per_row=1), x, x_rows, k, yt, ws, nws, None)

    assert f(None, 1, groups(qg, per_row=1), A, 32, 256, 0, A, 1 << 40, None) == NULLPTR
    assert call(a=None) == NULLPTR and call(b=None) == NULLPTR and call(y=None) == NULLPTR and call(x=None) == NULLPTR
    assert call(g=groups(qg, per_row=1, order=None)) == NULLPTR
    assert call(count=0) == ARG and call(count=9) == ARG and call(yt=2) == ARG
    assert call(g=groups(qg, per_row=2)) == SHAPE
    assert call(r=12) == SHAPE and call(r=0) == SHAPE and call(r=264) == SHAPE
    assert call(n=0) == SHAPE and call(n=3) == SHAPE and call(k=100) == SHAPE and call(x_rows=31) == SHAPE and call(x_rows=1 << 31) == SHAPE
    assert call(a=U) == ALIGN and call(b=U) == ALIGN and call(y=U) == ALIGN and call(x=U) == ALIGN and call(ws=U) == ALIGN
    assert call(scale=U) == ALIGN
    assert call(ws=None) == WORKSPACE and call(nws=15) == WORKSPACE


def test_binding_refuses_host_tensors(qg):
    with pytest.raises(ValueError):
        qg.group_rows(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        qg.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError):
        qg.QExperts(qg.QG_WFMT_INT8, 1, 16, 128, torch.zeros(1, 16, 128, dtype=torch.int8), torch.zeros(1, 16))


@needs_no_gpu
@pytest.mark.parametrize("yt", [0, 1])
def test_lora_outputs_must_not_share_bytes(qg, yt):
    # 32 rows of 64 columns from A on; the other output starts inside, ends
    # inside, is the same, or touches neither end
    size = 32 * 64 * (2 if yt else 4)
    f = qg.lib().qg_lora_add

    def call(y0, y1, n0=64, n1=64):
        m = (qg.CLora * 2)(qg.CLora(A, A, None, n0, 16, 0, y0), qg.CLora(A, A, None, n1, 16, 0, y1))
        return f(m, 2, groups(qg, per_row=1), A, 32, 256, yt, None, 0, None)

    base = 1 << 40
    assert call(base, base) == ARG
    assert call(base, base + size - 16) == ARG and call(base + size - 16, base) == ARG
    assert call(base, base + 16, 64, 4) == ARG
    # apart: the next check, of the missing workspace, answers
    assert call(base, base + size) == WORKSPACE and call(base + size, base) == WORKSPACE
