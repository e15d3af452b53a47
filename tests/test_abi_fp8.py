"""Host-side checks of the 8-bit path's entry points (CPU only): argument
validation returns the documented status codes and launches nothing, and the
binding refuses tensors that do not fit."""
import ctypes

import pytest
import torch

A, U = 1 << 40, (1 << 40) + 1  # a 16-B aligned fake address, and a misaligned one
FAR = [A + (j << 44) for j in range(8)]  # addresses far enough apart for every size here
needs_no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                  reason="passes fake device addresses; runs where no GPU is visible")
HIP, NULLPTR, SHAPE, ALIGN, ARG, WORKSPACE = 6, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def qg():
    import os

    import quantized_gemv_amd as q
    if not os.path.exists(q.LIB_PATH):
        from quantized_gemv_amd.build import build
        build()
    return q


def norm(qg, **kw):
    a = dict(x=FAR[0], xt=1, residual=FAR[1], residual_out=FAR[1], weight=FAR[2], wt=0, eps=1e-5, rows=4, k=256, out=3,
             y=FAR[3], s=FAR[4])
    a.update(kw)
    return qg.lib().qg_rms_norm(*a.values(), None)


@needs_no_gpu
def test_validation_rms_norm(qg):
    for name in ("x", "weight", "y", "s"):
        assert norm(qg, **{name: None}) == NULLPTR
    assert norm(qg, residual=None) == NULLPTR and norm(qg, residual_out=None) == NULLPTR
    for out in (0, 1):  # no scales there
        assert norm(qg, out=out, s=None, y=U) == ALIGN
    for name in ("xt", "wt"):
        assert norm(qg, **{name: 2}) == ARG and norm(qg, **{name: -1}) == ARG
    assert norm(qg, out=4) == ARG and norm(qg, out=-1) == ARG
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert norm(qg, eps=eps) == ARG
    for k in (0, 128 + 8, 64, qg.QG_ROW_MAX_K + 128, -128):
        assert norm(qg, k=k) == SHAPE
    for k in (0, 4, 12, qg.QG_ROW_MAX_K + 8):
        assert norm(qg, out=2, k=k) == SHAPE and norm(qg, out=1, k=k) == SHAPE
    assert norm(qg, rows=0) == SHAPE and norm(qg, rows=1 << 31) == SHAPE
    assert norm(qg, rows=1 << 26, k=qg.QG_ROW_MAX_K) == SHAPE
    for name in ("x", "weight", "y", "residual", "residual_out"):
        assert norm(qg, **{name: FAR[6] + 8}) == ALIGN
    assert norm(qg, s=FAR[6] + 2) == ALIGN


@needs_no_gpu
def test_overlaps_rms_norm(qg):
    xb = 4 * 256 * 2
    for name in ("x", "residual", "weight"):
        at = {"x": FAR[0], "residual": FAR[1], "weight": FAR[2]}[name]
        assert norm(qg, y=at) == ARG and norm(qg, s=at) == ARG, name
    assert norm(qg, y=FAR[0] + xb - 16) == ARG and norm(qg, s=FAR[0] + xb - 4) == ARG
    assert norm(qg, y=FAR[0] - 4 * 256 + 16) == ARG
    assert norm(qg, s=FAR[3] + 4 * 256 - 4) == ARG
    assert norm(qg, residual_out=FAR[1] + 16) == ARG and norm(qg, residual_out=FAR[0] + 16) == ARG
    assert norm(qg, residual_out=FAR[2]) == ARG
    assert norm(qg, y=FAR[5], residual_out=FAR[5]) == ARG and norm(qg, s=FAR[5] + 64, residual_out=FAR[5]) == ARG
    # in place, and next to one another: past every check (no device here)
    for ok in (dict(), dict(residual_out=FAR[0]), dict(residual_out=FAR[5]), dict(y=FAR[0] + xb), dict(s=FAR[3] + 4 * 256),
               dict(residual=None, residual_out=None)):
        assert norm(qg, **ok) == HIP, ok


@needs_no_gpu
def test_validation_swiglu_and_quantizers(qg):
    def swiglu(**kw):
        a = dict(x=FAR[0], xt=1, rows=4, n=256, out=3, y=FAR[1], s=FAR[2])
        a.update(kw)
        return qg.lib().qg_swiglu(*a.values(), None)

    for name in ("x", "y", "s"):
        assert swiglu(**{name: None}) == NULLPTR
    assert swiglu(xt=2) == ARG and swiglu(out=5) == ARG
    for bad in (dict(n=0), dict(n=136), dict(out=2, n=qg.QG_ROW_MAX_K + 8), dict(out=0, n=12), dict(rows=0),
                dict(rows=1 << 31), dict(rows=1 << 30, n=1 << 10), dict(out=1, n=(1 << 30) + 8)):
        assert swiglu(**bad) == SHAPE, bad
    assert swiglu(x=FAR[0] + 8) == ALIGN and swiglu(y=FAR[0] + 8) == ALIGN and swiglu(s=FAR[2] + 1) == ALIGN
    assert swiglu(y=FAR[0] + 2 * 4 * 256 * 2 - 16) == ARG and swiglu(s=FAR[0]) == ARG and swiglu(s=FAR[1]) == ARG
    assert swiglu() == HIP and swiglu(out=0, s=None) == HIP and swiglu(out=0, n=qg.QG_ROW_MAX_K + 8, s=None) == HIP

    def quant(**kw):
        a = dict(x=FAR[0], xt=0, rows=4, cols=256, q=FAR[1], s=FAR[2])
        a.update(kw)
        return qg.lib().qg_quantize_fp8(*a.values(), None)

    for name in ("x", "q", "s"):
        assert quant(**{name: None}) == NULLPTR
    assert quant(xt=3) == ARG
    for bad in (dict(cols=0), dict(cols=64), dict(cols=200), dict(rows=0), dict(rows=1 << 31),
                dict(rows=1 << 14, cols=1 << 27), dict(cols=(1 << 30) + 128)):
        assert quant(**bad) == SHAPE, bad
    assert quant(x=U) == ALIGN and quant(q=U) == ALIGN and quant(s=U) == ALIGN
    assert quant(q=FAR[0]) == ARG and quant(s=FAR[0] + 16) == ARG and quant(s=FAR[1] + 16) == ARG
    assert quant() == HIP

    def weight(**kw):
        a = dict(w=FAR[0], wt=1, n=130, k=256, codes=FAR[1], scale=FAR[2])
        a.update(kw)
        return qg.lib().qg_quantize_fp8_weight(*a.values(), None)

    for name in ("w", "codes", "scale"):
        assert weight(**{name: None}) == NULLPTR
    assert weight(wt=2) == ARG
    for bad in (dict(k=0), dict(k=192), dict(n=0), dict(n=1 << 31), dict(n=1 << 30, k=2048), dict(k=(1 << 30) + 128)):
        assert weight(**bad) == SHAPE, bad
    assert weight(w=U) == ALIGN and weight(codes=U) == ALIGN and weight(scale=U) == ALIGN
    assert weight(codes=FAR[0]) == ARG and weight(scale=FAR[0]) == ARG and weight(scale=FAR[1] + 16) == ARG
    assert weight() == HIP


@needs_no_gpu
def test_validation_product(qg):
    def product(x=FAR[0], s_x=FAR[1], m=4, y=FAR[2], yt=1, ws=None, nws=0, **kw):
        a = dict(fmt=qg.QG_WFMT_FP8, n=130, k=256, codes=FAR[3], scale=FAR[4])
        a.update(kw)
        w = qg.CWeight(a["fmt"], 0, a["n"], a["k"], a["codes"], None, a["scale"], None, None)
        return qg.lib().qg_qgemm_fp8(ctypes.byref(w), x, s_x, m, y, yt, ws, nws, None)

    assert qg.lib().qg_qgemm_fp8(None, A, A, 4, A, 1, None, 0, None) == NULLPTR
    for name in ("x", "s_x", "y", "codes", "scale"):
        assert product(**{name: None}) == NULLPTR
    for fmt in (qg.QG_WFMT_INT8, qg.QG_WFMT_INT8_T16, 9, -1):
        assert product(fmt=fmt) == ARG
    assert product(yt=2) == ARG and product(yt=-1) == ARG
    for bad in (dict(k=0), dict(k=64), dict(k=192), dict(k=qg.QG_BATCH_MAX_K + 128), dict(m=0), dict(m=1 << 30), dict(n=0),
                dict(n=1 << 26), dict(m=1 << 29, k=4096), dict(n=1 << 25, k=65536), dict(m=1 << 20, n=1 << 19), dict(m=1 << 28, n=1),
                dict(m=(1 << 20) + 1, n=1 << 16)):
        assert product(**bad) == SHAPE, bad
    for name in ("x", "y", "codes"):
        assert product(**{name: U}) == ALIGN
    assert product(s_x=U) == ALIGN and product(scale=U) == ALIGN
    for name in ("x", "s_x", "codes", "scale"):
        assert product(**{name: FAR[2] + 16}) == ARG, name
    # the rows that pad the last tile are the matrix's, too
    assert product(y=FAR[3] + 130 * 256) == HIP and product(y=FAR[3] + 130 * 256, fmt=qg.QG_WFMT_FP8_T16) == ARG
    assert product() == HIP and product(fmt=qg.QG_WFMT_FP8_T16, yt=0) == HIP
    # few tiles and a long k: parts of k meet in the workspace
    f = qg.lib().qg_qgemm_fp8_workspace_bytes
    big = dict(m=300, n=4096, k=11008)
    need = f(300, 4096, 11008, 1)
    assert need >= 2 * 300 * 4096 * 4 and need % (300 * 4096 * 4) == 0
    assert product(**big) == WORKSPACE and product(ws=FAR[5], nws=need - 1, **big) == WORKSPACE
    assert product(ws=FAR[5] + 8, nws=need, **big) == ALIGN
    for name, at in (("x", 0), ("s_x", 1), ("y", 2), ("codes", 3), ("scale", 4)):
        assert product(ws=FAR[at], nws=need, **big) == ARG, name
    assert product(ws=FAR[5], nws=need, **big) == HIP
    assert f(1, 4096, 4096, 1) == 0 and f(4096, 11008, 4096, 1) == 0
    assert f(300, 4096, 11007, 1) == 0 and f(0, 4096, 11008, 1) == 0 and f(300, 4096, 11008, 2) == 0


@needs_no_gpu
def test_other_products_refuse_the_format(qg):
    w = qg.CWeight(qg.QG_WFMT_FP8, 0, 64, 256, A, None, A, None, None)
    assert qg.lib().qg_qgemv(ctypes.byref(w), 0, A, 1, A, 0, None, None) == ARG
    assert qg.lib().qg_qgemv_batch(ctypes.byref(w), 4, A, 1, A, 0, None) == ARG



def test_binding_refuses(qg, monkeypatch):
    e4, f32, bf = torch.float8_e4m3fn, torch.float32, torch.bfloat16
    x = torch.zeros(4, 256, dtype=bf)
    with pytest.raises(ValueError, match="GPU tensor"):
        qg.rms_norm(x, torch.zeros(256))
    from quantized_gemv_amd import _binding as b

    def on_cpu(t, name, dtype=None):
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
            raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
        return t
    monkeypatch.setattr(b, "_dev", on_cpu)
    sent = []
    monkeypatch.setattr(b, "_call", lambda name, x, *a: sent.append(name))
    w = torch.ones(256)
    for bad in (dict(x=x[0]), dict(weight=torch.ones(255)), dict(weight=w.double()), dict(x=x.double()),
                dict(residual=x.float()), dict(residual=x[:2]), dict(residual_out=x), dict(out_dtype=torch.float16),
                dict(y=x.half()), dict(y=x[:3]), dict(s=torch.zeros(4)), dict(out_dtype=e4, s=torch.zeros(4, 2)),
                dict(out_dtype=torch.int8, s=torch.zeros(2, 4)), dict(x=torch.zeros(256, 4, dtype=bf).t())):
        a = dict(x=x, weight=w)
        a.update(bad)
        with pytest.raises(ValueError):
            qg.rms_norm(**a)
    assert not sent
    y, s = qg.rms_norm(x, w, residual=x.clone(), out_dtype=e4)
    assert y.dtype == e4 and s.shape == (2, 4) and sent == ["qg_rms_norm"]
    y, s = qg.swiglu(torch.zeros(4, 512), out_dtype=torch.int8)
    assert y.shape == (4, 256) and s.shape == (4,)
    with pytest.raises(ValueError):
        qg.swiglu(torch.zeros(4, 255))
    with pytest.raises(ValueError):
        qg.quantize_fp8(x, s=torch.zeros(4, 2))
    with pytest.raises(ValueError):
        qg.quantize_fp8(x, q=torch.zeros(4, 256))

    q, sx = qg.quantize_fp8(x)
    W = qg.QWeight(qg.QG_WFMT_FP8, 130, 256, torch.zeros(130, 256).to(e4), torch.zeros(2, 2))
    assert qg.qgemm_fp8(W, q, sx).shape == (4, 130)
    T = qg.QWeight(qg.QG_WFMT_FP8_T16, 130, 256, torch.zeros(144 * 256).to(e4), torch.zeros(2, 2))
    assert qg.qgemm_fp8(T, q, sx, y_dtype=f32).dtype == f32
    for bad in (dict(w=qg.QWeight(qg.QG_WFMT_INT8, 130, 256, W.codes, W.scale)), dict(x=x), dict(x=q[:, :128].contiguous()),
                dict(s_x=sx.t().contiguous()), dict(y_dtype=torch.float16), dict(y=torch.zeros(4, 129)),
                dict(w=qg.QWeight(qg.QG_WFMT_FP8, 130, 256, W.codes[:129], W.scale)),
                dict(w=qg.QWeight(qg.QG_WFMT_FP8_T16, 130, 256, W.codes, W.scale)),
                dict(w=qg.QWeight(qg.QG_WFMT_FP8, 130, 256, W.codes, W.scale[:1])),
                dict(w=qg.QWeight(qg.QG_WFMT_FP8, 130, 256, W.codes, W.scale.double()))):
        a = dict(w=W, x=q, s_x=sx)
        a.update(bad)
        with pytest.raises(ValueError):
            qg.qgemm_fp8(**a)


def test_outputs_that_require_a_gradient_are_refused(qg, monkeypatch):
    from quantized_gemv_amd import _binding as b
    monkeypatch.setattr(b, "_dev", lambda t, *a: t)
    monkeypatch.setattr(b, "_call", lambda *a: None)
    x, r = torch.zeros(4, 256), torch.zeros(4, 256, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        qg.rms_norm(x, torch.ones(256), residual=r)
    with torch.no_grad():
        qg.rms_norm(x, torch.ones(256), residual=r)
    # what autograd has saved is seen to change
    h = torch.zeros(4, 256)
    a = torch.ones(4, 256, requires_grad=True)
    loss = (a * h).sum()
    qg.rms_norm(x, torch.ones(256), residual=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    s = torch.zeros(2, 4, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        qg.quantize_fp8(x, s=s)
    s = torch.zeros(2, 4)
    loss = (torch.ones(2, 4, requires_grad=True) * s).sum()
    qg.quantize_fp8(x, s=s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_steps_of_weights_in_the_other_order_are_refused(qg, monkeypatch):
    from quantized_gemv_amd import _binding as b
    monkeypatch.setattr(b, "_dev", lambda t, *a: t)
    monkeypatch.setattr(b, "_call", lambda *a: None)
    e4 = torch.float8_e4m3fn
    x, s_x = torch.zeros(1, 384).to(e4), torch.zeros(3, 1)
    for scale in (torch.zeros(2, 3), torch.zeros(6)):
        qg.qgemm_fp8(qg.QWeight(qg.QG_WFMT_FP8, 200, 384, torch.zeros(200, 384).to(e4), scale), x, s_x)
    with pytest.raises(ValueError, match="scale"):
        qg.qgemm_fp8(qg.QWeight(qg.QG_WFMT_FP8, 200, 384, torch.zeros(200, 384).to(e4), torch.zeros(3, 2)), x, s_x)


def test_launches_keep_their_memory(qg, monkeypatch):
    """Tensors whose data is set anew (a module that moves) are still where the
    arguments point."""
    from quantized_gemv_amd import _binding as b
    monkeypatch.setattr(b, "_dev", lambda t, *a: t)
    w = torch.ones(256)
    a = qg.RmsNormLaunch(torch.zeros(4, 256), w)
    at = w.data_ptr()
    w.data = torch.zeros(256)
    assert at in [s.data_ptr() for s in a._keep]


def test_tiles_are_made_on_the_codes_device(qg, monkeypatch):
    """As the other calls of the path: the matrix's device need not be the current one."""
    from quantized_gemv_amd import _binding as b
    monkeypatch.setattr(b, "_dev", lambda t, *a: t)
    sent = []
    monkeypatch.setattr(b, "_call", lambda name, x, *a: sent.append((name, x.data_ptr())))
    W = qg.QWeight(qg.QG_WFMT_FP8, 130, 256, torch.zeros(130, 256).to(torch.float8_e4m3fn), torch.zeros(2, 2))
    T = qg.tiled16(W)
    assert sent == [("qg_pack_tiles16", W.codes.data_ptr())]
    assert T.fmt == qg.QG_WFMT_FP8_T16 and T.codes.numel() == 144 * 256
