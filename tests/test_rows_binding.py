"""The binding of the row-dependent products on the CPU: what its objects check
and keep.  Host tensors stand in for device tensors; nothing is launched."""
import copy
import gc
import io
import weakref

import numpy as np
import pytest
import torch


@pytest.fixture
def qg(monkeypatch):
    """The package, taking host tensors where it wants device tensors."""
    import os

    import quantized_gemv_amd as q
    if not os.path.exists(q.LIB_PATH):
        from quantized_gemv_amd.build import build
        build()

    def dev(t, name, dtype=None):
        if not isinstance(t, torch.Tensor) or not t.is_contiguous():
            raise ValueError(name)
        if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
            raise ValueError(name)
        return t

    monkeypatch.setattr(q._binding, "_dev", dev)
    monkeypatch.setattr(q._binding, "_raw_stream", lambda index: 7)
    return q


def plan(qg, rows=8, groups=4):
    i32 = dict(dtype=torch.int32)
    return qg.RowGroups(torch.zeros(groups + 1, **i32), torch.zeros(rows, **i32), torch.zeros(rows, **i32))


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def adapters(qg, r=16, n=32, groups=4, k=256):
    return qg.LoraAdapters(bf16(groups, r, k), bf16(groups, n, r), torch.ones(groups))


# Fields set anew after the adapters were made: a rank that the other matrix
# does not have, too few groups or scales, another type, a layout with gaps.
@pytest.mark.parametrize("field,value", [
    ("a", bf16(4, 32, 256)),
    ("b", bf16(4, 32, 8)),
    ("b", bf16(3, 32, 16)),
    ("b", torch.zeros(4, 32, 16)),
    ("b", bf16(4, 32, 32)[:, :, ::2]),
    ("b", None),
    ("scale", torch.ones(3)),
    ("scale", torch.ones(4, dtype=torch.float64)),
    ("scale", torch.ones(8)[::2]),
], ids=["rank of a", "rank of b", "groups of b", "type of b", "layout of b", "no b", "short scale", "type of scale",
        "layout of scale"])
def test_launch_checks_adapters_as_they_are_now(qg, field, value):
    ad, x, ys = adapters(qg), bf16(8, 256), [torch.zeros(8, 32)]
    qg.LoraLaunch(x, plan(qg), [ad], ys)
    setattr(ad, field, value)
    with pytest.raises(ValueError):
        qg.LoraLaunch(x, plan(qg), [ad], ys)


class Recorded:
    """A workspace that notes the streams it is recorded on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_workspace_is_recorded_on_other_streams(qg, monkeypatch):
    """The workspace that a launch object takes by itself belongs to the stream
    it was made on: the allocator has to hear of every other one."""
    calls = []
    monkeypatch.setattr(qg._binding, "_call", lambda name, x, *args: calls.append(name))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "stream %d" % qg._binding._raw_stream(-1))
    x, ys = bf16(8, 256), [torch.zeros(8, 32)]
    own = qg.LoraLaunch(x, plan(qg), [adapters(qg)], ys)
    given = qg.LoraLaunch(x, plan(qg), [adapters(qg)], ys, ws=torch.zeros(1 << 16, dtype=torch.uint8))
    own.ws, given.ws = Recorded(), Recorded()
    for stream in (7, 9, 7, 8):
        monkeypatch.setattr(qg._binding, "_raw_stream", lambda index: stream)
        own.launch()
        given.launch()
    assert own.ws.streams == ["stream 9", "stream 8"] and given.ws.streams == []
    assert calls == ["qg_lora_add"] * 8


def test_adds_in_place_are_seen_by_autograd(qg, monkeypatch):
    """An output that a backward pass has saved: that pass fails, as after any
    addition in place.  One that needs a gradient is refused, unless gradients
    are off."""
    monkeypatch.setattr(qg._binding, "_call", lambda name, x, *args: None)
    x, ys = bf16(8, 256), [torch.zeros(8, 32), torch.zeros(8, 48)]
    ads = [adapters(qg), adapters(qg, n=48)]
    weight = torch.ones(48, requires_grad=True)
    for y in ys:
        loss = (y * weight[:y.shape[1]]).sum()
        qg.lora_add(x, plan(qg), ads, ys)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    launch = qg.LoraLaunch(x, plan(qg), ads, ys)
    ys[1].requires_grad_()
    with pytest.raises(ValueError):
        launch.launch()
    with torch.no_grad():
        before = ys[1]._version
        launch.launch()
    assert ys[1]._version == before + 1
    with torch.inference_mode():  # tensors without versions
        qg.lora_add(bf16(8, 256), plan(qg), ads[:1], [torch.zeros(8, 32)])


def test_nothing_is_marked_as_written_by_a_refused_call(qg, monkeypatch):
    def refuse(name, x, *args):
        raise qg.QgError(2, name)

    monkeypatch.setattr(qg._binding, "_call", refuse)
    y = torch.zeros(8, 32)
    with pytest.raises(qg.QgError):
        qg.lora_add(bf16(8, 256), plan(qg), [adapters(qg)], [y])
    assert y._version == 0


def test_experts_follow_their_tensors(qg):
    """Codes and scales whose data is set anew (a module moved to another
    device does that to its parameters): the products get the new memory,
    checked, never the old."""
    codes = torch.nn.Parameter(torch.zeros(2, 20, 128, dtype=torch.int8), requires_grad=False)
    scale = torch.nn.Parameter(torch.ones(2, 20), requires_grad=False)
    w = qg.QExperts(qg.QG_WFMT_INT8, 2, 20, 128, codes, scale)
    for t in (codes, scale):
        old = t.data
        t.data = old.clone()
        assert t.data_ptr() != old.data_ptr()
        c = w.c_struct()
        assert (c.codes, c.scale) == (codes.data_ptr(), scale.data_ptr())
        assert (c.fmt, c.e, c.n, c.k) == (qg.QG_WFMT_INT8, 2, 20, 128)
    for t, bad in ((codes, torch.zeros(2, 19, 128, dtype=torch.int8)), (codes, torch.zeros(2, 20, 128)),
                   (scale, torch.ones(39)), (scale, torch.ones(2, 20, dtype=torch.float64))):
        good = t.data
        t.data = bad
        with pytest.raises(ValueError):
            w.c_struct()
        t.data = good
    assert w.c_struct().codes == codes.data_ptr()


def watched(dtype, *shape):
    """A zero tensor over memory of numpy's, and a reference that dies with that
    memory."""
    host = np.zeros(shape + (torch.empty((), dtype=dtype).element_size(),), np.uint8)
    t = torch.empty(0, dtype=dtype)
    t.set_(torch.from_numpy(host).untyped_storage(), 0, shape)
    return t, weakref.ref(host)


def replaced(tensors):
    """Their data set anew, as a module that moves does to its parameters."""
    for t in tensors:
        t.data = torch.ones(3, dtype=t.dtype)
    gc.collect()


def test_a_plan_keeps_the_memory_it_points_to(qg):
    i32 = torch.int32
    tensors, alive = zip(*(watched(i32, n) for n in (5, 8, 8)))
    more, more_alive = zip(watched(i32, 4, 2), watched(torch.float32, 4, 2))
    r = qg.Routing(more[0], more[1], qg.RowGroups(*tensors, 2))
    at = r.ptrs
    replaced(tensors + more)
    assert all(a() is not None for a in alive + more_alive) and r.ptrs == at
    assert [a().ctypes.data for a in more_alive + alive] == list(at)
    assert r.groups.c_struct().order == at[3] and r.groups.c_struct().offsets == at[2]
    del r
    gc.collect()
    assert not any(a() is not None for a in alive + more_alive)


def test_a_launch_keeps_the_memory_it_points_to(qg):
    bf = torch.bfloat16
    shapes = [(bf, 8, 256), (bf, 4, 16, 256), (bf, 4, 32, 16), (torch.float32, 4), (torch.float32, 8, 32)]
    (x, a, b, scale, y), alive = zip(*(watched(*s) for s in shapes))
    groups = plan(qg)
    launch = qg.LoraLaunch(x, groups, [qg.LoraAdapters(a, b, scale)], [y])
    replaced((x, a, b, scale, y))
    assert all(r() is not None for r in alive)
    m = launch.m[0]
    assert [r().ctypes.data for r in alive] == [launch.args[3].value, m.a, m.b, m.scale, m.y]
    del launch
    gc.collect()
    assert not any(r() is not None for r in alive)


@pytest.mark.parametrize("again", [copy.deepcopy, copy.copy, "saved"])
def test_copies_point_to_their_own_memory(qg, again):
    """Experts, plans and routings that are copied, or saved and loaded."""
    def saved(v):
        f = io.BytesIO()
        torch.save(v, f)
        return torch.load(io.BytesIO(f.getvalue()), weights_only=False)  # what this test has written

    i32 = dict(dtype=torch.int32)
    w = qg.QExperts(qg.QG_WFMT_INT8, 2, 20, 128, torch.ones(2, 20, 128, dtype=torch.int8), torch.ones(2, 20))
    r = qg.Routing(torch.zeros(4, 2, **i32), torch.zeros(4, 2), qg.RowGroups(torch.zeros(5, **i32), torch.zeros(8, **i32),
                                                                           torch.zeros(8, **i32), 2))
    w2, r2 = (saved if again == "saved" else again)((w, r)) if again is not copy.copy else (copy.copy(w), copy.copy(r))
    c = w2.c_struct()
    assert (c.codes, c.scale) == (w2.codes.data_ptr(), w2.scale.data_ptr())
    assert (c.fmt, c.e, c.n, c.k) == (qg.QG_WFMT_INT8, 2, 20, 128)
    p = r2.groups
    assert r2.ptrs == tuple(t.data_ptr() for t in (r2.ids, r2.weights, p.offsets, p.order, p.pos))
    assert p.c_struct().order == p.order.data_ptr() and (p.rows, p.groups, p.per_row) == (8, 4, 2)
    if again is not copy.copy:
        assert c.codes != w.codes.data_ptr() and r2.ptrs[0] != r.ptrs[0]
