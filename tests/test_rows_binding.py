"""The binding of the row-dependent products on the CPU: what its objects check
and keep.  Host tensors stand in for device tensors; nothing is launched."""
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
