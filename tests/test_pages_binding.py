"""The objects of the paged cache's binding: what is assigned to a field is what the calls pass on (no GPU)."""
import pytest
import torch

import quantized_skinny_matmul_gb300 as gq


class OnGpu:
    """A tensor that says it lives on the GPU, contiguous, at an address of its own."""

    def __init__(self, t):
        self.shape, self.dtype, self.is_cuda, self.t = t.shape, t.dtype, True, t

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.t.element_size()

    def data_ptr(self):
        return self.t.data_ptr()


SHAPES = dict(k=((4, 16, 64), torch.int8), v=((4, 16, 64), torch.int8), ks=((4,), torch.float32), vs=((4,), torch.float32),
              table=((1, 2, 2), torch.int32), base=((1, 2, 2), torch.int32), held=((1,), torch.int32), seen=((1,), torch.int32))


def tensors():
    return {n: OnGpu(torch.zeros(s, dtype=d)) for n, (s, d) in SHAPES.items()}


def passed(x, name):
    """The field as a call reads it."""
    return getattr(x.by_ref.contents, name) or 0


@pytest.mark.parametrize("name", SHAPES)
def test_an_assigned_tensor_is_the_one_passed(name):
    c, other = gq.KVPages(gq.GQ_KV_I8, **tensors()), tensors()[name]
    assert passed(c, name) == getattr(c, name).data_ptr() != other.data_ptr()
    setattr(c, name, other)
    assert getattr(c, name) is other and passed(c, name) == other.data_ptr()
    assert [passed(c, n) for n in ("kind", "B", "Hkv", "D", "P", "NB", "pages")] == [0, 1, 2, 64, 16, 2, 4]
    shape, dtype = SHAPES[name]
    for bad in (torch.zeros((*shape, 1), dtype=dtype), torch.zeros(shape, dtype=torch.float64)):
        with pytest.raises(ValueError, match=name):
            setattr(c, name, OnGpu(bad))
    with pytest.raises(ValueError, match="CUDA"):
        setattr(c, name, torch.zeros(shape, dtype=dtype))
    assert getattr(c, name) is other and passed(c, name) == other.data_ptr()      # a refused one changes nothing


def test_what_an_eviction_returns_is_assigned_in_one_line():
    c, t = gq.KVPages(gq.GQ_KV_I8, **tensors()), tensors()
    c.table, c.base, w, c.held = t["table"], t["base"], None, t["held"]
    assert [passed(c, n) for n in ("table", "base", "held")] == [t[n].data_ptr() for n in ("table", "base", "held")]


@pytest.mark.parametrize("name", ["kind", "B", "Hkv", "D", "P", "NB", "pages", "struct", "by_ref"])
def test_sizes_are_fixed(name):
    c = gq.KVPages(gq.GQ_KV_I8, **tensors())
    with pytest.raises(AttributeError, match=name):
        setattr(c, name, getattr(c, name))


def test_scores_pass_on_what_is_assigned():
    f32, i32 = (lambda n: OnGpu(torch.zeros(n))), (lambda n: OnGpu(torch.zeros(n, dtype=torch.int32)))
    sc = gq.AttnScores(0.125, cap=30.0, window=7, slopes=f32(4), first=i32(3), prefix=i32(3))
    assert (passed(sc, "scale"), passed(sc, "cap"), passed(sc, "window")) == (0.125, 30.0, 7)
    for name, t in (("slopes", f32(4)), ("first", i32(5)), ("prefix", i32(5))):
        assert passed(sc, name) == getattr(sc, name).data_ptr()
        setattr(sc, name, t)
        assert passed(sc, name) == t.data_ptr()
        with pytest.raises(ValueError, match=name):
            setattr(sc, name, OnGpu(torch.zeros(4, dtype=torch.float64)))
        setattr(sc, name, None)
        assert passed(sc, name) == 0
    sc.scale, sc.cap, sc.window = 0.5, 0.0, 9
    assert (passed(sc, "scale"), passed(sc, "cap"), passed(sc, "window")) == (0.5, 0.0, 9)
    with pytest.raises(AttributeError):
        sc.struct = None
