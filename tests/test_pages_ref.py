"""The 64-bit definitions of the paged cache on worked examples, and the calls' refusals (no GPU)."""
import ctypes

import numpy as np
import pytest

import pages_ref as ref
import quantized_skinny_matmul_gb300 as gq

FAKE = 0x10000            # 16-byte aligned, never dereferenced: checks fail first
ODD = 0x10008


def test_e4m3_values_and_rounding():
    assert ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6 and ref.E4M3[126] == 448.0
    y = np.array([0.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, 432.0, 18.0])
    assert ref.decode(1, ref.encode(1, y)).tolist() == [0, 16, 20, -16, 0, 2.0 ** -8, 448, 448, 18]
    assert ref.decode(0, ref.encode(0, np.array([0.5, 1.5, -2.5, 127.0]))).tolist() == [0, 2, -2, 127]


def test_append_worked_example():
    # a page of 16 holding one token under scale 0.5; the next token's 127 doubles the scale
    codes, scale = np.zeros((1, 16, 2), np.int8), np.array([0.5], np.float32)
    codes[0, 0] = [4, 5]
    x = np.array([[[127.0, 1.5]]], np.float32)
    c, s = ref.append(0, 16, codes, scale, np.zeros((1, 1, 1), np.int32), [1], [0, 1], x)
    assert s[0] == 1.0 and c[0, 0].tolist() == [2, 2] and c[0, 1].tolist() == [127, 2]      # 2.5 -> 2, 1.5 -> 2


def test_visible_worked_example():
    x, see = ref.visible(np.array([0, 32]), 4, 7, 34, 1, 2, 2)      # positions 0..3, 32..34
    assert x.tolist() == [0, 1, 2, 3, 32, 33, 34] and see.tolist() == [False, True, False, False, False, True, True]


def test_evict_worked_example():
    t = np.arange(5, dtype=np.int32).reshape(1, 1, 5)
    w = np.array([[[0.1, 3.0, 3.0, 0.2, 0.0]]], np.float32)
    got = ref.evict(16, t, t * 16, w, np.array([4 * 16 + 1]), 3, 1, 1)
    assert got[0].tolist() == [[[0, 1, 4, 2, 3]]] and got[3].tolist() == [33]
    assert np.allclose(got[2], [[[0.1, 3.0, 0.0, 0.0, 0.0]]])


# ---- refusals: before anything is launched --------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    from quantized_skinny_matmul_gb300 import _build
    _build.build()
    return gq.lib()


def cache(**kw):
    v = dict(kind=0, B=2, Hkv=2, D=128, P=32, NB=4, pages=16, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, base=FAKE,
             held=FAKE, seen=FAKE)
    v.update(kw)
    return gq.KVPagesStruct(**v)


BAD_CACHE = [(dict(kind=2), 1), (dict(D=96), 1), (dict(P=8), 1), (dict(P=48), 1), (dict(B=0), 1), (dict(Hkv=-1), 1),
             (dict(NB=0), 1), (dict(pages=0), 1), (dict(NB=1 << 26), 1), (dict(pages=1 << 31), 1),
             (dict(B=1 << 20, Hkv=1 << 12), 1), (dict(k=0), 1), (dict(vs=0), 1), (dict(table=ODD), 2), (dict(held=0), 1),
             (dict(seen=ODD), 2), (dict(v=ODD), 2)]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_refused_caches(lib, kw, status):
    c, sc = cache(**kw), gq.AttnScoresStruct(0.1, 0.0, 0, 0, 0, 0)
    assert lib.gq_kv_pages_append(c, FAKE, 256, FAKE, 256, FAKE, 2, 1, None) == status
    assert lib.gq_kv_pages_read(c, FAKE, FAKE, 2, 1, FAKE, FAKE, None) == status
    assert lib.gq_attn_pages(c, sc, FAKE, 512, FAKE, 2, 1, 4, FAKE, 512, 0, 0, 1.0, None) == status
    assert lib.gq_kv_pages_evict(c, FAKE, 4, 1, 1, FAKE, FAKE, FAKE, FAKE, None) == status
    assert lib.gq_last_error_message()


def test_refused_steps(lib):
    c = cache()
    ap = lambda k=FAKE, ldk=256, v=FAKE, ldv=256, cu=FAKE, T=2, n=1: lib.gq_kv_pages_append(c, k, ldk, v, ldv, cu, T, n, None)  # noqa: E731
    assert lib.gq_kv_pages_append(None, FAKE, 256, FAKE, 256, FAKE, 2, 1, None) == 1
    assert ap(k=0) == 1 and ap(v=ODD) == 2 and ap(cu=0) == 1 and ap(cu=ODD) == 2
    assert ap(ldk=252) == 1 and ap(ldv=258) == 1 and ap(T=0) == 1 and ap(n=0) == 1 and ap(n=3) == 1
    assert ap(T=1000, n=129) == 1                                     # does not fit NB * P
    assert lib.gq_kv_pages_read(c, FAKE, FAKE, 2, 1, 0, 0, None) == 1
    assert lib.gq_kv_pages_read(c, 0, FAKE, 2, 1, FAKE, 0, None) == 1
    assert lib.gq_kv_pages_read(c, FAKE, FAKE, 2, 1, FAKE, ODD, None) == 2


def test_refused_attention(lib):
    c = cache()

    def at(sc=(0.1, 0.0, 0, 0, 0, 0), q=FAKE, ldq=512, cu=FAKE, T=2, n=1, Hq=4, out=FAKE, ldo=512, wi=0, wo=0, decay=1.0):
        s = gq.AttnScoresStruct(*sc) if sc else None
        return lib.gq_attn_pages(c, s, q, ldq, cu, T, n, Hq, out, ldo, wi, wo, decay, None)

    nan, inf = float("nan"), float("inf")
    assert at(sc=None) == 1 and at(sc=(nan, 0, 0, 0, 0, 0)) == 1 and at(sc=(inf, 0, 0, 0, 0, 0)) == 1
    assert at(sc=(0.1, -1.0, 0, 0, 0, 0)) == 1 and at(sc=(0.1, nan, 0, 0, 0, 0)) == 1 and at(sc=(0.1, 0, -1, 0, 0, 0)) == 1
    assert at(sc=(0.1, 0, 0, ODD, 0, 0)) == 2 and at(sc=(0.1, 0, 0, 0, ODD, 0)) == 2 and at(sc=(0.1, 0, 0, 0, 0, ODD)) == 2
    assert at(Hq=3) == 1 and at(Hq=0) == 1 and at(Hq=130, ldq=130 * 128, ldo=130 * 128) == 1
    assert at(ldq=508) == 1 and at(ldo=514) == 1 and at(q=0) == 1 and at(out=ODD) == 2
    assert at(wi=FAKE) == 1 and at(wi=ODD, wo=FAKE) == 2 and at(wo=ODD) == 2 and at(wo=FAKE, decay=nan) == 1


def test_refused_evictions(lib):
    ev = lambda c=cache(), w=FAKE, budget=4, first=1, last=1, t=FAKE, b=FAKE, wo=FAKE, h=FAKE: lib.gq_kv_pages_evict(  # noqa: E731
        c, w, budget, first, last, t, b, wo, h, None)
    assert ev(first=-1) == 1 and ev(last=0) == 1 and ev(budget=1) == 1 and ev(first=2, last=3) == 1
    assert ev(w=0) == 1 and ev(t=0) == 1 and ev(b=ODD) == 2 and ev(wo=ODD) == 2 and ev(h=0) == 1
    assert ev(c=cache(NB=16385, pages=1 << 20, P=16)) == 1


class OnGpu:
    """What the packed-row checks look at, of a tensor that says it lives on the GPU."""

    def __init__(self, t):
        self.shape, self.dtype, self.is_cuda, self.stride = t.shape, t.dtype, True, t.stride


def test_binding_refuses_wrong_rows():
    import torch
    for bad, why in ((torch.zeros((3, 8, 32))[:, :, ::2], "contiguous"), (torch.zeros((3, 40)), "multiple"),
                     (torch.zeros((3, 2, 8)), "shape"), (torch.zeros((3, 32), dtype=torch.float16), "float32")):
        with pytest.raises(ValueError, match=why):
            gq._packed(OnGpu(bad), 16, "q")
    with pytest.raises(ValueError, match="CUDA"):
        gq._packed(torch.zeros((3, 32)), 16, "q")
    assert gq._packed(OnGpu(torch.zeros((3, 64))[:, 8:40]), 16, "q") == (3, 2, 64)
    assert gq._packed(OnGpu(torch.zeros((1, 2, 16))), 16, "q") == (1, 2, 32)


def test_binding_refuses_wrong_tensors():
    import torch
    ok = dict(kind=0, k=torch.zeros((4, 16, 64), dtype=torch.int8), v=torch.zeros((4, 16, 64), dtype=torch.int8),
              ks=torch.zeros(4), vs=torch.zeros(4), table=torch.zeros((1, 2, 2), dtype=torch.int32),
              base=torch.zeros((1, 2, 2), dtype=torch.int32), held=torch.zeros(1, dtype=torch.int32),
              seen=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        gq.KVPages(**ok)
    for name, bad in (("v", torch.zeros((4, 16, 32), dtype=torch.int8)), ("k", torch.zeros((4, 16, 64))),
                      ("ks", torch.zeros(3)), ("vs", torch.zeros(4, dtype=torch.float64)),
                      ("base", torch.zeros((1, 2, 3), dtype=torch.int32)), ("held", torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError, match=name if name != "k" else "k|v"):
            gq.KVPages(**{**ok, name: bad})
    with pytest.raises(ValueError, match="slopes"):
        gq.AttnScores(1.0, slopes=torch.zeros(4, dtype=torch.float64))
    assert ctypes.sizeof(gq.KVPagesStruct) == 15 * 8 and ctypes.sizeof(gq.AttnScoresStruct) == 40
