"""The definitions in tests/mx_ref.py against values worked out by hand (no GPU)."""
import numpy as np
import pytest

import mx_ref as ref


def block(*v):
    x = np.zeros((1, 32))
    x[0, :len(v)] = v
    return x


@pytest.mark.parametrize("kind, x, byte, codes", [
    # 6 is the largest e2m1: scale 1 (byte 127) for it, 2 just above
    (ref.E2M1, (6.0, -6.0, 0.25, 0.75, 2.5, 5.0), 127, (7, 15, 0, 2, 4, 6)),       # ties to the even code: 0.25 -> 0, 0.75 -> 1, 2.5 -> 2, 5 -> 4
    (ref.E2M1, (6.0000005, 1.0), 128, (5, 1)),                                   # 3.0000002 -> 3, 0.5
    (ref.E2M1, (3.0,), 126, (7,)),
    # 448 is the largest e4m3
    (ref.E4M3, (448.0, -1.0), 127, (126, 128 + 56)),
    (ref.E4M3, (448.00003, 2.0), 128, (0x76, 56)),
    (ref.E4M3, (448.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9), 127, (126, 0, 2, 1)),   # below the smallest: ties to even
    (ref.E4M3, (0.0,), 0, (0,)),
    (ref.E4M3, (2.0 ** -130,), 0, (64 - 8 * 8,)),                                 # 2^-3 of 2^-127 .. see below
])
def test_blocks_by_hand(kind, x, byte, codes):
    c, b = ref.quantize(block(*x), kind)
    assert b[0, 0] == byte
    if x == (2.0 ** -130,):
        # 2^-130 / 2^-127 = 2^-3: exponent field 4, fraction 0
        codes = (4 * 8,)
    assert tuple(c[0, :len(codes)]) == codes
    assert not c[0, len(x):].any()


def test_values_round_trip():
    for kind, n in ((ref.E2M1, 16), (ref.E4M3, 256)):
        codes = np.resize(np.arange(n), (1, 256)).astype(np.uint8)
        v = ref.values(codes, np.full((1, 8), 130, np.uint8), kind)
        assert v[0, 1] == (0.5 if kind == ref.E2M1 else 2.0 ** -9) * 8
        back = ref.unpack(ref.pack(codes, kind), kind)
        assert np.array_equal(back, codes)
        fine = np.isfinite(v).reshape(8, 32).all(-1)
        assert np.array_equal(ref.held(v.reshape(8, 32), kind)[fine], v.reshape(8, 32)[fine])
    assert np.isnan(ref.held(block(1.0, np.inf), ref.E4M3)).all()


def test_routing_by_hand():
    z = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = ref.route(z, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w = ref.route(z, 3, renormalize=False, factor=2.0)
    assert ids.tolist() == [[2, 1, 0]] and np.allclose(w, [[1.0, 0.5, 0.25]])          # equal ones: the lower index
    # groups (0, 1) and (2, 3): best 1 prefers the second, the sum of two the second too, a bias the first
    assert ref.route(z, 1, groups=2, top_groups=1)[0].tolist() == [[2]]
    assert ref.route(z, 2, groups=2, top_groups=1, best=2)[0].tolist() == [[2, 3]]
    assert ref.route(z, 2, bias=[1.0, 0, 0, 0], groups=2, top_groups=1)[0].tolist() == [[0, 1]]
    off, rows, pos = ref.plan(np.array([[2, 0], [0, 1], [-1, -1]]), 4)
    assert off.tolist() == [0, 2, 3, 4, 4] and rows.tolist() == [0, 1, 1, 0] and pos.tolist() == [[3, 0], [1, 2], [-1, -1]]
