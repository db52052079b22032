"""The microscaled formats, the norm, routing and the experts' products where a call is unusual: offsets that end early, rows of
any magnitude, values that are not finite, and sizes that take several turns, slices or launches (GPU only).

Codes, scales, chosen experts and plans have to be equal to the definitions in 64 bits; bounds of sums as in test_gpu_mx.py.
"""

import numpy as np
import pytest
import torch

import mx_ref as ref
import quantized_skinny_matmul_gb300 as gq
from test_gpu_mx import built, dev, mx, near, rows, weights  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu
E = 4


# ---- plans whose offsets end early, or begin late --------------------------------------------------


def plan_of(off, token):
    return gq.ExpertPlan(dev(np.asarray(off, np.int32)), dev(token), dev(np.zeros((1, 1), np.int32)))


@pytest.mark.parametrize("mean", [4, 40])
@pytest.mark.parametrize("last", [-1, 0, 2.5, 9.0], ids=str)
def test_a_last_offset_out_of_range(mean, last):
    """The last expert has no rows and the fault is reported; the others' rows are those of the activations, not what an
    earlier call left in the workspace."""
    N, K, T = 130, 96, 20
    w, W = weights(1, E, N, K)
    x, X = mx(rows(2, T, K)[1])
    R = E * mean
    token = np.random.default_rng(0).integers(0, T, R).astype(np.int32)
    good = np.arange(E + 1) * mean
    off = good.copy()
    off[E] = int(last * mean) if last >= 0 else last
    other = mx(rows(3, T, K)[1])[0]
    gq.mul_mat_mxfp4(w, other, plan_of(good, token), gather=True)          # what the workspace holds is other rows
    out = torch.full((R, N), 5.0, device="cuda")
    gq.mul_mat_mxfp4(w, x, plan_of(off, token), gather=True, out=out)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    for e in range(E - 1):
        r = slice(good[e], good[e + 1])
        want, S = ref.product(X[token[r]], W[e])
        near(out[r], want, ref.product_tolerance(K) * S, f"expert {e}")
    assert (out[int(good[E - 1]):] == 5).all()
    up, _ = weights(2, 2 * E, 64, K)
    want = gq.swiglu_mxfp4(up, x, plan_of(good, token), gather=True)
    gq.swiglu_mxfp4(up, other, plan_of(good, token), gather=True)
    got = gq.swiglu_mxfp4(up, x, plan_of(off, token), gather=True)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    n = int(good[E - 1])
    assert torch.equal(got.codes[:n], want.codes[:n]) and torch.equal(got.scales[:n], want.scales[:n])


@pytest.mark.parametrize("mean", [4, 40])
def test_rows_in_front_of_the_first_expert(mean):
    """A plan may begin behind row 0: what stands in front belongs to no expert, is not read and is not written."""
    N, K, T, front = 130, 96, 20, 7
    w, W = weights(1, E, N, K)
    x, X = mx(rows(2, T, K)[1])
    R = front + E * mean + 5
    token = np.random.default_rng(0).integers(0, T, R).astype(np.int32)
    token[:front], token[R - 5:] = -1, T + 3                               # indices of nothing
    off = front + np.arange(E + 1) * mean
    out = torch.full((R, N), 5.0, device="cuda")
    gq.mul_mat_mxfp4(w, x, plan_of(off, token), gather=True, out=out)
    assert gq.gq_last_error() == gq.GQ_OK
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want, S = ref.product(X[token[r]], W[e])
        near(out[r], want, ref.product_tolerance(K) * S, f"expert {e}")
    assert (out[:front] == 5).all() and (out[R - 5:] == 5).all()
