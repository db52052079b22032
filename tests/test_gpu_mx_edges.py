"""The microscaled formats, the norm, routing and the experts' products where a call is unusual: offsets that end early, rows of
any magnitude, values that are not finite, and sizes that take several turns, slices or launches (GPU only).

Codes, scales, chosen experts and plans have to be equal to the definitions in 64 bits; bounds of sums as in test_gpu_mx.py.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mx_ref as ref
import quantized_skinny_matmul_gb300 as gq
from test_gpu_mx import DT, U, built, dev, host, mx, near, router, rows, weights  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu
FLT_MAX = float(np.finfo(np.float32).max)
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


# ---- the norm ------------------------------------------------------------------------------------


def check_norm(x, w, eps, dtype="f32"):
    """Codes (signs too), scales and y of rows on the GPU."""
    t = dev(x, DT[dtype])
    K = t.shape[1]
    _, q, y = gq.rms_norm_mx(t, w, eps, y_dtype=torch.float32)
    _, only, _ = gq.rms_norm_mx(t, w, eps, residual=torch.zeros_like(t), y_dtype=torch.bfloat16)
    alone = torch.empty_like(y)
    gq.gq_rms_norm_mx(t, K, None, K, gq.GQ_TYPE_BF16 if dtype == "bf16" else gq.GQ_TYPE_F32, w, eps, None, K, alone, gq.GQ_TYPE_F32, None,
                      None, len(t), K)
    with np.errstate(all="ignore"):
        want = ref.norm(host(t), None if w is None else host(w), eps)
        codes, b = ref.quantize(want, ref.E4M3)
    assert np.array_equal(host(q.scales)[:, :K // 32], b)
    zero = want == 0
    assert np.array_equal(np.where(zero, 0, host(q.codes)), np.where(zero, 0, codes))
    assert not (host(q.codes)[zero] & 127).any()
    nonzero = torch.from_numpy(host(t) != 0).cuda()                        # (a sum with +0 makes a -0 of x +0)
    assert torch.equal(only.codes[nonzero], q.codes[nonzero]) and torch.equal(only.scales, q.scales)
    inside = np.abs(want) <= FLT_MAX * (1 - 2.0 ** -19)
    for v in (y, alone):
        v = host(v)
        near(v[inside], want[inside], (2.0 ** -20 + U) * np.abs(want[inside]) + 2.0 ** -120)
        assert np.array_equal(np.isnan(v), np.isnan(want))
        large = np.abs(want) > FLT_MAX * (1 + 2.0 ** -19)
        assert np.array_equal(v[large], np.sign(want[large]) * np.inf)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-40, 1e-60, 1e300])
@pytest.mark.parametrize("K", [32, 160, 4096])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_any_magnitude(dtype, K, eps):
    """Rows whose squares leave the range of f32, at either end."""
    size = [1e-44, 1e-42, 1e-38, 1e-30, 1e-25, 1e-21, 1e-19, 1e-15, 1e-12, 1.0, 1e12, 1e15, 1e17, 1e18, 1e19, 1e30, 3e37]
    x = np.random.default_rng(K).standard_normal((3, len(size), K)) * np.array(size)[None, :, None]
    x = np.clip(x.reshape(-1, K), -3.3e38, 3.3e38).astype(np.float32)
    host_rows = host(dev(x, DT[dtype]))
    x = x[(host_rows != 0).any(-1)]                                        # (a row of zeros with eps 0 is the next test's)
    check_norm(x, None, eps, dtype)
    check_norm(x, dev(1 + 0.3 * np.random.default_rng(1).standard_normal(K).astype(np.float32)), eps, dtype)


@pytest.mark.parametrize("K", [32, 160, 4096])
def test_norm_of_uneven_rows_and_zeros(K):
    rng = np.random.default_rng(K)
    x = rng.standard_normal((8, K)).astype(np.float32)
    x[0, 3] = 3e38                                                         # one value far above the others
    x[1, :] *= 1e-38
    x[1, 5] = 1.0
    x[2, :16] = 3e38
    x[2, 16:] = 1e-44
    x[3] = 0
    x[4] = -0.0
    x[4, 9] = 1e-30
    x[5, ::2] = 0                                                          # zeros in between, and whole blocks of them
    x[6, :-32] = 0
    x[7] = np.where(rng.random(K) < 0.5, -2, 2)                            # exactly 1 and -1 with eps 0
    for eps in (1e-6, 1e-60):
        check_norm(x, None, eps)
    check_norm(np.delete(x, 3, 0), None, 0.0)
    q = gq.rms_norm_mx(dev(x), None, 0.0)[1]                               # 0 / 0
    assert (q.scales[3, :K // 32] == 255).all() and not q.codes[3].any() and (q.scales[[0, 1, 2, 4, 5, 6, 7], :K // 32] != 255).all()


def test_norm_with_weights_of_any_magnitude():
    K = 32768
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, K)).astype(np.float32)
    w = rng.standard_normal(K).astype(np.float32)
    w[:32], w[32:64], w[64:96], w[96:128], w[128] = w[:32] * 1e30, w[32:64] * 1e-30, 0, 1e-44, FLT_MAX
    x[1] *= 1e15
    x[2] *= 1e-15
    x[3] *= 1e-36
    x[4] *= 1e30
    x[5] = 0
    x[5, 128], x[5, 7] = 1e25, -1e20                                       # y is 181 times the largest f32
    for eps in (0.0, 1e-6):
        check_norm(x, dev(w), eps)
    check_norm(x[:, :4096], dev(w[:4096]), 0.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_with_a_weight_that_is_not_finite(bad):
    """Its block, and that alone, holds no numbers, whatever the other columns of the row are."""
    K = 1024
    x = np.random.default_rng(4).standard_normal((300, K)).astype(np.float32)
    w = np.ones(K, np.float32)
    w[700] = bad
    q = gq.rms_norm_mx(dev(x), dev(w), 1e-6)[1]
    with np.errstate(all="ignore"):
        codes, b = ref.quantize(ref.norm(x, w, 1e-6), ref.E4M3)
    assert (b == 255).sum() == 300
    assert np.array_equal(host(q.scales)[:, :K // 32], b) and np.array_equal(host(q.codes), codes)


def test_the_sign_of_zeros_does_not_depend_on_the_row():
    """-0 has the code of -0, in rows that f32 decides and in rows that need more."""
    x = np.random.default_rng(5).standard_normal((300, 1024)).astype(np.float32)
    x[:, 3::7] = -0.0
    x[:, 5::7] = 0.0
    q = gq.rms_norm_mx(dev(x), None, 1e-6)[1]
    assert np.array_equal(host(q.codes), ref.quantize(ref.norm(x, None, 1e-6), ref.E4M3)[0])


@pytest.mark.parametrize("M, K", [(6000, 64), (3100, 1024), (700, 4096), (330, 16416)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_where_each_cta_takes_several_rows(M, K, dtype):
    """More rows than CTAs are resident, of ordinary and of extreme size in turn."""
    x = np.random.default_rng(M).standard_normal((M, K)).astype(np.float32)
    size = np.ones(M)
    size[3::11], size[5::13], size[-2:], size[7::17] = 1e20, 1e-22, 1e25, 0
    x = (x * size[:, None]).astype(np.float32)
    t, r = dev(x, DT[dtype]), dev(np.roll(x, 1, 1), DT[dtype])
    want_h = (t.float() + r.float()).to(DT[dtype])
    h, q = gq.rms_norm_mx(t, None, 1e-12, residual=r)
    assert torch.equal(h, want_h)
    want = ref.norm(host(want_h), None, 1e-12)
    codes, b = ref.quantize(want, ref.E4M3)
    assert np.array_equal(host(q.scales)[:, :K // 32], b)
    assert np.array_equal(np.where(want == 0, 0, host(q.codes)), np.where(want == 0, 0, codes))
    # in place: a CTA reads its next rows while it writes this one's sum
    out = gq.MXRows.empty(M, K)
    code = gq.GQ_TYPE_BF16 if dtype == "bf16" else gq.GQ_TYPE_F32
    gq.gq_rms_norm_mx(t, K, r, K, code, None, 1e-12, t, K, None, gq.GQ_TYPE_F32, out.codes, out.scales, M, K)
    assert torch.equal(t, want_h) and torch.equal(out.codes, q.codes) and torch.equal(out.scales, q.scales)


def test_norm_of_rows_that_share_a_mark():
    """A CTA marks the rows that it leaves for its end in 2048 bits: past 2048 turns, some share one."""
    K, turns = 32, 2048
    ctas = torch.cuda.get_device_properties(0).multi_processor_count * 32
    M = ctas * turns + 3 * ctas + 5
    x = torch.randn((M, K), generator=torch.Generator("cuda").manual_seed(0), device="cuda").bfloat16()
    wide = [0, 7, ctas + 3, ctas * turns + 1, ctas * (turns + 2) + 9, M - 1]
    x[wide] *= 1e25
    q = gq.rms_norm_mx(x, None, 1e-6)[1]
    at = torch.tensor(sorted(set(wide) | {(r + d) % M for r in wide for d in (1, ctas, ctas * turns, M - ctas * turns)}), device="cuda")
    want = ref.norm(host(x[at]), None, 1e-6)
    codes, b = ref.quantize(want, ref.E4M3)
    zero = want == 0
    assert np.array_equal(host(q.scales[at])[:, :1], b) and np.array_equal(np.where(zero, 0, host(q.codes[at])), np.where(zero, 0, codes))
    part = gq.rms_norm_mx(x[-2 * ctas:], None, 1e-6)[1]
    assert torch.equal(q.codes[-2 * ctas:], part.codes) and torch.equal(q.scales[-2 * ctas:], part.scales)


# ---- routing --------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [20, 100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n, k", [(64, 6), (40, 32)])
@pytest.mark.parametrize("best", [0, 1, 2])
def test_route_of_values_that_are_not_finite(T, score, n, k, best, dtype):
    """+infinity counts as the largest finite number, NaN as -infinity, among logits and biases: each token has top_k experts."""
    rng = np.random.default_rng(T)
    z = rng.integers(-3, 3, (T, n)).astype(np.float32)
    z[1, 5], z[2, [3, 30]], z[3], z[4, :] = np.inf, np.inf, np.inf, -np.inf
    z[4, 9], z[5, ::2], z[6, 7], z[6, 8], z[7], z[8] = np.inf, -np.inf, np.nan, np.inf, np.nan, -np.inf
    z[9, :12], z[10, 11], z[10, 12] = np.inf, 3e38, np.inf
    finite = (0.1 * rng.standard_normal(n)).astype(np.float32)
    masked, odd, large = finite.copy(), finite.copy(), finite.copy()
    masked[[0, 5, 17, 30]] = -np.inf
    odd[[3, 20]], odd[[9, 33]], odd[12] = np.inf, np.nan, -np.inf
    large[[2, 8, 21]] = 3e38
    opt = dict(groups=4, top_groups=4 if k > 20 else 2, best=best) if best else {}
    t = dev(z, DT[dtype])
    clean = np.where(np.isnan(host(t)), -np.inf, np.minimum(host(t), FLT_MAX))
    for bias in (None, finite, masked, odd, large):
        exact = None if bias is None else np.where(np.isnan(bias), -np.inf, np.minimum(bias.astype(np.float64), FLT_MAX))
        ids, w, plan = gq.route(t, router(dict(E=n, k=k, score=score, bias=None if bias is None else dev(bias), **opt)))
        with np.errstate(all="ignore"):
            want, ww = ref.route(clean, k, score, exact, **opt)
        assert np.array_equal(host(ids), want)
        # arguments of the exponential are small whole numbers, or leave 0
        near(w, ww, (6 + n / 32 + 16) * U * np.abs(ww) + 1e-38)
        off, rows_, pos = ref.plan(want, n)
        assert np.array_equal(host(plan.offsets), off) and np.array_equal(host(plan.pos), pos) and np.array_equal(host(plan.rows), rows_)


# ---- the example ------------------------------------------------------------------------------------


def test_the_example_sees_outputs_that_are_no_numbers():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "experts.py")
    spec = importlib.util.spec_from_file_location("experts_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(256, 96, 8, 2)
    x = torch.randn((5, 256), generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    out, parts = layer.forward(x, torch.zeros_like(x))
    worst, unit = example.check(layer, out, parts, 5)
    assert worst < 1e-4 and unit < 5e-4
    broken = out.clone()
    broken[2, 17] = float("nan")
    assert not example.check(layer, broken, parts, 5)[0] < 1e-4
    assert not example.check(layer, torch.full_like(out, float("nan")), parts, 5)[0] < 1e-4
    parts[-1].scales[3, 1] = 255
    worst, unit = example.check(layer, out, parts, 5)
    assert not worst < 1e-4 and not unit < 5e-4


# ---- sizes that take several slices or launches -------------------------------------------------------


def test_gathered_rows_in_slices():
    """More rows than the workspace's share of 512 MB holds: a second slice begins in the middle of an expert."""
    K, N, T = 32, 8, 1000
    n = (512 << 20) // (K + 16)
    R = n + 100000
    off = np.array([0, 5000000, n + 40000, n + 40000, R - 9])
    w, W = weights(1, 4, N, K)
    x, X = mx(rows(2, T, K)[1])
    gen = torch.Generator("cuda").manual_seed(0)
    token = torch.randint(0, T, (R,), generator=gen, device="cuda", dtype=torch.int32)
    plan = gq.ExpertPlan(dev(off.astype(np.int32)), token, dev(np.zeros((1, 1), np.int32)))
    out = torch.full((R, N), 5.0, device="cuda")
    gq.mul_mat_mxfp4(w, x, plan, gather=True, out=out)
    assert gq.gq_last_error() == gq.GQ_OK
    for e in range(4):
        want, S = ref.product(X, W[e])
        r = slice(int(off[e]), int(off[e + 1]))
        i = token[r].long()
        assert ((out[r].double() - dev(want)[i]).abs() <= dev(ref.product_tolerance(K) * S)[i]).all(), e
    assert (out[R - 9:] == 5).all()


def test_rows_that_take_several_launches():
    """A launch of rows numbers 2^30 groups of eight values: quantization, reading back and the sum over experts go on behind them."""
    K = 4096
    n = ((1 << 30) - 1) // (K // 8)
    M = n + 5
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(0))
    q = gq.quantize_mx(x)
    parts = [slice(0, 6), slice(n - 3, M)]
    for r in parts:
        p = gq.quantize_mx(x[r])
        assert torch.equal(q.codes[r], p.codes) and torch.equal(q.scales[r], p.scales)
    back = gq.dequantize_mx(q, torch.bfloat16)
    for r in parts:
        assert torch.equal(back[r], gq.dequantize_mx(gq.quantize_mx(x[r]), torch.bfloat16))
    del back, q
    e = gq.quantize_mx(x, gq.GQ_MX_E2M1)
    for r in parts:
        assert torch.equal(e.codes[r], gq.quantize_mx(x[r], gq.GQ_MX_E2M1).codes)
    del e
    y = torch.randn((7, K), device="cuda")
    pos = torch.randint(0, 7, (M, 2), device="cuda", dtype=torch.int32)
    w = torch.rand((M, 2), device="cuda")
    ints = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")  # noqa: E731
    out = gq.experts_combine(y, gq.ExpertPlan(ints(2), ints(7), pos), w, residual=x, dtype=torch.bfloat16)
    for r in parts:
        p = gq.ExpertPlan(ints(2), ints(7), pos[r].contiguous())
        assert torch.equal(out[r], gq.experts_combine(y, p, w[r].contiguous(), residual=x[r], dtype=torch.bfloat16))
    del x, out
    torch.cuda.empty_cache()
