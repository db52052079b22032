"""The microscaled formats, the norm, routing and the experts' products against their definitions in 64 bits (GPU only).

Codes, scales, chosen experts and plans have to be equal: they are decided exactly.  Sums: mx_ref.product_tolerance and
mx_ref.swiglu say how far f32 sums on the tensor cores may be off.  Routing weights: the f32 exponential is within 2 units,
its argument x - m is rounded once (|x - m| / 2 units of its result), sums and quotients round E / 32 + 16 times.
"""
import numpy as np
import pytest
import torch

import mx_ref as ref
import quantized_skinny_matmul_gb300 as gq

pytestmark = pytest.mark.gpu
U, BF = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    gq.gq_last_error()
    yield
    assert gq.gq_last_error() == gq.GQ_OK


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def rows(seed, M, K, dtype="f32"):
    """Activations with loud channels, as the GPU holds them, and as 64 bits."""
    x = np.random.default_rng(seed).standard_normal((M, K)).astype(np.float32)
    x[:, ::37] *= 8
    t = dev(x, DT[dtype])
    return t, host(t)


def weights(seed, n, N, K):
    """n matrices [N, K] quantized to 4 bits: repacked, and their values [n, N, K]."""
    w = np.random.default_rng(seed).standard_normal((n * N, K)) / np.sqrt(K)
    codes, b = ref.quantize(w, ref.E2M1)
    padded = np.zeros((n * N, ref.cols(K)), np.uint8)
    padded[:, :K // 32] = b
    return gq.repack_mxfp4(dev(ref.pack(codes, ref.E2M1)), dev(padded), N, K), ref.values(codes, b, ref.E2M1).reshape(n, N, K)


def mx(values):
    """Rows in e4m3 blocks from values on the host."""
    codes, b = ref.quantize(values, ref.E4M3)
    padded = np.full((len(values), ref.cols(values.shape[1])), 255, np.uint8)      # what the padding holds does not matter
    padded[:, :b.shape[1]] = b
    return gq.MXRows(dev(codes), dev(padded)), ref.values(codes, b, ref.E4M3)


def near(got, want, tol, what=""):
    got, want, tol = np.broadcast_arrays(host(got) if torch.is_tensor(got) else got, want, tol)
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, f"{what}: {len(bad)} of {got.size} off; first {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}, tol {tol[tuple(bad[0])]}"


# ---- blocks ----------------------------------------------------------------------------------


def edge_rows(K):
    """Zeros, ties at every border, values next to the scales' borders, tiny, subnormal and huge ones."""
    out = []
    for el in ref.ELEMENTS.values():
        border = (el[1:] + el[:-1]) / 2
        for v in np.array_split(np.concatenate([border, -border, el]), -(-(3 * len(el)) // 31)):
            out.append(np.concatenate([[el[-1]], v]))
        top = np.float32(el[-1])
        out += [[np.nextafter(top, np.float32(9999))], [np.nextafter(top, np.float32(0))], [top * 2.0 ** -40], [2.0 ** -126, 2.0 ** -130], [2.0 ** -149],
                [3e38, 1e30], [0.0, -0.0]]
    x = np.zeros((len(out), K), np.float32)
    for i, v in enumerate(out):
        x[i, (i % (K // 32)) * 32:][:len(v)] = v
    return x


@pytest.mark.parametrize("kind", [ref.E2M1, ref.E4M3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M, K", [(1, 32), (3, 96), (70, 544), (257, 1024)])
def test_quantize_and_read_back(kind, dtype, M, K):
    x = np.concatenate([edge_rows(K), rows(M + K, M, K)[1].astype(np.float32)])
    t = dev(x, DT[dtype])
    q = gq.quantize_mx(t, kind)
    codes, b = ref.quantize(host(t), kind)
    assert np.array_equal(host(q.codes), ref.pack(codes, kind))
    assert np.array_equal(host(q.scales)[:, :K // 32], b) and not host(q.scales)[:, K // 32:].any()
    v = ref.values(codes, b, kind)
    with np.errstate(over="ignore"):
        held = v.astype(np.float32)                                                # (3e38 is held as 2^128: infinity in f32 and bf16)
    assert np.array_equal(host(gq.dequantize_mx(q)), held)
    half, fine = host(gq.dequantize_mx(q, torch.bfloat16)), np.isfinite(held)
    assert np.array_equal(half[~fine], held[~fine])
    near(half[fine], v[fine], 2.0 ** -134)                                         # exact but below bf16's subnormals


def test_rows_of_a_wider_matrix_and_bad_values():
    x, _ = rows(1, 9, 256)
    x[2, 40], x[5, 64], x[5, 70] = float("nan"), float("inf"), -float("inf")
    q = gq.quantize_mx(x[:, 32:160])                                       # strided rows
    codes, b = ref.quantize(host(x)[:, 32:160], ref.E4M3)
    assert np.array_equal(host(q.codes), codes) and np.array_equal(host(q.scales)[:, :4], b)
    assert (b == 255).sum() == 2
    assert np.array_equal(np.isnan(host(gq.dequantize_mx(q))), np.repeat(b == 255, 32, -1))


# ---- the norm ----------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype, y", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("M, K", [(1, 32), (5, 96), (1, 4096), (700, 544), (3, 16416), (2, 32768)])
def test_norm(dtype, y, M, K):
    x, _ = rows(M, M, K, dtype)
    res, _ = rows(M + 1, M, K, dtype)
    w = dev(1 + 0.3 * np.random.default_rng(K).standard_normal(K).astype(np.float32))
    before = x.clone(), res.clone()
    h, q, out = gq.rms_norm_mx(x, w, 1e-5, residual=res, y_dtype=DT[y])
    assert torch.equal(x, before[0]) and torch.equal(res, before[1])
    assert torch.equal(h, (x.float() + res.float()).to(DT[dtype]))
    want = ref.norm(host(h), host(w), 1e-5)
    codes, b = ref.quantize(want, ref.E4M3)
    assert np.array_equal(host(q.codes) & 127, codes & 127) and np.array_equal(host(q.scales)[:, :K // 32], b)
    assert not host(q.scales)[:, K // 32:].any()
    near(out, want, (2.0 ** -20 + (BF if y == "bf16" else U)) * np.abs(want))


def test_norm_edges():
    K = 160
    x = np.random.default_rng(0).standard_normal((6, K)).astype(np.float32)
    x[1], x[2, 5], x[3, 40] = 0, np.nan, np.inf
    x[4] *= 1e-30                                  # the mean underflows: eps alone
    x[5] *= 1e15
    t = dev(x)
    h, q = gq.rms_norm_mx(t, None, 1e-6)
    assert h is t
    want = ref.norm(x, None, 1e-6)
    codes, b = ref.quantize(want, ref.E4M3)
    # a row with a NaN is NaN; one with an infinity is infinity times 0, or 0, by the definition
    fine = [0, 1, 4, 5]
    assert np.array_equal(host(q.codes)[fine] & 127, codes[fine] & 127) and np.array_equal(host(q.scales)[fine, :5], b[fine])
    v = host(gq.dequantize_mx(q))
    assert np.isnan(v[2]).all() and np.isnan(v[3, 32:64]).all()
    # in place, strided, and the outputs one by one
    wide = torch.randn((9, 2 * K), device="cuda").bfloat16()
    a, r = wide[:, :K], wide[:, K:]
    total, keep = (a.float() + r.float()).bfloat16(), a.clone()
    out = torch.empty((9, K), device="cuda")
    gq.gq_rms_norm_mx(a, 2 * K, r, 2 * K, gq.GQ_TYPE_BF16, None, 1e-6, r, 2 * K, out, gq.GQ_TYPE_F32, None, None, 9, K)
    assert torch.equal(r, total) and torch.equal(a, keep)
    want = ref.norm(host(total), None, 1e-6)
    near(out, want, 2.0 ** -19 * np.abs(want))


# ---- products ----------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M, N, K", [(1, 1, 32), (1, 128, 128), (3, 129, 96), (16, 257, 2080), (17, 100, 512), (64, 384, 1024), (65, 130, 160),
                                     (176, 128, 640), (177, 255, 2048), (400, 64, 4096), (1, 700, 11008)])
def test_product(dtype, M, N, K):
    w, W = weights(N, 1, N, K)
    x, xv = rows(M + K, M, K, dtype)
    X = ref.held(xv, ref.E4M3)
    want, E = ref.product(X, W[0])
    tol = ref.product_tolerance(K) * E
    f32 = gq.mul_mat_mxfp4(w, x)
    near(f32, want, tol)
    near(gq.mul_mat_mxfp4(w, mx(X)[0], dtype=torch.bfloat16), want, tol + BF * np.abs(want))
    wide = torch.full((M, N + 5), 7.0, device="cuda")
    assert torch.equal(gq.mul_mat_mxfp4(w, x, out=wide[:, 4:N + 4]), f32)            # any stride
    assert (wide[:, :4] == 7).all() and (wide[:, N + 4:] == 7).all()


def test_product_of_one_sign_and_wide_scales():
    """Sums that only grow, and blocks whose scales differ by 2^30, where cut-off bits would show."""
    K, N, M = 8192, 130, 20
    rng = np.random.default_rng(3)
    W = np.abs(rng.standard_normal((N, K))) * 2.0 ** rng.integers(-15, 15, (N, K // 32)).repeat(32, -1)
    codes, b = ref.quantize(W, ref.E2M1)
    padded = np.zeros((N, ref.cols(K)), np.uint8)
    padded[:, :K // 32] = b
    w = gq.repack_mxfp4(dev(ref.pack(codes, ref.E2M1)), dev(padded), N, K)
    x, X = mx(np.abs(rng.standard_normal((M, K))))
    want, E = ref.product(X, ref.values(codes, b, ref.E2M1))
    near(gq.mul_mat_mxfp4(w, x), want, ref.product_tolerance(K) * E)
    # every scale byte from 0 to 254 on one side, the inverse on the other
    b = np.arange(255, dtype=np.uint8)[:128, None].repeat(4, 1)
    codes = np.full((128, 128), 4, np.uint8)                                  # 2
    padded = np.zeros((128, 16), np.uint8)
    for low in (0, 127):
        padded[:, :4] = b + low
        w = gq.repack_mxfp4(dev(ref.pack(codes, ref.E2M1)), dev(padded), 128, 128)
        q = np.full((1, 16), 255, np.uint8)
        q[0, :4] = 190 - low
        got = host(gq.mul_mat_mxfp4(w, gq.MXRows(dev(np.full((1, 128), 0x38, np.uint8)), dev(q))))    # 1.0
        assert np.array_equal(got[0], 256 * 2.0 ** (b[:, 0] + low + 190.0 - low - 254))


def test_not_a_number_stays_in_its_row():
    w, W = weights(5, 1, 200, 256)
    x, xv = rows(6, 40, 256)
    X = ref.held(xv, ref.E4M3)
    good = gq.mul_mat_mxfp4(w, x)
    x[7, 100], x[33, 0] = float("nan"), float("inf")
    got = gq.mul_mat_mxfp4(w, x)
    bad = torch.isnan(got).any(1)
    assert bad.nonzero().flatten().tolist() == [7, 33] and torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], good[~bad])
    # a weight block's NaN: its row of W, a column of the output
    codes, b = ref.quantize(W[0], ref.E2M1)
    padded = np.zeros((200, 16), np.uint8)
    padded[:, :8] = b
    padded[150, 3] = 255
    w = gq.repack_mxfp4(dev(ref.pack(codes, ref.E2M1)), dev(padded), 200, 256)
    got = gq.mul_mat_mxfp4(w, mx(X)[0])
    assert torch.isnan(got[:, 150]).all() and torch.isnan(got).sum() == 40


# ---- experts -----------------------------------------------------------------------------------


def expert_case(seed, counts, T, behind=0):
    """A plan with so many rows for each expert, tokens at random, and room behind the last row."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1])
    token = np.random.default_rng(seed).integers(0, T, R + behind).astype(np.int32)
    return gq.ExpertPlan(dev(off), dev(token), dev(np.zeros((1, 1), np.int32))), off, token, R


COUNTS = [[1], [0, 0, 3], [5, 0, 16, 1, 0, 17, 2], [70, 0, 30, 64], [300, 1, 0, 177, 90], [0] * 500 + [2] + [0] * 522 + [1]]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("N, K", [(1, 32), (129, 160), (256, 1056)])
def test_experts(counts, gather, N, K):
    E, T = len(counts), 50
    if E > 100:
        N, K = 1 + N % 3, 32
    plan, off, token, R = expert_case(sum(counts), counts, T, behind=9)
    w, W = weights(E, E, N, K)
    x, X = mx(rows(N + K, T if gather else R + 9, K)[1])
    out = torch.full((R + 9, N), -3.0, device="cuda")
    assert gq.mul_mat_mxfp4(w, x, plan, gather=gather, out=out) is out
    assert (out[R:] == -3).all()                                              # rows behind the last expert's are left alone
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want, S = ref.product(X[token[r]] if gather else X[r], W[e])
        near(out[r], want, ref.product_tolerance(K) * S, f"expert {e}")


def check_blocks(q, v, off_by, what=""):
    """Blocks within half a step of the values (half a unit of 4 significant bits, or of the smallest element; the scale may be the
    next one where the largest value is at its border), which are off by so much themselves."""
    if not len(v):
        return
    b = host(q.scales)[:, :q.K // 32].astype(np.float64)
    most = (np.abs(v) + off_by).reshape(len(v), -1, 32).max(-1)
    top = 448 * 2.0 ** (b - 127)
    assert np.all(most <= top * (1 + 1e-6) + off_by.reshape(len(v), -1, 32).max(-1) * 2), what
    assert np.all((b == 0) | (most * (1 + 1e-6) >= top / 2)), what
    near(gq.dequantize_mx(q), v, 2.0 ** -4 * np.abs(v) + np.repeat(2.0 ** (b - 127 - 10), 32, -1) + 1.1 * off_by, what)


@pytest.mark.parametrize("counts", COUNTS[:-1], ids=str)
@pytest.mark.parametrize("F, K", [(32, 32), (160, 96), (544, 2304)])
def test_gated_unit(counts, F, K):
    E, T = len(counts), 50
    plan, off, token, R = expert_case(F, counts, T, behind=3)
    w, W = weights(F, 2 * E, F, K)
    x, X = mx(2 * rows(K, T, K)[1])
    got = gq.swiglu_mxfp4(w, x, plan, gather=True)
    codes, scales = got.codes[:R], got.scales[:R]
    assert not scales[:, F // 32:].any()
    v, tol = np.zeros((R, F)), np.zeros((R, F))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        v[r], tol[r] = ref.swiglu(X[token[r]], W[2 * e], W[2 * e + 1])
    check_blocks(gq.MXRows(codes.contiguous(), scales.contiguous()), v, tol)
    # without a plan, and the same rows in the plan's order without gathering: the same bits
    if E == 1:
        dense = gq.swiglu_mxfp4(w, gq.MXRows(x.codes[plan.rows[:R].long()].contiguous(), x.scales[plan.rows[:R].long()].contiguous()))
        assert torch.equal(dense.codes, codes) and torch.equal(dense.scales, scales)
    idx = plan.rows.long()
    again = gq.swiglu_mxfp4(w, gq.MXRows(x.codes[idx].contiguous(), x.scales[idx].contiguous()), plan)
    assert torch.equal(again.codes[:R], codes) and torch.equal(again.scales[:R], scales)


def test_gated_unit_of_extreme_values():
    """Gates far below 0 (silu 0), rows of zeros, a NaN row."""
    F, K = 64, 32
    w, W = weights(9, 2, F, K)
    X = np.zeros((40, K))
    X[1:20] = 300 * np.random.default_rng(1).standard_normal((19, K))
    X[20:] = 2.0 ** -100 * np.random.default_rng(2).standard_normal((20, K))
    q, X = mx(X)
    q.codes[30] = 0
    q.scales[30] = 255
    X[30] = np.nan
    got = gq.swiglu_mxfp4(w, q)
    v = host(gq.dequantize_mx(got))
    assert np.isnan(v[30]).all() and not np.isnan(np.delete(v, 30, 0)).any() and not v[0].any()
    keep = np.delete(np.arange(40), 30)
    want, tol = ref.swiglu(X[keep], W[0], W[1])
    idx = dev(keep)
    check_blocks(gq.MXRows(got.codes[idx].contiguous(), got.scales[idx].contiguous()), want, tol + 2.0 ** -140)


@pytest.mark.parametrize("mean", [4, 40])
def test_plans_out_of_range(mean):
    """Experts whose offsets are wrong have no rows, indices outside the activations read as zeros, and both are reported."""
    E, N, K, T = 4, 130, 96, 20
    w, W = weights(1, E, N, K)
    x, X = mx(rows(2, T, K)[1])
    R = E * mean
    token = np.random.default_rng(0).integers(0, T, R).astype(np.int32)
    good = np.arange(E + 1, dtype=np.int32) * mean
    for case in range(4):
        off, tok = good.copy(), token.copy()
        if case == 0:
            off[2] = 1                       # expert 1 has a negative number of rows, expert 2 more than its share
        elif case == 1:
            off[4] = R + 1
        elif case == 2:
            off[0] = -5
        else:
            tok[[0, mean, R - 1]] = [-1, T, 2 ** 31 - 1]
        plan = gq.ExpertPlan(dev(off), dev(tok), dev(np.zeros((1, 1), np.int32)))
        out = torch.full((R, N), 5.0, device="cuda")
        gq.mul_mat_mxfp4(w, x, plan, gather=True, out=out)
        assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
        lost = {0: [1], 1: [3], 2: [0], 3: []}[case]
        written = np.zeros(R, bool)
        for e in range(E):
            if e in lost:
                continue
            r = slice(off[e], off[e + 1])
            written[r] = True
            there = (tok[r] >= 0) & (tok[r] < T)
            want, S = ref.product(X[np.where(there, tok[r], 0)] * there[:, None], W[e])
            if case != 0:                    # (rows that two experts claim hold what one of them makes of them)
                near(out[r], want, ref.product_tolerance(K) * S, f"case {case} expert {e}")
        if case != 0:
            assert (out[dev(~written)] == 5).all()
    assert gq.gq_last_error() == gq.GQ_OK


# ---- routing -----------------------------------------------------------------------------------

ROUTES = [dict(E=1, k=1), dict(E=7, k=3, score="sigmoid", bias=True), dict(E=40, k=4, score="sigmoid", bias=True, groups=5, top_groups=2, best=2),
          dict(E=96, k=10, bias=True, groups=32, top_groups=7), dict(E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4, best=2, factor=2.5),
          dict(E=512, k=32, bias=True, renormalize=False), dict(E=1000, k=10), dict(E=1024, k=32, score="sigmoid", groups=2, top_groups=1, best=2),
          dict(E=64, k=32, score="sigmoid", bias=True), dict(E=128, k=2, groups=4, top_groups=2, best=2, renormalize=False)]


def check_route(z, c, got, used=None):
    ids, w, plan = got
    E, k = c["E"], c["k"]
    used = len(z) if used is None else used
    opt = {n: c[n] for n in ("score", "groups", "top_groups", "best", "renormalize", "factor") if n in c}
    want, ww = ref.route(host(z)[:used], k, bias=None if c.get("bias") is None else host(c["bias"]), **opt)
    all_ids = np.full((len(z), k), -1, np.int32)
    all_ids[:used] = want
    assert np.array_equal(host(ids), all_ids)
    zz = np.where(np.isfinite(host(z)[:used]), host(z)[:used], 0)
    spread = np.abs(zz).max() * 2 if zz.size else 0
    near(host(w)[:used], ww, (spread + E / 32 + 16) * U * np.abs(ww) + 1e-38)
    assert not host(w)[used:].any()
    off, rows_, pos = ref.plan(all_ids, E)
    assert np.array_equal(host(plan.offsets), off) and np.array_equal(host(plan.pos), pos)
    assert np.array_equal(host(plan.rows)[:len(rows_)], rows_)


def router(c):
    names = dict(score="score", groups="groups", top_groups="top_groups", best="group_best", renormalize="renormalize", factor="factor")
    return gq.Router(c["E"], c["k"], bias=c.get("bias"), **{names[n]: c[n] for n in names if n in c})


@pytest.mark.parametrize("c", ROUTES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 31, 32, 33, 700])
def test_route(c, dtype, T):
    rng = np.random.default_rng(T)
    c = dict(c)
    if c.get("bias"):
        c["bias"] = dev(0.1 * rng.standard_normal(c["E"]).astype(np.float32))
    wide = dev(1.5 * rng.standard_normal((T, c["E"] + 8 + T % 2)).astype(np.float32), DT[dtype])
    wide = wide[:, :c["E"] + 8]
    z = wide[:, 8:]                                                            # any stride
    check_route(z, c, gq.route(z, router(c)))


@pytest.mark.parametrize("T", [20, 100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("grouped", [False, True])
def test_route_ties_masks_and_close_values(T, score, grouped):
    """Equal logits, logits of -infinity and NaN, biases that make values equal or closer than f32 can tell."""
    E, k = 64, 6
    rng = np.random.default_rng(T)
    z = rng.integers(-3, 3, (T, E)).astype(np.float32)                        # many ties
    z[1], z[2, ::2], z[3, 5], z[4, :E - 2] = -np.inf, -np.inf, np.nan, -np.inf
    z[5] = 1.0
    z[6] = 1 + np.arange(E) * 2.0 ** -23                                      # neighbouring f32 values
    z[7] = -np.arange(E) * 1e-7
    opt = dict(groups=8, top_groups=3, best=2) if grouped else {}
    bias = dev((1e-8 * rng.integers(-3, 3, E)).astype(np.float32))
    for b in (None, bias, torch.zeros(E, device="cuda")):
        c = dict(E=E, k=k, score=score, bias=b, **opt)
        check_route(dev(z), c, gq.route(dev(z), router(c)))


@pytest.mark.parametrize("T, used", [(9, 0), (9, 4), (9, 9), (300, 0), (300, 137), (300, 300)])
def test_route_of_a_padded_batch(T, used):
    c = dict(E=32, k=4)
    z = dev(np.random.default_rng(T).standard_normal((T, 32)).astype(np.float32))
    z[used:] = float("nan")
    check_route(z, c, gq.route(z, router(c), used=dev(np.array([used], np.int32))), used)
    for bad, counts in ((-1, 0), (T + 1, T)):
        y = torch.randn((T, 32), device="cuda")
        check_route(y, c, gq.route(y, router(c), used=dev(np.array([bad], np.int32))), counts)
        assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG


# ---- together ----------------------------------------------------------------------------------


@pytest.mark.parametrize("rtype, otype", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), (None, "f32")])
@pytest.mark.parametrize("T, k, N", [(1, 1, 8), (7, 8, 264), (300, 3, 4096)])
def test_combine(rtype, otype, T, k, N):
    rng = np.random.default_rng(T)
    R = T * k
    y = rng.standard_normal((R, N)).astype(np.float32)
    pos = rng.permutation(R).astype(np.int32).reshape(T, k)
    if T > 1:
        pos[1, 0], pos[2] = -1, R                                              # outside: adds nothing
    w = rng.random((T, k)).astype(np.float32)
    plan = gq.ExpertPlan(dev(np.array([0, R], np.int32)), dev(np.zeros(R, np.int32)), dev(pos))
    res = None if rtype is None else dev(rng.standard_normal((T, N + 8)).astype(np.float32), DT[rtype])[:, :N]
    got = gq.experts_combine(dev(y), plan, dev(w), residual=res, dtype=DT[otype])
    there = (pos >= 0) & (pos < R)
    terms = np.where(there, w.astype(np.float64), 0)[..., None] * y.astype(np.float64)[np.where(there, pos, 0)]
    base = 0 if res is None else host(res)
    want, S = terms.sum(1) + base, np.abs(terms).sum(1) + np.abs(base)
    near(got, want, (k + 1) * U * S + (BF * np.abs(want) if otype == "bf16" else 0))
    if rtype == otype and rtype:
        assert torch.equal(gq.experts_combine(dev(y), plan, dev(w), residual=res, out=res), got)     # in place


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 7, 8, 9, 16, 17])
def test_product_of_values_is_the_product_of_their_blocks(M, dtype):
    """Bit for bit, however the rows are quantized on the way: short, ragged and long rows, one tile and many, special blocks."""
    for N, K, ld in ((1, 32, 32), (130, 96, 104), (300, 992, 992), (128 * 3, 4096 + 160, 4256 + 8), (20011, 320, 320), (130, 15008, 15008)):
        w, _ = weights(M, 1, N, K)
        room = torch.randn((M, ld), generator=torch.Generator("cuda").manual_seed(K + M), device="cuda")
        room[:, K:] = float("nan")                       # between the rows
        x = room.to(dtype)[:, :K]
        x[M // 2, :32] = 0
        x[0, 32:64] *= 1e-38
        if K > 64 and M > 1:
            x[M - 1, 64 + M] = float("inf")
        got = gq.mul_mat_mxfp4(w, x)
        want = gq.mul_mat_mxfp4(w, gq.quantize_mx(x))
        assert torch.equal(torch.nan_to_num(got, nan=7.5), torch.nan_to_num(want, nan=7.5)), (N, K)
        assert torch.isnan(want[:M - 1]).sum() == 0 and (M == 1 or K <= 64 or torch.isnan(want[M - 1]).all())
    assert gq.gq_last_error() == gq.GQ_OK


def test_product_of_few_values_needs_no_workspace():
    """Captured on a stream that never ran a product."""
    w, _ = weights(3, 1, 256, 512)
    x = torch.randn((2, 512), device="cuda")
    want = gq.mul_mat_mxfp4(w, x)
    out = torch.zeros_like(want)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        gq.mul_mat_mxfp4(w, x, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("E,mean", [(5, 3), (70, 2), (5, 20)])
def test_ranges_that_overlap_belong_to_the_first_expert(E, mean):
    """Offsets that go back: no row is computed for two experts, and the experts behind keep theirs."""
    N, K = 130, 96
    w, W = weights(1, E, N, K)
    R = E * mean
    x, X = mx(rows(2, R, K)[1])
    off = np.arange(E + 1, dtype=np.int32) * mean
    off[E - 2] = 0                                       # expert E - 3 has less than none, expert E - 2 what others have
    plan = gq.ExpertPlan(dev(off), dev(np.arange(R, dtype=np.int32)), dev(np.zeros((1, 1), np.int32)))
    for gather in (True, False):
        out = torch.full((R, N), 5.0, device="cuda")
        gq.mul_mat_mxfp4(w, x, plan, gather=gather, out=out)
        assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
        for e in range(E):
            r = slice(e * mean, (e + 1) * mean)
            if e in (E - 3, E - 2):
                assert (out[r] == 5).all()
                continue
            want, S = ref.product(X[r], W[e])
            near(out[r], want, ref.product_tolerance(K) * S, f"expert {e}")
    assert gq.gq_last_error() == gq.GQ_OK


class Block:
    """norm, router, experts, sum: one feed-forward layer of experts, as it is used."""

    def __init__(self, K, F, E, k, seed=0):
        rng = np.random.default_rng(seed)
        self.K, self.E = K, E
        self.norm = dev(1 + 0.1 * rng.standard_normal(K).astype(np.float32))
        self.gate = dev((rng.standard_normal((E, K)) / np.sqrt(K)).astype(np.float16))
        self.up, self.U = weights(seed + 1, 2 * E, F, K)
        self.down, self.D = weights(seed + 2, E, K, F)
        self.router = gq.Router(E, k)

    def __call__(self, x, residual, used=None):
        h, q, y = gq.rms_norm_mx(x, self.norm, 1e-5, residual=residual, y_dtype=torch.float32)
        logits = gq.mul_mat_f16_f32(self.gate, y)
        ids, w, plan = gq.route(logits, self.router, used)
        act = gq.swiglu_mxfp4(self.up, q, plan, gather=True)
        return gq.experts_combine(gq.mul_mat_mxfp4(self.down, act, plan), plan, w, residual=h), (h, q, logits, ids, w, plan, act)

    def check(self, out, parts, used):
        """Each step from what the step before gave."""
        h, q, logits, ids, w, plan, act = parts
        X = host(gq.dequantize_mx(q))
        codes, b = ref.quantize(ref.norm(host(h), host(self.norm), 1e-5), ref.E4M3)
        assert np.array_equal(host(q.codes) & 127, codes & 127)
        check_route(logits, dict(E=self.E, k=self.router.top_k), (ids, w, plan), used)
        off, token, pos = host(plan.offsets), host(plan.rows), host(plan.pos)
        R = off[-1]
        v, tol, y, S = np.zeros((R, act.K)), np.zeros((R, act.K)), np.zeros((R, self.K)), np.zeros((R, self.K))
        A = host(gq.dequantize_mx(act))
        for e in range(self.E):
            r = slice(off[e], off[e + 1])
            v[r], tol[r] = ref.swiglu(X[token[r]], self.U[2 * e], self.U[2 * e + 1])
            y[r], S[r] = ref.product(A[r], self.D[e])
        check_blocks(gq.MXRows(act.codes[:R].contiguous(), act.scales[:R].contiguous()), v, tol)
        there = pos >= 0
        y, S = np.append(y, np.zeros((1, self.K)), 0), np.append(S, np.zeros((1, self.K)), 0)
        terms = np.where(there, host(w), 0)[..., None] * y[np.where(there, pos, R)]
        off_by = (np.where(there, host(w), 0)[..., None] * S[np.where(there, pos, R)]).sum(1)
        near(out, terms.sum(1) + host(h), ref.product_tolerance(act.K) * off_by + 12 * U * (np.abs(terms).sum(1) + np.abs(host(h))))


@pytest.mark.parametrize("T, K, F, E, k", [(1, 256, 96, 8, 2), (9, 512, 160, 16, 4), (90, 288, 64, 5, 3), (600, 256, 128, 4, 2)])
def test_a_layer_of_experts(T, K, F, E, k):
    block = Block(K, F, E, k)
    out, parts = block(rows(T, T, K)[0], rows(T + 1, T, K)[0])
    block.check(out, parts, T)


@pytest.mark.parametrize("T, used", [(6, (6, 2, 0, 5)), (120, (120, 7, 0, 99))])
def test_captured_and_replayed(T, used):
    """One captured step, replayed with other tokens and other numbers of them, beside a second graph of another block on another
    stream; each replay's results are those of the step run by itself."""
    blocks, graphs = [Block(256, 96, 8, 3, seed=s) for s in (0, 10)], []
    for block in blocks:
        s = dict(x=torch.empty((T, 256), device="cuda"), r=torch.empty((T, 256), device="cuda"), used=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 stream=torch.cuda.Stream(), graph=torch.cuda.CUDAGraph())
        s["x"].normal_()
        s["r"].normal_()
        s["stream"].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s["stream"]):
            block(s["x"], s["r"], s["used"])                                   # the workspace is there before the capture
        s["stream"].synchronize()
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            s["out"], s["parts"] = block(s["x"], s["r"], s["used"])
        graphs.append(s)
    for turn, n in enumerate(used):
        for i, s in enumerate(graphs):
            s["x"].copy_(rows(turn * 2 + i, T, 256)[0])
            s["used"].fill_(n)
        torch.cuda.synchronize()
        for s in graphs:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        for block, s in zip(blocks, graphs):
            out, parts = block(s["x"], s["r"], s["used"])
            assert torch.equal(out, s["out"]) and torch.equal(parts[3], s["parts"][3])
            assert torch.equal(out[n:], parts[0][n:])                          # padding: the residual alone
        block.check(out, parts, n)


def test_a_capture_that_needs_more_workspace_is_refused():
    w, _ = weights(0, 1, 64, 8192)
    x = torch.randn((3000, 8192), device="cuda")
    out = torch.empty((3000, 64), device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with pytest.raises(gq.GQError) as e, torch.cuda.graph(g, stream=s):
        gq.mul_mat_mxfp4(w, x, out=out)
    assert e.value.status == gq.GQ_ERR_NO_MEMORY


def test_many_calls_in_a_row_on_two_streams():
    """Products of several sizes, over and over, on two streams at once: the same bits each time."""
    block = Block(512, 192, 8, 2)
    big = Block(256, 64, 4, 2, seed=5)
    cases = [(block, rows(1, 3, 512)[0]), (big, rows(2, 800, 256)[0]), (block, rows(3, 70, 512)[0])]
    want = [b(x, x)[0].clone() for b, x in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(60):
        with torch.cuda.stream(streams[i % 2]):
            j = i % 3
            got.append((j, cases[j][0](cases[j][1], cases[j][1])[0]))
    torch.cuda.synchronize()
    for j, out in got:
        assert torch.equal(out, want[j])


def test_results_do_not_depend_on_the_batch():
    """A row's product does not change with the rows around it, as long as the same kernel does them."""
    w, _ = weights(0, 1, 384, 1536)
    x, _ = rows(4, 700, 1536)
    whole = gq.mul_mat_mxfp4(w, x)
    assert torch.equal(gq.mul_mat_mxfp4(w, x[100:500].contiguous()), whole[100:500])
