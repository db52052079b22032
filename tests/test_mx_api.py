"""What the microscaled entry points and their binding refuse, before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

import quantized_skinny_matmul_gb300 as gq

FAKE, ODD = 0x10000, 0x10008            # never dereferenced: the checks fail first
F32, BF16, E2M1, E4M3 = gq.GQ_TYPE_F32, gq.GQ_TYPE_BF16, gq.GQ_MX_E2M1, gq.GQ_MX_E4M3


@pytest.fixture(scope="module")
def lib():
    from quantized_skinny_matmul_gb300 import _build
    _build.build()
    return gq.lib()


def refused(call, good, bad, status=gq.GQ_ERR_INVALID_ARG):
    """Each (place, value) of `bad` in the arguments `good` is refused."""
    for i, v in bad:
        args = list(good)
        args[i] = v
        assert call(*args) == status, (call.__name__, i, v)
        assert gq.lib().gq_last_error_message()


def pointers(call, good, places):
    for i in places:
        refused(call, good, [(i, 0)])
        refused(call, good, [(i, ODD)], gq.GQ_ERR_MISALIGNED)


def test_sizes(lib):
    assert [gq.gq_mx_scale_cols(K) for K in (32, 512, 544, 4096)] == [16, 16, 32, 128]
    assert gq.gq_mx_scale_cols(0) == gq.gq_mx_scale_cols(33) == gq.gq_mx_scale_cols(-32) == 0
    assert gq.gq_mxfp4_repacked_bytes(1, 128, 128) == 8704 and gq.gq_mxfp4_repacked_bytes(3, 129, 160) == 3 * 4 * 8704
    for bad in ((0, 128, 128), (1, 0, 128), (1, 128, 100), (2049, 128, 128), (2000, 128 * 1024, 128 * 1024)):
        assert gq.gq_mxfp4_repacked_bytes(*bad) == 0


def test_rows(lib):
    q = (FAKE, 64, F32, E4M3, FAKE, FAKE, 3, 64, None)
    refused(lib.gq_quantize_mx, q, [(1, 60), (1, 66), (2, 2), (3, 2), (6, 0), (7, 48), (7, 0)])
    refused(lib.gq_quantize_mx, (FAKE, 68, BF16, E4M3, FAKE, FAKE, 3, 64, None), [(1, 68)])      # rows of bf16 start on 16 bytes
    pointers(lib.gq_quantize_mx, q, (0, 4, 5))
    d = (FAKE, FAKE, E2M1, FAKE, BF16, 3, 64, None)
    refused(lib.gq_dequantize_mx, d, [(2, -1), (4, 7), (5, 0), (6, 40)])
    pointers(lib.gq_dequantize_mx, d, (0, 1, 3))
    n = (FAKE, 64, FAKE, 64, F32, FAKE, 1e-5, FAKE, 64, FAKE, F32, FAKE, FAKE, 3, 64, None)
    refused(lib.gq_rms_norm_mx, n, [(1, 63), (3, 32), (4, 5), (6, -1.0), (6, float("nan")), (6, float("inf")), (8, 0), (10, 9),
                                    (11, 0), (12, 0), (13, -1), (14, 63), (14, 32800)])
    refused(lib.gq_rms_norm_mx, (FAKE, 64, 0, 64, F32, 0, 1e-5, 0, 64, 0, F32, 0, 0, 3, 64, None), [(0, FAKE)])   # no output
    refused(lib.gq_rms_norm_mx, n, [(i, ODD) for i in (0, 2, 5, 7, 9, 11, 12)], gq.GQ_ERR_MISALIGNED)


def test_weights(lib):
    r = (FAKE, FAKE + (1 << 20), FAKE + (1 << 24), 2, 128, 128, None)
    refused(lib.gq_repack_mxfp4, r, [(3, 0), (3, 3000), (4, 0), (5, 100), (2, FAKE), (2, FAKE + (1 << 20)), (2, FAKE + 64)])
    pointers(lib.gq_repack_mxfp4, r, (0, 1, 2))


def mx_rows(rows=40, codes=FAKE, scales=FAKE):
    return ctypes.pointer(gq.MXRowsStruct(rows, codes, scales))


def plan(E=4, R=40, offsets=FAKE, rows=FAKE):
    return ctypes.pointer(gq.ExpertRowsStruct(E, R, offsets, rows))


def test_products(lib):
    m = (FAKE, mx_rows(), plan(), FAKE, 256, F32, 256, 64, None)
    refused(lib.gq_mul_mat_mxfp4_mx, m, [(1, None), (1, mx_rows(0)), (1, mx_rows(1 << 30)), (1, mx_rows(codes=0)), (1, mx_rows(scales=0)),
                                         (2, plan(0)), (2, plan(1025)), (2, plan(R=0)), (2, plan(offsets=0)), (2, plan(R=41, rows=0)),
                                         (4, 255), (5, 3), (6, 0), (7, 50), (7, 0)])
    refused(lib.gq_mul_mat_mxfp4_mx, m, [(1, mx_rows(codes=ODD)), (1, mx_rows(scales=ODD)), (2, plan(offsets=FAKE + 2)),
                                         (2, plan(rows=FAKE + 1))], gq.GQ_ERR_MISALIGNED)
    pointers(lib.gq_mul_mat_mxfp4_mx, m, (0, 3))
    s = (FAKE, mx_rows(), plan(), FAKE, FAKE, 96, 64, None)
    refused(lib.gq_swiglu_mxfp4_mx, s, [(1, None), (5, 100), (5, 0), (6, 16), (2, plan(0))])
    pointers(lib.gq_swiglu_mxfp4_mx, s, (0, 3, 4))
    x = (FAKE, FAKE, 64, F32, FAKE, 256, F32, 3, 256, 64, None)
    refused(lib.gq_mul_mat_mxfp4, x, [(2, 60), (2, 66), (3, 4), (5, 250), (6, 4), (7, 0), (8, 0), (9, 33)])
    pointers(lib.gq_mul_mat_mxfp4, x, (0, 1, 4))


def router(E=64, top_k=8, score=0, groups=8, top_groups=4, best=2, renorm=1, factor=1.0, bias=FAKE):
    return ctypes.pointer(gq.RouterStruct(E, top_k, score, groups, top_groups, best, renorm, factor, bias))


def test_routing(lib):
    r = (router(), FAKE, 64, F32, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, None)
    refused(lib.gq_route, r, [(0, None), (0, router(E=0)), (0, router(E=1025, groups=1, top_groups=1)), (0, router(top_k=0)), (0, router(top_k=33)),
                              (0, router(E=64, groups=32, top_groups=1, top_k=3)), (0, router(score=2)), (0, router(groups=3)),
                              (0, router(groups=64)), (0, router(top_groups=0)), (0, router(top_groups=9)), (0, router(best=3)),
                              (0, router(factor=float("inf"))), (2, 63), (3, 2), (10, 0), (10, 1 << 28), (5, 0), (6, 0), (7, 0), (8, 0), (9, 0)])
    refused(lib.gq_route, r, [(0, router(bias=ODD)), (1, ODD), (5, ODD), (6, ODD), (7, ODD), (8, ODD), (9, ODD), (4, FAKE + 2)], gq.GQ_ERR_MISALIGNED)
    c = (FAKE, 40, FAKE, FAKE, 8, FAKE, 64, F32, FAKE, 64, F32, 5, 64, None)
    refused(lib.gq_experts_combine, c, [(1, 0), (4, 0), (4, 33), (6, 60), (7, 2), (9, 66), (10, 5), (11, 0), (12, 60)])
    pointers(lib.gq_experts_combine, c, (0, 2, 3, 8))
    refused(lib.gq_experts_combine, c, [(5, ODD)], gq.GQ_ERR_MISALIGNED)


class OnGpu:
    """A tensor that says it lives on the GPU."""

    def __init__(self, t):
        self.t, self.shape, self.dtype, self.is_cuda, self.device = t, t.shape, t.dtype, True, t.device

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_objects(lib):
    codes, scales = OnGpu(torch.zeros((3, 64), dtype=torch.uint8)), OnGpu(torch.zeros((3, 16), dtype=torch.uint8))
    x = gq.MXRows(codes, scales)
    assert (x.rows, x.K, x.kind) == (3, 64, E4M3) and x.codes is codes and x.scales is scales
    c = x.by_ref.contents
    assert (c.rows, c.codes, c.scales) == (3, codes.data_ptr(), scales.data_ptr())
    assert gq.MXRows(codes, scales, E2M1).K == 128
    for bad in (torch.zeros((3, 15), dtype=torch.uint8), torch.zeros((2, 16), dtype=torch.uint8), torch.zeros((3, 16), dtype=torch.int8)):
        with pytest.raises(ValueError, match="scales"):
            gq.MXRows(codes, OnGpu(bad))
    with pytest.raises(ValueError, match="CUDA"):
        gq.MXRows(codes.t, scales)
    e = gq.MXRows.empty(5, 544, E2M1, "cpu")
    assert e.codes.shape == (5, 272) and e.scales.shape == (5, 32) == (5, gq.gq_mx_scale_cols(544))
    assert e.codes.data_ptr() == e.codes_ptr and e.scales.data_ptr() == e.scales_ptr
    for rows, K in ((0, 64), (3, 0), (3, 48)):
        with pytest.raises(ValueError, match="32"):
            gq.MXRows.empty(rows, K, E4M3, "cpu")

    ints = lambda *s: OnGpu(torch.zeros(s, dtype=torch.int32))   # noqa: E731
    p = gq.ExpertPlan(ints(5), ints(12), ints(6, 2))
    assert (p.E, p.R) == (4, 12)
    assert p.by_ref(True).contents.rows == p.rows.data_ptr() and not p.by_ref(False).contents.rows
    with pytest.raises(ValueError, match="pos"):
        gq.ExpertPlan(ints(5), ints(12), OnGpu(torch.zeros((6, 2))))
    w = gq.MXWeights(OnGpu(torch.zeros(4 * 8704, dtype=torch.uint8)), 4, 100, 64)
    with pytest.raises(ValueError, match="data"):
        gq.MXWeights(OnGpu(torch.zeros(8704, dtype=torch.uint8)), 4, 100, 64)
    for args, what in (((w, gq.MXRows(codes, scales, E2M1), p), "e4m3"), ((w, x, None), "matrices"), ((w, x, gq.ExpertPlan(ints(4), ints(3), ints(3, 1))), "matrices")):
        with pytest.raises(ValueError, match=what):
            gq.mul_mat_mxfp4(*args)
    with pytest.raises(ValueError, match="matrices"):
        gq.swiglu_mxfp4(w, x, p)
    with pytest.raises(ValueError, match="plan"):
        gq.mul_mat_mxfp4(gq.MXWeights(OnGpu(torch.zeros(8704, dtype=torch.uint8)), 1, 100, 64), x, gather=True)
    with pytest.raises(ValueError, match="out"):
        gq.mul_mat_mxfp4(w, x, p, out=OnGpu(torch.zeros((12, 99))))
    with pytest.raises(ValueError, match="score"):
        gq.Router(8, 2, score="tanh")
    with pytest.raises(ValueError, match="bias"):
        gq.Router(8, 2, bias=OnGpu(torch.zeros(7)))
    with pytest.raises(ValueError, match="experts"):
        gq.route(OnGpu(torch.zeros((3, 7))), gq.Router(8, 2))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        gq.quantize_mx(OnGpu(torch.zeros((3, 64), dtype=torch.float16)))
    with pytest.raises(ValueError, match="contiguous"):
        gq.quantize_mx(OnGpu(torch.zeros((64, 3)).T))
    with pytest.raises(ValueError, match="residual"):
        gq.rms_norm_mx(OnGpu(torch.zeros((3, 64))), None, 1e-5, residual=OnGpu(torch.zeros((3, 64), dtype=torch.bfloat16)))


def test_what_calls_point_at_cannot_be_changed(lib):
    """The structs hold addresses and sizes: a field that could be assigned would leave them behind."""
    x = gq.MXRows.empty(5, 64, E4M3, "cpu")
    p = gq.ExpertPlan(*(OnGpu(torch.zeros(n, dtype=torch.int32)) for n in ((5,), (12,), (6, 2))))
    r = gq.Router(8, 2)
    for thing, names in ((x, ("rows", "K", "kind", "codes", "scales", "codes_ptr")), (p, ("E", "R", "offsets", "rows", "pos")),
                         (r, ("E", "top_k", "bias", "struct"))):
        for name in names:
            before = getattr(thing, name)
            with pytest.raises(AttributeError):
                setattr(thing, name, 3)
            assert getattr(thing, name) is before
