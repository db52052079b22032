"""Run with GQ_LIBRARY naming the GQ_DEBUG build (tests/test_gpu_debug_build_mx.py does): the router and the
products of microscaled blocks, every tile shape, with plans and without; the status word must stay clean."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import numpy as np  # noqa: E402
import torch  # noqa: E402

import mx_ref as ref  # noqa: E402
import quantized_skinny_matmul_gb300 as gq  # noqa: E402


def blocks(seed, rows, K, kind):
    q = gq.quantize_mx(torch.randn((rows, K), generator=torch.Generator("cuda").manual_seed(seed), device="cuda") / K ** 0.5, kind)
    return q, gq.dequantize_mx(q).double().cpu().numpy()


def main():
    assert gq.LIB_PATH == os.environ["GQ_LIBRARY"], gq.LIB_PATH
    for M, N, K in ((1, 130, 4096), (2, 300, 96), (9, 700, 1056), (16, 128, 512), (50, 257, 2080), (300, 20000, 160), (700, 2300, 1056)):
        wq, W = blocks(N, N, K, gq.GQ_MX_E2M1)
        x = 4 * torch.randn((M, K), generator=torch.Generator("cuda").manual_seed(M), device="cuda")
        got = gq.mul_mat_mxfp4(gq.repack_mxfp4(wq.codes, wq.scales, N, K), x)
        want, S = ref.product(gq.dequantize_mx(gq.quantize_mx(x)).double().cpu().numpy(), W)
        assert np.all(np.abs(got.cpu().numpy() - want) <= ref.product_tolerance(K) * S), (M, N, K)
    for T, E, k, F, K, score, groups in ((1, 8, 2, 96, 256, "softmax", 1), (33, 40, 4, 160, 288, "sigmoid", 5), (300, 8, 3, 544, 160, "softmax", 1),
                                         (900, 4, 2, 96, 256, "sigmoid", 2)):
        uq, U = blocks(1, 2 * E * F, K, gq.GQ_MX_E2M1)
        dq, D = blocks(2, E * K, F, gq.GQ_MX_E2M1)
        x, X = blocks(3, T, K, gq.GQ_MX_E4M3)
        logits = torch.randn((T, E), generator=torch.Generator("cuda").manual_seed(4), device="cuda")
        bias = torch.linspace(-0.1, 0.1, E, device="cuda")
        ids, w, plan = gq.route(logits, gq.Router(E, k, score, bias, groups, groups, 1))
        act = gq.swiglu_mxfp4(gq.repack_mxfp4(uq.codes, uq.scales, F, K), x, plan, gather=True)
        y = gq.mul_mat_mxfp4(gq.repack_mxfp4(dq.codes, dq.scales, K, F), act, plan).cpu().numpy()
        A, D = gq.dequantize_mx(act).double().cpu().numpy(), D.reshape(E, K, F)
        want = ref.route(logits.cpu().numpy(), k, score, bias.cpu().numpy())[0]
        assert np.array_equal(ids.cpu().numpy(), want)
        pos = plan.pos.cpu().numpy()
        for e in range(E):
            r = pos[want == e]
            out, S = ref.product(A[r], D[e])
            assert np.all(np.abs(y[r] - out) <= ref.product_tolerance(F) * S), (T, e)
    torch.cuda.synchronize()
    status = gq.gq_last_error()
    assert status == gq.GQ_OK, f"gq_last_error() = {status}: {gq.lib().gq_last_error_message().decode()}"
    print("debug build clean")


if __name__ == "__main__":
    main()
