"""What the microscaled entry points and their binding refuse, at sizes that wrap around and with arguments
that contradict each other (no GPU: the checks come first)."""
import pytest
import torch

import quantized_skinny_matmul_gb300 as gq
from test_mx_api import FAKE, F32, OnGpu, lib, refused, router  # noqa: F401 (lib: a fixture)


def test_token_counts_that_wrap_around(lib):  # noqa: F811
    r = (router(), FAKE, 64, F32, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 5, None)
    refused(lib.gq_route, r, [(10, 1 << 27), (10, 1 << 61), (10, (1 << 61) + 1), (10, (1 << 63) - 1), (10, -1)])


def test_an_output_of_another_type_than_asked_for(lib):  # noqa: F811
    """`dtype` beside `out` has to be its type."""
    w = gq.MXWeights(OnGpu(torch.zeros(8704, dtype=torch.uint8)), 1, 100, 64)
    x = gq.MXRows(OnGpu(torch.zeros((3, 64), dtype=torch.uint8)), OnGpu(torch.zeros((3, 16), dtype=torch.uint8)))
    ints = lambda *s: OnGpu(torch.zeros(s, dtype=torch.int32))   # noqa: E731
    plan = gq.ExpertPlan(ints(5), ints(12), ints(6, 2))
    for out, dtype in ((torch.zeros((3, 100)), torch.bfloat16), (torch.zeros((3, 100), dtype=torch.bfloat16), torch.float32)):
        with pytest.raises(ValueError, match="out"):
            gq.mul_mat_mxfp4(w, x, dtype=dtype, out=OnGpu(out))
        with pytest.raises(ValueError, match="out"):
            gq.mul_mat_mxfp4(w, OnGpu(torch.zeros((3, 64))), dtype=dtype, out=OnGpu(out))
    with pytest.raises(ValueError, match="out"):
        gq.experts_combine(OnGpu(torch.zeros((12, 64))), plan, OnGpu(torch.zeros((6, 2))), dtype=torch.bfloat16, out=OnGpu(torch.zeros((6, 64))))
