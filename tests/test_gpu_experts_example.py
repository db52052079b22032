"""examples/experts.py at small sizes: norm, scores, router, experts and their sum together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "experts.py")


# Sums of K = 256 and fewer: tensor-core sums within (K / 32 + 1) * 2^-22 + (K / 512 + 8) * 2^-24 < 2.7e-6 of sum |terms|, which
# is about 0.64 sqrt(K) = 10 for such rows, so 2.7e-5 per value; the unit's is times |up| and |silu(gate)|, both below 5 here,
# against a largest value of a block near 1: below 5e-4.  The output's, against a largest of 1 or more, with weights whose
# sum is 1: below 1e-4.
@pytest.mark.parametrize("hidden,inner,experts,top_k,prompt", [(256, 96, 8, 2, 70), (224, 160, 20, 6, 33)])
def test_a_layer_of_experts(hidden, inner, experts, top_k, prompt):
    spec = importlib.util.spec_from_file_location("experts_example", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    us, err, unit = example.run(hidden, inner, experts, top_k, prompt, steps=7)
    assert us > 0
    assert err < 1e-4
    assert unit < 5e-4
