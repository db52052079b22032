"""examples/paged_decode.py at small sizes: products, cache, attention and eviction together."""
import importlib.util
import os

import pytest

import quantized_skinny_matmul_gb300 as gq

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")


# From the definition: scores carry 2^-24 for each of D products and of the fp16 pairs (2^-22), times
# |z| of tens; relative to the largest output element that is well below 1e-4.
@pytest.mark.parametrize("kind,D,page,budget", [(gq.GQ_KV_I8, 128, 32, 6), (gq.GQ_KV_E4M3, 64, 16, 4)])
def test_decode_within_a_budget(kind, D, page, budget):
    spec = importlib.util.spec_from_file_location("paged_decode", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    _, pages, err = example.run(batch=3, prompt=150, steps=70, budget=budget, hidden=512, heads=8, kv_heads=2, D=D,
                                page=page, kind=kind)
    assert err < 1e-4
    # 71 tokens after prompts of 150, 113 and 76; a sequence that never had more pages keeps them all
    assert pages == [min(budget, -(-(n + 71) // page)) for n in (150, 113, 76)]
