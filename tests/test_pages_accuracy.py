"""The close bounds of the paged attention see what they are there for (no GPU)."""
import numpy as np
import pytest

import pages_accuracy as acc


@pytest.mark.parametrize("kind,G,D,P,new", [(0, 4, 128, 16, 1), (1, 1, 64, 32, 4), (0, 2, 128, 32, 48)])
def test_a_query_in_one_term_is_seen(kind, G, D, P, new):
    p = acc.few_keys(40, kind, G, D, P, new)
    want, _, E, S, _ = acc.reference(p)
    off = np.abs(acc.reference(p, acc.one_term(p["q"].astype(np.float64)))[0] - want)
    assert np.any(off > 2 * acc.few_keys_bound(D, S, E))


@pytest.mark.parametrize("kind,G,D,P,new", [(0, 4, 128, 16, 1), (1, 1, 64, 32, 4), (0, 2, 128, 32, 48)])
def test_weights_in_one_term_are_seen(kind, G, D, P, new):
    """The weights' part of the output alone: half a step of 11 bits, in turn up and down."""
    p = acc.few_keys(40, kind, G, D, P, new)
    _, _, E, S, _ = acc.reference(p)
    gen = np.random.default_rng(1)
    # a row's values times weights that are each off by up to 2^-12 of themselves, seen as a part of E
    share = gen.dirichlet(np.ones(40), size=E.shape)
    off = np.abs((share * gen.uniform(-1, 1, share.shape) * 2.0 ** -12).sum(-1)) * E
    assert np.any(off > 2 * acc.few_keys_bound(D, S, E))
