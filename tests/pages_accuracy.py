"""Bounds of the paged attention's error that are close enough to see a lost term, and the problems they are for.

u = 2^-24.  A score is D / 16 tensor-core steps of products of exact codes and a query in two fp16 terms (4u), each
step adding with truncation (2u), then at most 8 roundings; a weight e^z carries the score's error and ex2's,
and its share of the denominator the same again.  Of few keys the sums add less than 64u.
"""
import numpy as np

import pages_ref as ref

U = 2.0 ** -24


def few_keys(seed, kind, G, D, P, new):
    """Some 40 keys, so that an error of a score shows, and rows of a prompt or of a single token."""
    return ref.problem(seed, kind, 6, 2, G, D, P, [40, 37, 41, 30, 45, 50], [new] * 6)


def few_keys_bound(D, S, E):
    return (2 * (4 + D / 8 + 8) * S[..., None] + 64) * U * E + 1e-30


def reference(p, q=None):
    names = ("kind", "P", "k", "ks", "v", "vs", "table", "base", "held", "seen", "cu")
    q = p["q"] if q is None else q
    return ref.attend(*(p[n] for n in names), q, ref.SCALE(q.shape[2]))


def one_term(x):
    """x in one fp16 term, the row's largest value being scaled to fp16's upper end."""
    up = 2.0 ** (14 - np.floor(np.log2(np.abs(x).max(-1, keepdims=True))))
    return (x * up).astype(np.float16).astype(np.float64) / up
