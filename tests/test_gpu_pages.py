"""The paged 8-bit KV cache (gq_kv_pages_append, gq_kv_pages_read, gq_attn_pages, gq_kv_pages_evict)
against the definitions written out in numpy and 64 bits (GPU only).

* Scales are one IEEE f32 division and codes are exact decisions on both sides: they must be
  equal, and so must everything eviction gives (integers and copied weights).
* Attention: f32 arithmetic against 64 bits.  With u = 2^-24, S the bound of the scores that
  count in a row (sum of |terms|, plus the distance bias, plus 4 cap) and E = sum p |v|:
    - a score is D / 16 MMA steps of exact fp16 products on the query's two terms (4u of each
      element), accumulated in f32 (2u a step), then the scales, the cap's tanh (relative 4u),
      the bias and the change to base 2 (a rounding each) and the subtraction of the maximum:
      at most 34 u S; ex2 is within 4u relative: a weight is off by 2 (34 S + 4) u with the
      denominator's share;
    - sums over T tokens in f32, at most T / 8 + 16 sequential additions per lane, MMA step and
      warp, counted at 2u, each weight being within 4u of its two fp16 terms; the running
      maximum rescales by powers that are within 4u each and the pieces' joins add as much.
  Together and doubled: 2 (70 S + T / 2 + 64) u times E (outputs) or the share (page weights).
"""
import math

import numpy as np
import pytest
import torch

import pages_ref as ref
import quantized_skinny_matmul_gb300 as gq
from test_gpu_parity import dev, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    assert gq.gq_last_error() == gq.GQ_OK


def cache_of(p):
    names = ("k", "v", "ks", "vs", "table", "base", "held", "seen")
    return gq.KVPages(p["kind"], *(dev(p[n]) for n in names))


def check_attention(p, out, w=None, weights=None, decay=1.0, **opt):
    D = p["q"].shape[2]
    T = int(max(p["held"] + np.diff(p["cu"])))
    want, ww, E, S, rel = ref.attend(p["kind"], p["P"], p["k"], p["ks"], p["v"], p["vs"], p["table"], p["base"], p["held"],
                                     p["seen"], p["cu"], p["q"], ref.SCALE(D), weights=weights, decay=decay, **opt)
    got = host(out).astype(np.float64)
    assert np.all(np.isfinite(got))
    tol = ref.tolerance(S[..., None], T) * E + 1e-30
    bad = np.argwhere(np.abs(got - want) > tol)
    assert bad.size == 0, f"{len(bad)} outputs off; first {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}, tol {tol[tuple(bad[0])]}"
    if w is not None:
        gw = host(w).astype(np.float64)
        tw = 2.0 * (70.0 * rel + (T / 2.0 + 64.0) * ww) * U + 4 * U * np.abs(ww) + 1e-30
        bad = np.argwhere(np.abs(gw - ww) > tw)
        assert bad.size == 0, f"{len(bad)} page weights off; first {bad[0]}: {gw[tuple(bad[0])]} for {ww[tuple(bad[0])]}"
    return want


def run_attention(p, weights=None, decay=1.0, **opt):
    D = p["q"].shape[2]
    sc = gq.AttnScores(ref.SCALE(D), cap=opt.get("cap", 0.0), window=opt.get("window", 0),
                       **{n: (dev(opt[n]) if opt.get(n) is not None else None) for n in ("slopes", "first", "prefix")})
    max_n = int(np.diff(p["cu"]).max())
    return gq.attn_pages(cache_of(p), dev(p["q"]), dev(p["cu"]), max_n, sc,
                         weights=None if weights is None else dev(weights), decay=decay)


# ---- append and read back ----------------------------------------------------------------------


def edge_values(gen, shape):
    """Rows that are zero, tie exactly at code borders, are tiny, subnormal or huge."""
    x = gen.standard_normal(shape).astype(np.float32)
    for t in range(shape[0]):
        kind = t % 7
        if kind == 0:
            x[t] = 0.0
        elif kind == 1:
            x[t] = gen.integers(-126, 127, size=shape[1:]) + np.float32(0.5)
            x[t, :, 0] = 127.0
        elif kind == 2:
            x[t] *= np.float32(1e-30)
        elif kind == 3:
            x[t] *= np.float32(1e-42)
        elif kind == 4:
            x[t] = np.float32(2.0) ** gen.integers(-12, 9, size=shape[1:]) * np.float32(1.0625)   # e4m3 borders
            x[t, :, 0] = 448.0
    return x


@pytest.mark.parametrize("kind", [gq.GQ_KV_I8, gq.GQ_KV_E4M3])
@pytest.mark.parametrize("D,P,held,new", [
    (64, 16, [0, 5, 16, 33], [1, 1, 1, 1]),
    (128, 32, [0, 31, 32, 7, 64], [1, 1, 1, 0, 2]),
    (128, 16, [3, 0], [47, 16]),
    (64, 128, [0, 127, 1], [300, 2, 127]),
    (128, 64, [10, 64, 0], [1, 129, 64]),
    (128, 128, [120], [9]),
])
def test_append_is_exact(kind, D, P, held, new):
    p = ref.problem(D + P, kind, len(held), 3, 1, D, P, held, new)
    T = int(p["cu"][-1])
    x = {n: edge_values(p["gen"], (T, 3, D)) for n in ("k", "v")}
    # the rows of a fused product's output: strided
    rows = torch.zeros((T, 3 * D * 2 + 8), device="cuda")
    rows[:, 4:4 + 3 * D] = dev(x["k"].reshape(T, -1))
    rows[:, 4 + 3 * D:4 + 6 * D] = dev(x["v"].reshape(T, -1))
    k, v = rows[:, 4:4 + 3 * D], rows[:, 4 + 3 * D:4 + 6 * D]
    c = cache_of(p)
    base0 = p["base"].copy()
    for _ in range(2):   # twice: the second changes nothing
        gq.kv_pages_append(c, k, v, dev(p["cu"]), max(new))
        for name in ("k", "v"):
            codes, scale = ref.append(kind, P, p[name], p[name + "s"], p["table"], p["held"], p["cu"], x[name])
            assert np.array_equal(host(getattr(c, name + "s")).view(np.uint32), scale.view(np.uint32)), name
            got = ref.decode(kind, host(getattr(c, name)))
            want = ref.decode(kind, codes)
            bad = np.argwhere(got != want)
            assert bad.size == 0, (name, bad[:3], got[tuple(bad[0])], want[tuple(bad[0])])
    begun = host(c.base)
    for b in range(len(held)):
        for j in range(p["table"].shape[2]):
            first = j * P
            if held[b] <= first < held[b] + new[b]:
                assert np.all(begun[b, :, j] == p["seen"][b] + first - held[b])
            else:
                assert np.array_equal(begun[b, :, j], base0[b, :, j])
    # and read back, from odd slots
    start = np.array([h // 2 for h in held], np.int32)
    n = [h + m - s for h, m, s in zip(held, new, start)]
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    rk, rv = gq.kv_pages_read(c, dev(start), dev(cu), int(cu[-1]), max(n))
    for name, r in (("k", rk), ("v", rv)):
        r, codes, scale = host(r), host(getattr(c, name)), host(getattr(c, name + "s"))
        for b in range(len(held)):
            for i in range(n[b]):
                s = start[b] + i
                pg = p["table"][b, :, s // P]
                want = (ref.decode(kind, codes[pg, s % P]) * scale[pg].astype(np.float64)[:, None]).astype(np.float32)
                assert np.array_equal(r[cu[b] + i], want)


def test_append_many_steps_matches_one_by_one():
    """Tokens appended one at a time, the page's scale growing: each step as defined."""
    kind, D, P = gq.GQ_KV_I8, 64, 16
    p = ref.problem(3, kind, 1, 2, 1, D, P, [0], [40])
    c, gen = cache_of(p), np.random.default_rng(8)
    codes, scale = p["k"].copy(), p["ks"].copy()
    cu = np.array([0, 1], np.int32)
    for t in range(40):
        x = (gen.standard_normal((1, 2, D)) * (1 + 0.3 * t)).astype(np.float32)
        c.held.fill_(t)
        c.seen.fill_(t)
        gq.kv_pages_append(c, dev(x), dev(x), dev(cu), 1)
        codes, scale = ref.append(kind, P, codes, scale, p["table"], np.array([t]), cu, x)
    assert np.array_equal(host(c.k), codes) and np.array_equal(host(c.ks), scale)
    assert np.array_equal(host(c.base)[0, 0, :3], [0, 16, 32])


def test_bad_lengths_and_pages_are_reported():
    p = ref.problem(4, 0, 3, 2, 1, 64, 16, [5, 20, 9], [1, 1, 1])
    before = p["k"].copy()
    p["held"][0] = -1                                       # a negative length
    p["held"][1] = p["table"].shape[2] * 16                 # no room for the new token
    p["table"][2, 1, 0] = 10 ** 6                           # no such page
    c, x = cache_of(p), np.ones((3, 2, 64), np.float32)
    gq.kv_pages_append(c, dev(x), dev(x), dev(p["cu"]), 1)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    assert gq.gq_last_error() == gq.GQ_OK
    changed = np.argwhere((host(c.k) != before).any((1, 2)))[:, 0]
    assert set(changed) <= {p["table"][2, 0, 0]}
    out, w = run_attention(p, weights=np.ones(p["table"].shape, np.float32))
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    out, w = host(out), host(w)
    assert np.all(out[:2] == 0.0) and np.all(out[2, 1] == 0.0) and np.all(np.isfinite(out))
    assert np.any(out[2, 0] != 0.0) and np.all(w[:2] == 0.0)


# ---- attention -----------------------------------------------------------------------------------

#  kind, Hkv, G, D, P, held, new, gaps
SHAPES = [
    (0, 2, 1, 128, 32, [0], [1], False),                         # one token sees itself
    (0, 3, 4, 128, 16, [1, 15, 16, 17], [1, 1, 1, 1], False),
    (1, 2, 8, 64, 16, [31, 32, 33, 100], [1, 1, 1, 1], True),
    (0, 1, 7, 128, 64, [1000], [1], True),                       # one long sequence over many CTAs
    (1, 1, 3, 128, 128, [127, 128, 300], [1, 0, 2], False),
    (0, 2, 16, 64, 32, [70, 0], [3, 5], False),                  # more rows than one tile
    (1, 2, 2, 128, 64, [40, 0, 129], [33, 64, 7], True),         # prompt chunks
    (0, 1, 64, 64, 128, [90], [2], False),
    (0, 5, 1, 64, 16, [3] * 200, [1] * 200, False),              # many short sequences
    (0, 1, 4, 128, 32, [150], [100], False),                     # tiles of 128 rows: two pairs
    (1, 2, 1, 64, 16, [0, 700, 3], [290, 33, 1], True),          # and rows, in one batch
    (0, 1, 3, 64, 128, [260, 5], [86, 200], True),
    (0, 2, 2, 64, 16, [5] * 330, [20] * 330, False),             # a first tile each, and no second one
    (0, 2, 3, 64, 16, [5] * 330, [20] * 330, False),
    (0, 1, 4, 128, 32, [2500, 0], [40, 100], False),             # few tiles, many keys: shares of one sequence's keys
    (1, 1, 8, 64, 16, [5000], [17], True),
]


@pytest.mark.parametrize("kind,Hkv,G,D,P,held,new,gaps", SHAPES)
@pytest.mark.parametrize("opts", ["plain", "cap", "bias", "window", "prefix", "all"])
def test_attention(kind, Hkv, G, D, P, held, new, gaps, opts):
    p = ref.problem(len(held) + D + P + G, kind, len(held), Hkv, G, D, P, held, new, gaps)
    T, opt = int(p["cu"][-1]), {}
    qpos = np.concatenate([p["seen"][b] + np.arange(new[b]) for b in range(len(held))])
    if opts in ("cap", "all"):
        opt["cap"] = 5.0 if opts == "cap" else 30.0
    if opts in ("bias", "all"):
        opt["slopes"] = ref.alibi(Hkv * G)
    if opts in ("window", "all"):
        opt["window"] = 1 if opts == "window" and P == 16 else 37
    if opts in ("prefix", "all"):
        opt["prefix"] = np.where(np.arange(T) % 3 == 2, 0, 21 + np.arange(T) % 50).astype(np.int32)
    if opts == "all":
        opt["first"] = (qpos // 50 * 50).astype(np.int32)
    weights = p["gen"].random(p["table"].shape).astype(np.float32)
    out, w = run_attention(p, weights=weights, decay=0.75, **opt)
    check_attention(p, out, w, weights=weights, decay=0.75, **opt)
    again = run_attention(p, **opt)
    assert torch.equal(again, out)           # with or without weights, and every time, the same bits


def test_rows_that_see_nothing_are_zero():
    p = ref.problem(5, 1, 2, 2, 4, 128, 16, [40, 0], [3, 2])
    first = np.array([10 ** 6, 0, 10 ** 6, 10 ** 6, 0], np.int32)     # a document that has not begun
    out, w = run_attention(p, weights=np.zeros(p["table"].shape, np.float32), first=first)
    check_attention(p, out, w, weights=np.zeros(p["table"].shape, np.float32), first=first)
    assert np.all(host(out)[first > 0] == 0.0)


def test_unused_slots_may_hold_anything():
    """NaN codes past the last token, unused pages and unused table entries change nothing."""
    p = ref.problem(6, 1, 2, 2, 2, 128, 32, [37, 64], [1, 1])
    want = host(run_attention(p))
    for b, n in enumerate((38, 65)):
        for h in range(2):
            for j in range(p["table"].shape[2]):
                pg = p["table"][b, h, j]
                live = min(max(0, n - 32 * j), 32)
                p["k"][pg, live:] = p["v"][pg, live:] = 0x7F
                if live == 0:
                    p["ks"][pg] = p["vs"][pg] = np.nan
                    p["table"][b, h, j] = -5
    assert np.array_equal(host(run_attention(p)), want)


def test_scales_of_every_size():
    """Page scales from 1e-30 to 1e30, zeros among them: the values keep their weight."""
    p = ref.problem(7, 0, 1, 2, 2, 64, 16, [200], [1])
    p["vs"] *= np.float32(10.0) ** np.linspace(-30, 30, len(p["vs"])).astype(np.float32)
    p["vs"][p["table"][0, 0, 3]] = 0.0
    p["ks"][p["table"][0, 1, 4]] = 0.0
    check_attention(p, run_attention(p))


@pytest.mark.parametrize("new", [1, 20])
def test_many_weights_far_below_the_largest(new):
    """2,000 keys of weight e^-18 beside the step's own: each is carried to 2^-33 of the largest."""
    N, G, D, P = 2000, 8, 64, 16
    p = ref.problem(10, 0, 1, 1, G, D, P, [N], [new])
    p["q"][:] = 18.0 / (D * ref.SCALE(D))
    p["ks"][:] = p["vs"][:] = np.float32(1 / 127)
    for i in range(N + new):
        page, slot = p["table"][0, 0, i // P], i % P
        p["k"][page, slot], p["v"][page, slot] = (0, 100) if i < N else (127, 0)
    want, *_ = ref.attend(0, P, p["k"], p["ks"], p["v"], p["vs"], p["table"], p["base"], p["held"], p["seen"], p["cu"], p["q"],
                          ref.SCALE(D))
    got = host(run_attention(p)).astype(np.float64)
    # scales of 1/127 < 2^-6 times codes of 100; and z = 18 carries 2^-22 and a few roundings: 1e-4 of a weight
    bound = N * 2.0 ** (-6 - 33) * 100
    assert np.all(want > 3 * bound)
    assert np.all(np.abs(got - want) <= bound + 1e-4 * want)


def test_strided_rows_and_streams():
    p = ref.problem(8, 0, 2, 2, 4, 128, 64, [500, 77], [1, 1])
    want = host(run_attention(p))
    c, cu, Hq, D = cache_of(p), dev(p["cu"]), 8, 128
    rows = torch.zeros((2, 3 * Hq * D), device="cuda")
    rows[:, Hq * D:2 * Hq * D] = dev(p["q"].reshape(2, -1))
    out = torch.full((2, 2 * Hq * D), 3.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sc = gq.AttnScores(ref.SCALE(D))
    with torch.cuda.stream(s):
        gq.attn_pages(c, rows[:, Hq * D:2 * Hq * D], cu, 1, sc, out=out[:, Hq * D:])
    s.synchronize()
    assert np.array_equal(host(out[:, Hq * D:]).reshape(2, Hq, D), want)
    assert torch.all(out[:, :Hq * D] == 3.0)


def test_a_step_in_a_graph():
    """Append, attention with weights and eviction captured once and replayed: the eager results."""
    kind, D, P, B, Hkv, G = 0, 64, 16, 2, 2, 2
    gen = np.random.default_rng(9)
    steps = [gen.standard_normal((B, (G + 2) * Hkv * D)).astype(np.float32) for _ in range(60)]

    def build():
        c = gq.KVPages.empty(B, Hkv, D, 64, P, kind)
        return c, torch.zeros((B, Hkv, c.NB), device="cuda"), torch.empty((B, (G + 2) * Hkv * D), device="cuda")

    cu = dev(np.arange(B + 1, dtype=np.int32))
    sc = gq.AttnScores(ref.SCALE(D))

    def step(c, w, x, out):
        q, k, v = x[:, :G * Hkv * D], x[:, G * Hkv * D:(G + 1) * Hkv * D], x[:, (G + 1) * Hkv * D:]
        gq.kv_pages_append(c, k, v, cu, 1)
        gq.gq_attn_pages(c, sc, q, x.stride(0), cu, B, 1, G * Hkv, out, G * Hkv * D, w, w, 0.9)
        c.held += 1
        c.seen += 1
        gq.gq_kv_pages_evict(c, w, 3, 1, 1, c.table, c.base, w, c.held)     # in place

    eager, (c, w, x) = [], build()
    out = torch.empty((B, G * Hkv, D), device="cuda")
    for s in steps:
        x.copy_(dev(s))
        step(c, w, x, out)
        eager.append(host(out))
    assert np.all(host(c.held) <= 48) and np.all(host(c.seen) == 60)
    c, w, x = build()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(c, w, x.zero_(), out)          # sizes the stream's workspace
        st.synchronize()
        for t in (c.k, c.v, c.ks, c.vs, c.base, c.held, c.seen, w):
            t.zero_()
        c.table.copy_(torch.arange(c.table.numel(), dtype=torch.int32, device="cuda").reshape(c.table.shape))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step(c, w, x, out)
        for s, want in zip(steps, eager):
            x.copy_(dev(s))
            graph.replay()
            st.synchronize()
            assert np.array_equal(host(out), want)


@pytest.mark.parametrize("kind,Hkv,G,D,P,held,new", [
    (0, 1, 8, 128, 32, [3000], [30]),                        # shares of one tile's keys, joined
    (1, 2, 2, 64, 16, [60] * 100, [25] * 100),               # many items of one block, second tiles empty
    (0, 2, 4, 128, 64, [500, 0, 9], [70, 200, 1]),           # tiles and rows in one batch
])
def test_prompts_in_a_graph_and_in_a_row(kind, Hkv, G, D, P, held, new):
    """Every launch of a long row of them, eager and replayed, gives the first one's bits."""
    p = ref.problem(12, kind, len(held), Hkv, G, D, P, held, new)
    c, q, cu, sc = cache_of(p), dev(p["q"]), dev(p["cu"]), gq.AttnScores(ref.SCALE(D))
    w = dev(p["gen"].random(p["table"].shape).astype(np.float32))
    out, new_w = torch.empty_like(q), torch.empty_like(w)

    def call():
        gq.gq_attn_pages(c, sc, q, Hkv * G * D, cu, q.shape[0], max(new), Hkv * G, out, Hkv * G * D, w, new_w, 0.5)

    call()
    want = out.clone(), new_w.clone()
    check_attention(p, out, new_w, weights=host(w), decay=0.5)
    for _ in range(200):
        call()
    assert torch.equal(out, want[0]) and torch.equal(new_w, want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            call()
            call()
        out.zero_()
        for _ in range(50):
            graph.replay()
        st.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(new_w, want[1])
    assert gq.gq_last_error() == gq.GQ_OK


# ---- eviction ------------------------------------------------------------------------------------


@pytest.mark.parametrize("held,budget,first,last", [
    ([16 * 9, 16 * 9 - 15, 16 * 4, 0], 4, 1, 1),
    ([16 * 1000 - 3, 16 * 700, 16 * 3], 512, 4, 2),
    ([16 * 33], 3, 1, 2),                                    # no room for any of the others
    ([16 * 5, 16 * 2500], 2400, 0, 1),
    ([16 * 8], 10 ** 9, 2, 2),                               # nothing to drop
])
@pytest.mark.parametrize("grid", [0, 8])
def test_evict(held, budget, first, last, grid):
    p = ref.problem(len(held) + budget % 97, 0, len(held), 3, 1, 64, 16, held, [0] * len(held), gaps=True)
    w = p["gen"].standard_normal(p["table"].shape).astype(np.float32)     # any finite weights, negative ones too
    if grid:
        w = np.round(w * grid) / np.float32(grid)                         # ties
    c = cache_of(p)
    got = gq.kv_pages_evict(c, dev(w), budget, first, last)
    want = ref.evict(16, p["table"], p["base"], w, p["held"], budget, first, last)
    for g, x in zip(got, want):
        assert np.array_equal(host(g), x)
    wd = dev(w)
    gq.gq_kv_pages_evict(c, wd, budget, first, last, c.table, c.base, wd, c.held)    # in place
    for g, x in zip((c.table, c.base, wd, c.held), want):
        assert np.array_equal(host(g), x)


def test_append_attend_evict_long_run():
    """Hundreds of steps within a fixed budget of pages: every page always owned once, distances kept."""
    kind, D, P, B, Hkv = 1, 64, 16, 1, 2
    c = gq.KVPages.empty(B, Hkv, D, 6 * P, P, kind)
    w = torch.zeros((B, Hkv, c.NB), device="cuda")
    cu, sc, gen = dev(np.array([0, 1], np.int32)), gq.AttnScores(ref.SCALE(D), slopes=dev(ref.alibi(2))), torch.Generator("cuda").manual_seed(2)
    for _ in range(200):
        x = torch.randn((1, 4 * D), generator=gen, device="cuda")
        gq.kv_pages_append(c, x[:, :2 * D], x[:, 2 * D:], cu, 1)
        _, w = gq.attn_pages(c, x[:, :2 * D], cu, 1, sc, weights=w, decay=0.95)
        c.held += 1
        c.seen += 1
        gq.gq_kv_pages_evict(c, w, 5, 1, 1, c.table, c.base, w, c.held)
    assert int(c.seen) == 200 and 4 * P < int(c.held) <= 5 * P
    t, b = host(c.table), host(c.base)
    for h in range(Hkv):
        assert set(t[0, h]) == set(range(h * c.NB, (h + 1) * c.NB))
        n = -(-int(c.held) // P)
        assert b[0, h, 0] == 0 and np.all(np.diff(b[0, h, :n]) >= P) and b[0, h, n - 1] + int(c.held) - (n - 1) * P == 200
