"""The paged 8-bit KV cache where a call is unusual: lengths and tables that are out of range, limits of
positions, masked pages unlike the visible ones, steps of many rows (GPU only).  Bounds as in test_gpu_pages.py."""
import numpy as np
import pytest
import torch

import pages_accuracy as acc
import pages_ref as ref
import quantized_skinny_matmul_gb300 as gq
from test_gpu_pages import built, cache_of, check_attention, run_attention  # noqa: F401 (built: a fixture)
from test_gpu_parity import dev, host

pytestmark = pytest.mark.gpu


def repeated(p, times):
    """The problem of one sequence as the 1st, 3rd, .. of a batch whose cu goes to n and back to 0."""
    n, B = int(p["cu"][1]), 2 * times - 1
    q = dict(p, cu=np.array([0, n] * times, np.int32))
    for name in ("table", "base", "held", "seen"):
        q[name] = np.repeat(p[name], B, axis=0)
    return q


# ---- lengths, tables and cu that are out of range -------------------------------------------------


@pytest.mark.parametrize("Hkv,G,new,times", [(1, 8, 512, 40), (2, 8, 1100, 8)])
def test_a_cu_that_goes_back_stays_within_the_plan(Hkv, G, new, times):
    """Far more pairs of tiles than rows: what is written stays in bounds, and the fault is reported."""
    p = ref.problem(20, 0, 1, Hkv, G, 64, 64, [70], [new])
    out = run_attention(repeated(p, times))
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    check_attention(p, out)                  # all the sequences that name the rows are the same one
    check_attention(p, run_attention(p))     # and the next call finds everything as it should be
    assert gq.gq_last_error() == gq.GQ_OK


@pytest.mark.parametrize("new", [1, 3, 60])
def test_positions_below_the_slots_are_reported(new):
    """A next position below the tokens held: skipped, and no slot is sought below the first."""
    p = ref.problem(21, 0, 2, 1, 2, 64, 16, [100, 40], [new, new])
    p["seen"][0] = 30
    before = p["k"].copy()
    c, x = cache_of(p), np.ones((2 * new, 1, 64), np.float32)
    gq.kv_pages_append(c, dev(x), dev(x), dev(p["cu"]), new)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    changed = np.argwhere((host(c.k) != before).any((1, 2)))[:, 0]
    assert set(changed) <= set(p["table"][1, 0])
    first = np.where(np.arange(2 * new) < new, 2 ** 31 - 1, 0).astype(np.int32)     # of documents far ahead
    out, w = run_attention(p, weights=np.ones(p["table"].shape, np.float32), first=first)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    p["held"][0] = p["seen"][0] = 0          # the reference: a sequence that sees only itself, whose rows are then left out
    want, ww, E, S, rel = ref.attend(0, 16, p["k"], p["ks"], p["v"], p["vs"], p["table"], p["base"], p["held"], p["seen"],
                                     p["cu"], p["q"], ref.SCALE(64), weights=np.ones(p["table"].shape), first=first)
    assert np.all(host(out)[:new] == 0.0) and np.all(host(w)[0] == 0.0)
    assert np.all(np.abs(host(out) - want)[new:] <= (ref.tolerance(S[..., None], 40 + new) * E)[new:])
    assert np.all(np.abs(host(w) - ww)[1] <= (ref.tolerance(0, 40 + new) * ww + ref.tolerance(1, 0) * rel)[1])


def test_an_eviction_s_tensors_assigned_to_the_cache():
    """The next call works on the new tensors, whatever becomes of the old ones' memory."""
    p = ref.problem(22, 0, 2, 2, 2, 64, 16, [16 * 9, 16 * 7], [0, 0])
    w = p["gen"].random(p["table"].shape).astype(np.float32)
    c = cache_of(p)
    c.table, c.base, _, c.held = gq.kv_pages_evict(c, dev(w), 4)
    junk = [torch.full((4096,), 2 ** 30, dtype=torch.int32, device="cuda") for _ in range(64)]     # over the freed ones
    p["table"], p["base"], _, p["held"] = ref.evict(16, p["table"], p["base"], w, p["held"], 4, 1, 1)
    p.update(cu=np.array([0, 1, 2], np.int32), q=p["gen"].standard_normal((2, 4, 64)).astype(np.float32))
    x = p["gen"].standard_normal((2, 2, 64)).astype(np.float32)
    gq.kv_pages_append(c, dev(x), dev(x), dev(p["cu"]), 1)
    p.update({n: host(getattr(c, n)) for n in ("k", "v", "ks", "vs", "base")})
    for b in range(2):                       # the token's page begins where its table row says
        assert np.all(p["base"][b, :, p["held"][b] // 16] == p["seen"][b])
    check_attention(p, gq.attn_pages(c, dev(p["q"]), dev(p["cu"]), 1, gq.AttnScores(ref.SCALE(64))))
    assert len(junk) == 64 and gq.gq_last_error() == gq.GQ_OK


# ---- limits of positions ---------------------------------------------------------------------------


@pytest.mark.parametrize("new", [1, 50])             # rows, tiles
@pytest.mark.parametrize("P,held", [(64, 70), (128, 130), (128, 500), (32, 70)])
def test_a_prefix_without_end(P, held, new):
    """INT32_MAX, all is seen: a last page whose groups of 32 tokens are partly unused gathers its own share only."""
    p = ref.problem(23, 0, 2, 2, 1, 64, P, [held, 3], [new, 1])
    prefix = np.full(new + 1, 2 ** 31 - 1, np.int32)
    weights = p["gen"].random(p["table"].shape).astype(np.float32)
    out, w = run_attention(p, weights=weights, decay=0.5, prefix=prefix)
    check_attention(p, out, w, weights=weights, decay=0.5, prefix=prefix)


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("least", [-2 ** 31, -2 ** 31 + 5, -1])
def test_documents_and_prefixes_that_begin_far_below_zero(least, new):
    """The least int32 as a start or as a prefix's end is as good as none."""
    p = ref.problem(24, 1, 1, 2, 1, 64, 16, [200], [new])
    for name in ("first", "prefix"):
        opt = {name: np.full(new, least, np.int32)}
        weights = p["gen"].random(p["table"].shape).astype(np.float32)
        out, w = run_attention(p, weights=weights, window=150, **opt)
        check_attention(p, out, w, weights=weights, window=150, **opt)


@pytest.mark.parametrize("new", [2, 50])
def test_pages_that_are_none_gather_nothing(new):
    """A block of tokens without a usable page: its weight is what decay leaves of the old one."""
    p = ref.problem(25, 0, 2, 2, 1, 64, 128, [300, 300], [new, new])
    weights = p["gen"].random(p["table"].shape).astype(np.float32)
    run_attention(p, weights=weights)        # (leaves sums of its own where the next call's are kept)
    q = dict(p, table=p["table"].copy(), base=p["base"].copy())
    p["table"][0, 0, 1], p["table"][1, 1, 0] = 10 ** 6, -1
    q["base"][0, 0, 1] = q["base"][1, 1, 0] = 1 << 29        # the reference: positions that nobody sees
    out, w = run_attention(p, weights=weights, decay=0.5)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    check_attention(q, out, w, weights=weights, decay=0.5)


@pytest.mark.parametrize("G,T,max_n,cu", [
    (1, 200, 100, [0, 30, 130]),             # the host's numbers say that both have 100
    (2, 100, 100, [0, 3]),
    (1, 100, 100, [0, 0]),
    (1, 300, 100, [0, 100, 100, 140]),
])
def test_fewer_rows_than_the_call_is_made_for(G, T, max_n, cu):
    """A padded step, as a captured one is: every sequence's rows are worked out, those past cu[B] are left alone."""
    new = np.diff(cu)
    p = ref.problem(26, 0, len(new), 2, G, 64, 32, [150] * len(new), new)
    n, weights = cu[-1], p["gen"].random(p["table"].shape).astype(np.float32)
    q = torch.randn((T, 2 * G, 64), device="cuda")
    q[:n] = dev(p["q"])
    out, w, nan = torch.full((T, 2 * G, 64), 7.0, device="cuda"), dev(weights), np.full(p["table"].shape, np.nan, np.float32)
    run_attention(p if n else ref.problem(26, 0, 1, 2, G, 64, 32, [0], [1]))
    for new_w in (dev(nan), dev(nan)):       # (sums of the first call are there in the second)
        gq.gq_attn_pages(cache_of(p), gq.AttnScores(ref.SCALE(64)), q, 2 * G * 64, dev(p["cu"]), T, max_n, 2 * G, out,
                         2 * G * 64, w, new_w, 0.5)
        check_attention(p, out[:n], new_w, weights=weights, decay=0.5)
        assert torch.all(out[n:] == 7.0)
    assert gq.gq_last_error() == gq.GQ_OK


@pytest.mark.parametrize("G,T,max_n,cu", [
    (1, 200, 100, [0, 30, 200]),             # tiles alone, by the host's numbers
    (1, 250, 100, [0, 30, 200, 250]),        # tiles and rows
    (2, 5, 2, [0, 1, 4, 5]),                 # rows
    (1, 170, 100, [0, 170]),
])
def test_more_new_tokens_than_said_give_zero_rows(G, T, max_n, cu):
    new = np.diff(cu)
    p = ref.problem(27, 1, len(new), 2, G, 64, 32, [150] * len(new), new)
    weights = p["gen"].random(p["table"].shape).astype(np.float32)
    want, ww, E, S, rel = ref.attend(1, 32, p["k"], p["ks"], p["v"], p["vs"], p["table"], p["base"], p["held"], p["seen"],
                                     p["cu"], p["q"], ref.SCALE(64), weights=weights)
    out = torch.full((T, 2 * G, 64), 7.0, device="cuda")
    _, w = gq.attn_pages(cache_of(p), dev(p["q"]), dev(p["cu"]), max_n, gq.AttnScores(ref.SCALE(64)), weights=dev(weights),
                         out=out)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    out, w, N = host(out), host(w), 150 + max_n
    for b, n in enumerate(new):
        rows = slice(cu[b], cu[b + 1])
        if n > max_n:
            assert np.all(out[rows] == 0.0) and np.all(w[b] == 0.0)
        else:
            assert np.all(np.abs(out - want)[rows] <= (ref.tolerance(S[..., None], N) * E)[rows])
            assert np.all(np.abs(w - ww)[b] <= (ref.tolerance(0, N) * ww + ref.tolerance(1, 0) * rel)[b])


@pytest.mark.parametrize("kind", [gq.GQ_KV_I8, gq.GQ_KV_E4M3])
@pytest.mark.parametrize("D", [64, 128])
def test_what_cannot_be_read_back_is_zero(kind, D):
    """Sequences whose slots are out of range, and pages that are none."""
    p = ref.problem(28, kind, 5, 2, 1, D, 16, [60] * 5, [0] * 5)
    NB = p["table"].shape[2]
    p["table"][3, 1, 1] = 10 ** 6
    start, n = np.array([-1, 5, NB * 16 - 3, 10, 0], np.int32), [20, 40, 4, 30, 90]
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    T, max_n = int(cu[-1]), 60               # the last one has more than max_n
    got = [torch.full((T, 2, D), 7.0, device="cuda") for _ in range(2)]
    gq.gq_kv_pages_read(cache_of(p), dev(start), dev(cu), T, max_n, *got)
    assert gq.gq_last_error() == gq.GQ_ERR_INVALID_ARG
    for name, r in zip(("k", "v"), got):
        r = host(r)
        for b in (0, 2, 4):
            assert np.all(r[cu[b]:cu[b + 1]] == 0.0), b
        for b in (1, 3):
            for i in range(n[b]):
                s = start[b] + i
                for h in range(2):
                    pg = p["table"][b, h, s // 16]
                    want = 0.0 if pg == 10 ** 6 else ref.decode(kind, p[name][pg, s % 16]) * np.float64(p[name + "s"][pg])
                    assert np.array_equal(r[cu[b] + i, h], np.broadcast_to(np.float32(want), D)), (b, i, h)




# ---- masked pages unlike the visible ones ----------------------------------------------------------


@pytest.mark.parametrize("kind", [gq.GQ_KV_I8, gq.GQ_KV_E4M3])
@pytest.mark.parametrize("Hkv,G,D,P,new,more", [
    (2, 1, 128, 16, 2, 0), (2, 1, 64, 32, 4, 160), (1, 4, 128, 16, 2, 0), (1, 3, 64, 64, 5, 160),        # rows: alone, and
    (2, 5, 128, 128, 8, 160), (1, 4, 128, 16, 2, 160),                                                   # many units a warp
    (2, 1, 128, 16, 60, 0), (1, 4, 64, 32, 40, 0), (1, 8, 128, 128, 70, 0), (1, 2, 64, 16, 300, 0),        # tiles
])
@pytest.mark.parametrize("opts", ["first", "window", "prefix"])
def test_values_of_masked_pages_do_not_matter(kind, Hkv, G, D, P, new, more, opts):
    """Pages whose values are 2^60 times the others': rows that do not see them keep their own values whole."""
    # (`more` sequences fill the GPU, so that a CTA has whole items and a warp several units)
    p = ref.problem(29, kind, 1 + more, Hkv, G, D, P, [300] + [640] * more, [new] + [1] * more)
    T, qpos = new + more, p["seen"][0] + np.arange(new + more)
    border = 300 // P * P // 2 // P * P      # the loud pages begin with the sequence and end here
    for h in range(Hkv):
        p["vs"][p["table"][0, h, :border // P]] *= np.float32(2.0 ** 60)
    if opts == "first":                      # every other row sees them
        opt = dict(first=np.where(np.arange(T) % 2 == 1, 0, border).astype(np.int32))
    elif opts == "window":                   # the first rows see one token of them, or a few
        opt = dict(window=int(qpos[0] - border + 1 + min(3, new // 2)))
    else:                                    # none but the odd rows' prefix
        opt = dict(window=int(qpos[0] - border), prefix=np.where(np.arange(T) % 2 == 1, border // 2, 0).astype(np.int32))
    weights = np.ones(p["table"].shape, np.float32)
    out, w = run_attention(p, weights=weights, **opt)
    opt = {n: v[:new] if n != "window" else v for n, v in opt.items()}
    one = dict(p, held=p["held"][:1], seen=p["seen"][:1], cu=p["cu"][:2], q=p["q"][:new], table=p["table"][:1], base=p["base"][:1])
    names = ("kind", "P", "k", "ks", "v", "vs", "table", "base", "held", "seen", "cu", "q")
    want, ww, E, S, rel = ref.attend(*(one[n] for n in names), ref.SCALE(D), weights=weights[:1], **opt)
    # the rows that see none of the loud pages (those that do are bound by them, by a share of 2^-33 at least)
    start = np.maximum(opt.get("first", np.zeros(new, np.int64)), qpos[:new] - opt.get("window", 10 ** 6) + 1)
    quiet = (start >= border) & (opt.get("prefix", np.zeros(new)) == 0)
    assert quiet.sum() >= new // 2
    N = 300 + new
    assert np.all(np.abs(host(out)[:new] - want)[quiet] <= (ref.tolerance(S[..., None], N) * E)[quiet])
    assert np.all(np.abs(host(w)[0] - ww[0]) <= ref.tolerance(0, N) * ww[0] + ref.tolerance(1, 0) * rel[0])
    assert np.all(np.isfinite(host(out)))


# ---- accuracy ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", [gq.GQ_KV_I8, gq.GQ_KV_E4M3])
@pytest.mark.parametrize("G,D,P,new", [(1, 128, 16, 1), (4, 128, 32, 1), (2, 64, 16, 1), (8, 128, 64, 1), (8, 64, 16, 1),   # rows
                                       (2, 128, 32, 48), (1, 64, 64, 60)])                                                  # tiles
def test_queries_and_weights_keep_both_terms(kind, G, D, P, new):
    p = acc.few_keys(40, kind, G, D, P, new)
    want, _, E, S, _ = acc.reference(p)
    assert np.all(np.abs(host(run_attention(p)) - want) <= acc.few_keys_bound(D, S, E))


def one_sign(kind, D, B, Hkv, G, L, new, gen):
    """A cache whose values are all positive, and queries of zero: every key weighs the same, and a sum that is
    not rounded to nearest shows in full.  The outputs of a few rows, and what they should be."""
    P = 64
    NB = -(-(L + new) // P)
    pages = B * Hkv * NB
    k = torch.zeros((pages, P, D), dtype=torch.int8 if kind == 0 else torch.uint8, device="cuda")
    lo, hi = (60, 128) if kind == 0 else (0x40, 0x7F)
    v = torch.randint(lo, hi, (pages, P, D), generator=gen, device="cuda", dtype=k.dtype)
    vs = torch.rand(pages, generator=gen, device="cuda") / 2 + 0.5
    table = torch.arange(pages, device="cuda", dtype=torch.int32).reshape(B, Hkv, NB)
    base = (torch.arange(NB, device="cuda", dtype=torch.int32) * P).expand(B, Hkv, NB).contiguous()
    held = torch.full((B,), L, dtype=torch.int32, device="cuda")
    c = gq.KVPages(kind, k, v, torch.ones_like(vs), vs, table, base, held, held.clone())
    cu = (torch.arange(B + 1, device="cuda") * new).to(torch.int32)
    out = gq.attn_pages(c, torch.zeros((B * new, Hkv * G, D), device="cuda"), cu, new, gq.AttnScores(1.0))
    got, want = [], []
    for b, i in ((0, 0), (B - 1, new - 1)):
        pg = table[b, 0].long()
        x = (v[pg] if kind == 0 else v[pg].view(torch.float8_e4m3fn).float()).double() * vs[pg].double()[:, None, None]
        got.append(out[b * new + i, 0].double())
        want.append(x.reshape(-1, D)[:L + i + 1].mean(0))
    assert gq.gq_last_error() == gq.GQ_OK
    return torch.stack(got), torch.stack(want)


@pytest.mark.parametrize("kind", [gq.GQ_KV_I8, gq.GQ_KV_E4M3])
@pytest.mark.parametrize("D,B,Hkv,G,L,new,steps,adds", [
    # rows, a sequence in a CTA: 146 units a warp, flushed every 8 of them (2 steps each); 18 flushes and 7 warps to add
    (64, 304, 1, 1, 32767, 1, 16, 25), (128, 304, 1, 8, 32767, 1, 16, 25),
    # rows, not flushed: 16 units a warp at most
    (128, 304, 1, 1, 3500, 1, 32, 7),
    # tiles: 256 blocks of 8 steps for each of the two terms, flushed every 4
    (64, 2, 16, 8, 32767, 96, 64, 64), (128, 2, 16, 8, 32767, 96, 64, 64),
])
def test_long_sums_are_rounded(kind, D, B, Hkv, G, L, new, steps, adds):
    """A step is off by at most 2^-23 of the sum so far, an addition by 2^-24; 16 more for the terms and the end."""
    got, want = one_sign(kind, D, B, Hkv, G, L, new, torch.Generator("cuda").manual_seed(3))
    assert float(((got - want).abs() / want).max()) <= (2 * steps + adds + 16) * 2.0 ** -24


# ---- steps whose sums do not fit at once -------------------------------------------------------------


def roomy(p, NB):
    """The same cache with room for NB pages a sequence and head (the entries of the others are never looked at)."""
    B, Hkv, old = p["table"].shape
    q = dict(p)
    for name in ("table", "base"):
        q[name] = np.zeros((B, Hkv, NB), np.int32)
        q[name][..., :old] = p[name]
    return q


@pytest.mark.parametrize("kind,Hkv,G,P,held,new,NB,opts", [
    (0, 1, 16, 16, [40, 0], [400, 200], 20000, ""),                     # 419 rows at a time: within the first sequence
    (1, 2, 4, 16, [100, 5, 30], [70, 1, 60], 1 << 17, "prefix"),        # 128 rows; keys past the slice's own are seen
    (0, 1, 8, 32, [300], [150], 1 << 19, "window"),                     # 32 rows
    (0, 1, 32, 128, [30] * 10, [1] * 10, 1 << 18, "first"),             # 4 rows, of as many sequences
    (1, 1, 64, 16, [200], [3], 1 << 22, ""),                            # one row's are more than a slice is to have
])
def test_weights_in_slices(kind, Hkv, G, P, held, new, NB, opts):
    p = roomy(ref.problem(31, kind, len(held), Hkv, G, 64, P, held, new), NB)
    T, opt = int(p["cu"][-1]), {}
    if opts == "prefix":
        opt["prefix"] = np.where(np.arange(T) % 2 == 0, 160, 0).astype(np.int32)
    elif opts == "window":
        opt["window"] = 45
    elif opts == "first":
        opt["first"] = np.where(np.arange(T) % 3 == 0, 25, 0).astype(np.int32)
    weights = np.zeros(p["table"].shape, np.float32)
    weights[..., :40] = p["gen"].random((len(held), Hkv, 40))
    before = torch.cuda.mem_get_info()[0]
    out, w = run_attention(p, weights=weights, decay=0.75, **opt)
    used = before - torch.cuda.mem_get_info()[0]
    check_attention(p, out, w, weights=weights, decay=0.75, **opt)
    assert gq.gq_last_error() == gq.GQ_OK
    assert used < 3 << 30                    # (a workspace at least doubles when it grows)
    again = run_attention(p, weights=weights, decay=0.75, **opt)
    assert torch.equal(again[0], out) and torch.equal(again[1], w)


@pytest.mark.parametrize("kind,G,D,P,new", [(0, 1, 128, 32, 1), (1, 4, 128, 16, 1), (0, 8, 64, 32, 1), (1, 2, 64, 64, 4),
                                            (0, 8, 128, 128, 1), (1, 1, 64, 16, 2), (0, 5, 128, 64, 3),
                                            (0, 1, 128, 32, 48), (1, 4, 64, 16, 12)])       # the last two: tiles
@pytest.mark.parametrize("opts", ["plain", "grow", "shrink", "masks"])
def test_flushed_sums_under_changing_maxima_and_scales(kind, G, D, P, new, opts):
    """Long sequences, sums flushed many times: maxima and value scales that grow or fall on the way."""
    B, Hkv, pool = 160, 2, 192
    L = 8000 // P * P - 3
    p = ref.problem(41, kind, 1, 1, G, D, P, [pool * P], [1], extra=0)       # a pool of pages, shared by the sequences
    gen, NB = p["gen"], -(-(L + new) // P)
    table = gen.integers(0, pool, (B, Hkv, NB)).astype(np.int32)
    if opts in ("grow", "shrink"):           # a page's scales by its number, the numbers in order
        order = np.sort(table, -1) if opts == "grow" else -np.sort(-table, -1)
        table = np.ascontiguousarray(order)
        p["vs"][:] = p["vs"] * np.float32(2.0) ** (np.arange(len(p["vs"])) // 4 - 24)
        p["ks"][:] = p["ks"] * np.linspace(0.2, 3.0, len(p["ks"])).astype(np.float32)
    held = np.full(B, L, np.int32)
    base = np.ascontiguousarray(np.broadcast_to(np.arange(NB, dtype=np.int32) * P, (B, Hkv, NB)))
    cu = (np.arange(B + 1) * new).astype(np.int32)
    p.update(table=table, base=base, held=held, seen=held.copy(), cu=cu, q=gen.standard_normal((B * new, Hkv * G, D)).astype(np.float32))
    opt = {}
    if opts == "masks":
        t = np.arange(B * new)
        opt = dict(cap=20.0, window=6000, prefix=np.where(t % 2 == 0, 700, 0).astype(np.int32),
                   first=np.where(t % 3 == 0, 150, 0).astype(np.int32), slopes=ref.alibi(Hkv * G) / 64)
    weights = gen.random(table.shape).astype(np.float32)
    out, w = run_attention(p, weights=weights, decay=0.5, **opt)
    assert gq.gq_last_error() == gq.GQ_OK and bool(torch.isfinite(out).all())
    for b in (0, 77, B - 1):
        rows = slice(cu[b], cu[b + 1])
        one = dict(p, held=held[:1], seen=held[:1], cu=cu[:2], q=p["q"][rows], table=table[b:b + 1], base=base[b:b + 1])
        opt_b = {n: x[rows] if n in ("first", "prefix") else x for n, x in opt.items()}
        check_attention(one, out[rows], w[b:b + 1], weights=weights[b:b + 1], decay=0.5, **opt_b)
