"""The paged 8-bit KV cache in numpy and 64 bits: the definitions of gq.h written out, for the GPU tests."""
import math

import numpy as np

E4M3 = np.array([((m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)) for e in range(16)
                 for m in range(8)][:127])      # the values of codes 0 .. 126 (127 is NaN)


def decode(kind, codes):
    if kind == 0:
        return codes.astype(np.int8).astype(np.float64)
    u = codes.astype(np.uint8)
    mag = np.append(E4M3, np.nan)[u & 127]
    return np.where(u >= 128, -mag, mag)


def encode(kind, y):
    """Codes of the nearest values to y, ties to the even code."""
    if kind == 0:
        return np.clip(np.rint(y), -127, 127).astype(np.int8)
    borders, a = (E4M3[1:] + E4M3[:-1]) / 2, np.abs(y)
    below, upto = np.searchsorted(borders, a, "left"), np.searchsorted(borders, a, "right")
    return (np.where(below % 2 == 0, below, upto) + 128 * np.signbit(y)).astype(np.uint8)


def append(kind, P, codes, scale, table, held, cu, x):
    """codes [pages, P, D], scale [pages] after the step's x [T, Hkv, D] (copies; one of keys and values)."""
    codes, scale = codes.copy(), scale.copy()
    top = np.float32(127.0 if kind == 0 else 448.0)
    B, Hkv, _ = table.shape
    for b in range(B):
        n = cu[b + 1] - cu[b]
        for j in range(held[b] // P, -(-(held[b] + n) // P)):
            new = [s for s in range(j * P, j * P + P) if held[b] <= s < held[b] + n]
            for h in range(Hkv if new else 0):
                pg, fill = table[b, h, j], max(0, held[b] - j * P)
                rows = x[[cu[b] + s - held[b] for s in new], h]
                old = scale[pg] if fill else np.float32(0)
                s = max(old, np.float32(np.abs(rows).max()) / top)
                assert s.dtype == np.float32
                val = np.concatenate([decode(kind, codes[pg, :fill]) * np.float64(old), rows.astype(np.float64)])
                y = val / np.float64(s) if s > 0 else np.zeros_like(val)
                if not (s == 0 and kind):
                    y = y + 0.0
                codes[pg, :fill + len(new)] = encode(kind, y)
                scale[pg] = s
    return codes, scale


def visible(base_row, P, N, qpos, first, prefix, window):
    x = (base_row[:, None].astype(np.int64) + np.arange(P)).reshape(-1)[:N]
    near = (x <= qpos) & ((qpos - x < window) if window else True)
    return x, (x >= first) & (near | (x < prefix))


def attend(kind, P, k, ks, v, vs, table, base, held, seen, cu, q, scale, cap=0.0, window=0, slopes=None, first=None,
           prefix=None, weights=None, decay=1.0):
    """(out [T, Hq, D], weights, E [T, Hq, D], S [T, Hq], rel [B, Hkv, NB]): E = sum p |v|, S bounds the scores of
    a row, rel the sum of the page's shares times their rows' S."""
    B, Hkv, NB = table.shape
    T, Hq, D = q.shape
    G = Hq // Hkv
    out, E, S = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    w, rel = np.zeros((B, Hkv, NB)), np.zeros((B, Hkv, NB))
    for b in range(B):
        n = cu[b + 1] - cu[b]
        N = held[b] + n
        used = -(-N // P)
        if weights is not None:
            w[b, :, :used] = decay * weights[b, :, :used].astype(np.float64)
        for h in range(Hkv):
            ids = table[b, h, :used]
            K = (decode(kind, k[ids]) * ks[ids].astype(np.float64)[:, None, None]).reshape(-1, D)[:N]
            V = (decode(kind, v[ids]) * vs[ids].astype(np.float64)[:, None, None]).reshape(-1, D)[:N]
            for i in range(n):
                t, qp = cu[b] + i, seen[b] + i
                x, see = visible(base[b, h, :used], P, N, qp, first[t] if first is not None else 0,
                                 prefix[t] if prefix is not None else 0, window)
                if not see.any():
                    continue
                for g in range(G):
                    a = q[t, h * G + g].astype(np.float64)
                    z = scale * (K[see] @ a)
                    size = scale * (np.abs(K[see]) @ np.abs(a)) + 4 * cap
                    if cap:
                        z = cap * np.tanh(z / cap)
                    if slopes is not None:
                        z = z - np.float64(slopes[h * G + g]) * np.abs(qp - x[see])
                        size = size + np.float64(slopes[h * G + g]) * np.abs(qp - x[see])
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    out[t, h * G + g] = p @ V[see]
                    E[t, h * G + g] = p @ np.abs(V[see])
                    # far tokens with no weight do not matter: the largest bound among those that count
                    S[t, h * G + g] = size[p > 2.0 ** -60].max()
                    share = np.zeros(used * P)
                    share[:N][see] = p
                    w[b, h, :used] += share.reshape(used, P).sum(1)
                    rel[b, h, :used] += share.reshape(used, P).sum(1) * S[t, h * G + g]
    return out, w, E, S, rel


def evict(P, table, base, w, held, budget, keep_first, keep_last):
    table, base, w, out = table.copy(), base.copy(), w.copy(), held.copy()
    B, Hkv, _ = table.shape
    for b in range(B):
        n = -(-int(held[b]) // P)
        if n <= budget:
            continue
        out[b] = held[b] - (n - budget) * P
        for h in range(Hkv):
            mid = sorted(range(keep_first, n - keep_last), key=lambda j: (-w[b, h, j], j))
            keep = set(mid[:budget - keep_first - keep_last]) | set(range(keep_first)) | set(range(n - keep_last, n))
            order = sorted(keep) + [j for j in range(n) if j not in keep]
            for a in (table, base, w):
                a[b, h, :n] = a[b, h, order]
            w[b, h, budget:n] = 0.0
    return table, base, w, out


def tolerance(S, T):
    """Bound of an output's or a page weight's relative error; see tests/test_gpu_pages.py."""
    return 2.0 * (70.0 * S + T / 2.0 + 64.0) * 2.0 ** -24


def problem(seed, kind, B, Hkv, G, D, P, held, new, gaps=False, extra=2):
    """A filled cache (held tokens and the step's new ones in place) and the step's queries, numpy."""
    gen = np.random.default_rng(seed)
    held, new = np.asarray(held, np.int32), np.asarray(new, np.int32)
    NB = int(max(1, max(-(-(h + n) // P) for h, n in zip(held, new)))) + extra
    pages = B * Hkv * NB + 3
    table = gen.permutation(pages)[:B * Hkv * NB].astype(np.int32).reshape(B, Hkv, NB)
    base = np.full((B, Hkv, NB), -(1 << 20), np.int32)
    seen = held.copy()
    for b in range(B):
        ob, nb = -(-int(held[b]) // P), -(-int(held[b] + new[b]) // P)
        gone = int(gen.integers(0, ob + 1)) if gaps and ob > 1 else 0
        seen[b] += gone * P
        for h in range(Hkv):
            old = np.sort(gen.permutation(max(0, ob + gone - 1))[:max(0, ob - 1)])
            row = np.concatenate([old, np.arange(ob - 1 + gone, nb + gone)]) if ob else np.arange(nb)
            base[b, h, :nb] = row * P
    arr = {}
    for name in ("k", "v"):
        x = gen.standard_normal((pages, P, D)) * np.where(np.arange(D) % 16 == 0, 3.0, 1.0)
        s = np.abs(x).max((1, 2)) / (127.0 if kind == 0 else 448.0)
        arr[name] = encode(kind, x / s[:, None, None])
        arr[name + "s"] = s.astype(np.float32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = gen.standard_normal((int(cu[-1]), Hkv * G, D)).astype(np.float32)
    return dict(kind=kind, P=P, table=table, base=base, held=held, seen=seen, cu=cu, q=q, gen=gen, **arr)


def alibi(Hq):
    return (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)


SCALE = lambda D: 1.0 / math.sqrt(D)  # noqa: E731
