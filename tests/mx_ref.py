"""The microscaled formats, the norm, routing and the experts' products in numpy and 64 bits, from their definitions."""
import numpy as np

E2M1, E4M3 = 0, 1
U = 2.0 ** -24

# the elements that are not negative, in the order of their codes
ELEMENTS = {E2M1: np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0]),
            E4M3: np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]}


def cols(K):
    return -(-K // 512) * 16


def quantize(x, kind):
    """(codes uint8 [M, K], one per value, sign in the top bit of the element; scale bytes [M, K / 32])."""
    el = ELEMENTS[kind]
    x = np.asarray(x, np.float64)
    M, K = x.shape
    y = x.reshape(M, K // 32, 32)
    with np.errstate(invalid="ignore"):
        fine = np.isfinite(y).all(-1)
    most = np.where(fine, np.abs(np.where(np.isfinite(y), y, 0)).max(-1), 0)
    b = np.zeros(most.shape, np.int64)
    for step in range(255):                                  # the smallest byte that leaves nothing above the largest element
        b = np.where(most > el[-1] * 2.0 ** (b - 127.0), b + 1, b)
    size = np.where(fine[..., None], np.abs(y), 0) / 2.0 ** (b[..., None] - 127.0)
    border = (el[1:] + el[:-1]) / 2
    lo, hi = np.searchsorted(border, size, "left"), np.searchsorted(border, size, "right")
    code = np.where(lo % 2 == 0, lo, hi)
    sign = np.signbit(y) & fine[..., None]
    top = 8 if kind == E2M1 else 128
    return (code + top * sign).astype(np.uint8).reshape(M, K), np.where(fine, b, 255).astype(np.uint8)


def pack(codes, kind):
    """The codes as they lie in memory."""
    return codes if kind == E4M3 else codes[:, 0::2] | codes[:, 1::2] << 4


def unpack(codes, kind):
    return codes if kind == E4M3 else np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)


def values(codes, b, kind):
    """What codes (one per value) and scale bytes stand for."""
    top = 8 if kind == E2M1 else 128
    el = np.append(ELEMENTS[kind], np.nan)
    v = el[np.minimum(codes & (top - 1), len(el) - 1)] * np.where(codes & top, -1.0, 1.0)
    p = np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))
    return (v.reshape(*b.shape, 32) * p[..., None]).reshape(codes.shape)


def held(x, kind):
    return values(*quantize(x, kind), kind)


def norm(h, w, eps):
    h = np.asarray(h, np.float64)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return y if w is None else y * np.asarray(w, np.float64)


def product(X, W):
    """(X W^T, sum of |terms|)."""
    return X @ W.T, np.abs(X) @ np.abs(W).T


def product_tolerance(K):
    """Per sum of |terms|: the tensor cores cut at most two units (2^-23) off the running sum for each 32 columns, and each take-over
    of the accumulators (every 512 columns or more) rounds once, as does the end and up to three joins of shared columns."""
    return (K / 32 + 1) * 2.0 ** -22 + (K / 512 + 8) * U


def swiglu(X, Wg, Wu):
    """(silu(gate) * up, how far f32 sums may be off it)."""
    g, eg = product(X, Wg)
    u, eu = product(X, Wu)
    s = g / (1 + np.exp(-g))
    tol = product_tolerance(X.shape[1])
    # |d silu| <= 1.1 |d gate|; the fast exponential and reciprocal, and two products: 2^-19 with |gate| up to 64
    return s * u, 1.1 * np.abs(u) * eg * tol + np.abs(s) * eu * tol + 2.0 ** -19 * np.abs(s * u)


def route(z, k, score="softmax", bias=None, groups=1, top_groups=1, best=1, renormalize=True, factor=1.0):
    """(ids, weights): the values of exact arithmetic, equal ones by the lower index."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, np.float64))
    T, E = z.shape
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if score == "softmax":
            m = z.max(-1, keepdims=True)
            e = np.where(np.isfinite(m), np.exp(z - np.where(np.isfinite(m), m, 0)), 0)
            p = e / np.maximum(e.sum(-1, keepdims=True), 1e-300)
        else:
            p = 1 / (1 + np.exp(-z))
    c = p + np.asarray(bias, np.float64) if bias is not None else z
    allowed = np.ones((T, E), bool)
    if top_groups < groups:
        v = np.sort((c if bias is not None or best == 1 else p).reshape(T, groups, -1), -1)[..., ::-1][..., :best].sum(-1)
        order = np.argsort(-v, -1, kind="stable")[:, :top_groups]
        g = np.zeros((T, groups), bool)
        np.put_along_axis(g, order, True, -1)
        allowed = np.repeat(g, E // groups, -1)
    ids = np.zeros((T, k), np.int32)
    for t in range(T):
        e = np.flatnonzero(allowed[t])
        ids[t] = e[np.argsort(-c[t, e], kind="stable")[:k]]
    w = np.take_along_axis(p, ids, -1)
    if renormalize:
        s = w.sum(-1, keepdims=True)
        w = np.where(s > 0, w / np.where(s > 0, s, 1), w)
    return ids, w * factor


def plan(ids, E):
    """(offsets, token of each row, row of each choice); ids -1 have none."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    there = np.flatnonzero(flat >= 0)
    order = there[np.argsort(flat[there], kind="stable")]
    pos = np.full(T * k, -1, np.int32)
    pos[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[there], minlength=E))]).astype(np.int32)
    return offsets, (order // k).astype(np.int32), pos.reshape(T, k)
