"""Workloads of a layer of experts over microscaled 4-bit weights, and of the operators it is made of.

The microscaled formats hold a row in blocks of 32 values with one power of two per block: 2^(b - 127)
for the smallest byte b that leaves no value of the block above the element type's largest (6 for the
4-bit e2m1, 448 for the 8-bit e4m3); each value is the nearest element times that power (ties to even).

Each case runs one operator: "quantize" (rows into such blocks, read back as the values they stand
for), "norm" (the residual's addition, the root-mean-square norm, its output in e4m3 blocks), "product"
(rows, quantized to e4m3 blocks, times 4-bit weights), "route" (scores of the experts, the choice of
top_k, and the rows sorted by expert), "experts" (each row times its expert's weights) or "ffn" (gate
and up products of the chosen experts, silu(gate) * up in e4m3 blocks, the down products, and the
weighted sum of each token's experts added to the residual).

With `own` false the operators run in their plain form, elementary torch operations in 32 bits (64
where a value next to a border decides a code or a choice); with `own` true they are the calls a user
makes of quantized_skinny_matmul_gb300.
"""
import math

import torch

own = False

_BF16, _F32 = torch.bfloat16, torch.float32


def _case(name, **kw):
    c = dict(name=name, op="product", M=1, N=4096, K=4096, bf16=False, kind="e4m3", residual=True,
             E=64, top_k=8, score="softmax", bias=False, groups=1, top_groups=1, best=1, renorm=True, factor=1.0)
    c.update(kw)
    return c


def listed():
    return [
        # a weight matrix brought into 4 bits when a model is loaded
        _case("quantize: weights 11008 x 4096, e2m1", op="quantize", M=11008, kind="e2m1"),
        # a prompt's activations in front of several products, bf16 in
        _case("quantize: prompt 2047 x 4096, e4m3", op="quantize", M=2047, bf16=True),
        # the norm of one decoded token: latency
        _case("norm: 1 x 4096", op="norm"),
        # the norm of a long prompt, bf16 residual stream
        _case("norm: 8191 x 4096, bf16", op="norm", M=8191, bf16=True),
        # one token through an attention projection
        _case("product: 1 row, 4096 x 4096"),
        # a small serving batch through a feed-forward matrix
        _case("product: 16 rows, 11008 x 4096", M=16, N=11008),
        # a prompt through the way back, bf16 activations
        _case("product: 2047 rows, 4096 x 11008, bf16", M=2047, K=11008, bf16=True),
        # the router of one token, softmax scores
        _case("route: 1 x 64, softmax", op="route", E=64),
        # the router of a prompt: sigmoid scores, a bias for balance, 4 of 8 groups
        _case("route: 8192 x 256, sigmoid, groups", op="route", M=8192, E=256, score="sigmoid", bias=True, groups=8,
              top_groups=4, best=2, factor=2.5),
        # one token's experts: their weights' bandwidth and latency
        _case("ffn: 1 token, 8 of 64 experts", op="ffn", N=1408, K=2048),
        # a serving batch, few rows for each expert, some experts without any
        _case("experts: 61 tokens, 8 of 64 experts", op="experts", M=61, N=2816, K=2048),
        # a prompt: hundreds of rows for most experts
        _case("ffn: 4095 tokens, 8 of 64 experts, bf16", op="ffn", M=4095, N=1408, K=2048, bf16=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "product", "product", "route", "experts", "ffn"])
    K, bf16 = 32 * _log(rng, 1, 344), rng.random() < 0.5
    if op in ("quantize", "norm"):
        M = _log(rng, 1, 11008 if op == "quantize" else 8191)
        while M * K > (11008 if op == "quantize" else 8191) * 4096:
            M = (M + 1) // 2
        return _pick(op=op, M=M, K=K, bf16=bf16, kind=rng.choice(["e4m3", "e2m1"]) if op == "quantize" else "e4m3",
                     residual=rng.random() < 0.7)
    if op == "product":
        M, N = _log(rng, 1, 2047), _log(rng, 1, 11008)
        while N * K > 4096 * 11008:
            N = (N + 1) // 2
        return _pick(M=M, N=N, K=K, bf16=bf16)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 2 if groups > 1 else 1, 256 // groups)
        top_groups = rng.randint(1, groups)
        return _pick(op=op, M=_log(rng, 1, 8192), E=E, bf16=bf16, top_k=rng.randint(1, min(10, top_groups * (E // groups))),
                     score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                     best=rng.choice([1, 2]), renorm=rng.random() < 0.7, factor=rng.choice([1.0, 2.5]))
    E = _log(rng, 1, 128)
    k, N, K, M = rng.randint(1, min(E, 8)), 32 * _log(rng, 1, 88), 32 * _log(rng, 1, 128), _log(rng, 1, 4095)
    while E * N * K > 64 * 1408 * 2048:
        N = 32 * ((N // 32 + 1) // 2)
        K = 32 * ((K // 32 + 1) // 2)
    while M * k * N * K > 4095 * 8 * 1408 * 2048:
        M = (M + 1) // 2
    return _pick(op=op, M=M, N=N if op == "ffn" else N - rng.randint(0, 31), K=K, E=E, top_k=k, bf16=bf16, residual=rng.random() < 0.7)


def _pick(**kw):
    c = _case("", **kw)
    del c["name"]
    return c


# ---- the inputs ------------------------------------------------------------------------------


def _rows(gen, M, K, dtype, dev):
    """Activations: normal values, a few channels loud."""
    x = torch.randn((M, K), generator=gen, device=dev)
    x[:, ::97] *= 8.0
    return x.to(dtype)


def _scale_cols(K):
    """Bytes of a row's scales: one for each block of 32, and zeros up to a multiple of 16."""
    return -(-K // 512) * 16


def _weights(gen, n, N, K, dev):
    """n matrices [N, K] of normal values in 4-bit blocks: packed codes [n * N, K / 2] and scales."""
    b, v = _mx(torch.randn((n * N, K), generator=gen, device=dev) * K ** -0.5, "e2m1")
    # the code of each of the 8 magnitudes (twice the value), and the sign bit
    table = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], dtype=torch.uint8, device=dev)
    q = table[(v.abs() * 2).int()] + 8 * (v < 0).to(torch.uint8)
    scales = torch.zeros((n * N, _scale_cols(K)), dtype=torch.uint8, device=dev)
    scales[:, :K // 32] = b
    return q[:, 0::2] + 16 * q[:, 1::2], scales


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, M, N, K, E, k = c["op"], c["M"], c["N"], c["K"], c["E"], c["top_k"]
    dtype = _BF16 if c["bf16"] else _F32
    s = {"case": c, "dtype": dtype}
    if op == "route":
        s["logits"] = (1.5 * torch.randn((M, E), generator=gen, device=dev)
                       + 0.5 * torch.randn((E,), generator=gen, device=dev)).to(dtype)
        s["bias"] = 0.1 * torch.randn((E,), generator=gen, device=dev) if c["bias"] else None
        if own:
            s["router"] = _router(c, s["bias"])
        return s
    s["x"] = _rows(gen, M, K, dtype, dev)
    if op == "norm":
        s["residual"] = _rows(gen, M, K, dtype, dev) if c["residual"] else None
        s["w"] = 1.0 + 0.2 * torch.randn((K,), generator=gen, device=dev)
    if op == "product":
        s["codes"], s["scales"] = _weights(gen, 1, N, K, dev)
        if own:
            import quantized_skinny_matmul_gb300 as gq
            s["weights"] = gq.repack_mxfp4(s["codes"], s["scales"], N, K)
    if op in ("experts", "ffn"):
        # what the norm and the router before the experts left: rows in e4m3 blocks, a plan, weights
        b, v = _mx(s["x"].float(), "e4m3")
        s["xb"] = torch.zeros((M, _scale_cols(K)), dtype=torch.uint8, device=dev)
        s["xb"][:, :K // 32] = b
        s["xq"] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        logits = 1.5 * torch.randn((M, E), generator=gen, device=dev) + 0.7 * torch.randn((E,), generator=gen, device=dev)
        top = logits.sort(dim=-1, descending=True, stable=True)
        s["ids"], s["weight"] = top.indices[:, :k].to(torch.int32).contiguous(), torch.softmax(top.values[:, :k], -1)
        s["offsets"], s["rows"], s["pos"] = _plan(s["ids"], E)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["residual"] = _rows(gen, M, K, dtype, dev) if c["residual"] else None
        parts = 2 if op == "ffn" else 1
        s["codes"], s["scales"] = _weights(gen, E * parts, N, K, dev)
        if op == "ffn":
            s["codes2"], s["scales2"] = _weights(gen, E, K, N, dev)
        if own:
            import quantized_skinny_matmul_gb300 as gq
            s["weights"] = gq.repack_mxfp4(s["codes"], s["scales"], N, K)
            if op == "ffn":
                s["weights2"] = gq.repack_mxfp4(s["codes2"], s["scales2"], K, N)
            s["mx"] = gq.MXRows(s["xq"], s["xb"], gq.GQ_MX_E4M3)
            s["plan"] = gq.ExpertPlan(s["offsets"], s["rows"], s["pos"])
    return s


def _router(c, bias):
    import quantized_skinny_matmul_gb300 as gq
    return gq.Router(c["E"], c["top_k"], score=c["score"], bias=bias, groups=c["groups"], top_groups=c["top_groups"],
                     group_best=c["best"], renormalize=c["renorm"], factor=c["factor"])


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"quantize": _quantize, "norm": _norm, "product": _product, "route": _route, "experts": _experts, "ffn": _ffn}[op](s)
    import quantized_skinny_matmul_gb300 as gq
    if op == "quantize":
        return gq.dequantize_mx(gq.quantize_mx(s["x"], gq.GQ_MX_E2M1 if c["kind"] == "e2m1" else gq.GQ_MX_E4M3), _BF16)
    if op == "norm":
        h, mx = gq.rms_norm_mx(s["x"], s["w"], 1e-5, residual=s["residual"])
        return h, gq.dequantize_mx(mx, _BF16)
    if op == "product":
        return gq.mul_mat_mxfp4(s["weights"], s["x"], dtype=s["dtype"])
    if op == "route":
        ids, weight, plan = gq.route(s["logits"], s["router"])
        return ids, weight, plan.offsets, plan.rows, plan.pos
    if op == "experts":
        return gq.mul_mat_mxfp4(s["weights"], s["mx"], plan=s["plan"], gather=True, dtype=s["dtype"])
    act = gq.swiglu_mxfp4(s["weights"], s["mx"], plan=s["plan"], gather=True)
    down = gq.mul_mat_mxfp4(s["weights2"], act, plan=s["plan"], dtype=_F32)
    return gq.experts_combine(down, s["plan"], s["weight"], residual=s["residual"], dtype=_BF16)


def _two(e):
    """2^e in 32 bits, exact: -126 <= e <= 127."""
    return ((e + 127).to(torch.int32) << 23).view(_F32)


def _mx(x, kind):
    """Rows as blocks: (scale bytes [M, K / 32], elements [M, K] in x's type)."""
    M, K = x.shape
    y = x.reshape(M, K // 32, 32)
    top, bits, low = (0.75, 1, 0) if kind == "e2m1" else (0.875, 3, -6)      # largest: top * 2^3, top * 2^9
    m, e = torch.frexp(y.abs().amax(-1))
    b = torch.where(m > 0, e - (3 if kind == "e2m1" else 9) + (m > top) + 127, 0).clamp(0, 254)
    # x / 2^(b - 127), in two exact steps
    y = y * _two((127 - b) // 2)[..., None].to(x.dtype) * _two((127 - b) - (127 - b) // 2)[..., None].to(x.dtype)
    step = _two((torch.frexp(y)[1] - 1).clamp(min=low) - bits).to(x.dtype)
    return b.to(torch.uint8), ((y / step).round() * step).reshape(M, K)


def _values(b, v):
    """What scale bytes and elements stand for, in 32 bits."""
    half = (b.int() - 127) // 2
    return (v.reshape(v.shape[0], -1, 32) * _two(half)[..., None] * _two(b.int() - 127 - half)[..., None]).reshape(v.shape)


def _weight_values(s, codes, scales, N, K):
    """4-bit weights as f32 [n, N, K]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].reshape(-1, K)
    return _values(scales[:, :K // 32], v).reshape(-1, N, K)


def _quantize(s):
    return _values(*_mx(s["x"].float(), s["case"]["kind"])).to(_BF16)


def _norm(s):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["dtype"])
    d = h.double()
    y = d * torch.rsqrt((d * d).mean(-1, keepdim=True) + 1e-5) * s["w"].double()
    b, v = _mx(y, "e4m3")
    return h, _values(b, v.float()).to(_BF16)


def _product(s):
    c = s["case"]
    W = _weight_values(s, s["codes"], s["scales"], c["N"], c["K"])[0]
    return (_values(*_mx(s["x"].float(), "e4m3")) @ W.T).to(s["dtype"])


def _plan(ids, E):
    """Rows sorted by expert, each expert's in the order of the tokens: (offsets [E + 1], token of each row, row of each choice)."""
    T, k = ids.shape
    order = ids.reshape(-1).sort(stable=True)
    pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos[order.indices] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    offsets = torch.searchsorted(order.values, torch.arange(E + 1, dtype=torch.int32, device="cuda"))
    return offsets.to(torch.int32), (order.indices // k).to(torch.int32), pos.reshape(T, k)


def _route(s):
    c = s["case"]
    E, k, g = c["E"], c["top_k"], c["groups"]
    z = s["logits"].double()
    if c["score"] == "softmax":
        p = (z - z.amax(-1, keepdim=True)).exp()
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + (-z).exp())
    choice = p if s["bias"] is None else p + s["bias"].double()
    if c["top_groups"] < g:
        best = choice.reshape(-1, g, E // g).sort(dim=-1, descending=True).values[..., :c["best"]].sum(-1)
        rank = best.sort(dim=-1, descending=True, stable=True).indices.argsort(-1)
        choice = choice.masked_fill((rank >= c["top_groups"]).repeat_interleave(E // g, -1), -math.inf)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(-1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    ids = ids.to(torch.int32)
    return ids, (w * c["factor"]).float(), *_plan(ids, E)


def _by_expert(s, X, W, index):
    """Row r of the plan: X[index[r]] times its expert's matrix, f32.  Rows are padded to the fullest expert's,
    or, where they are fewer than the experts, each takes its own copy of the weights."""
    R, E = index.shape[0], s["case"]["E"]
    r = torch.arange(R, device="cuda")
    off = s["offsets"].long()
    owner = torch.searchsorted(off[1:], r, right=True)
    if R <= E:
        return (W[owner] @ X[index][..., None])[..., 0]
    padded = torch.zeros((E, s["most"], X.shape[1]), device="cuda")
    padded[owner, r - off[owner]] = X[index]
    return (padded @ W.transpose(1, 2))[owner, r - off[owner]]


def _inputs(s):
    return _values(s["xb"][:, :s["case"]["K"] // 32], s["xq"].view(torch.float8_e4m3fn).float())


def _experts(s):
    c = s["case"]
    W = _weight_values(s, s["codes"], s["scales"], c["N"], c["K"])
    return _by_expert(s, _inputs(s), W, s["rows"].long()).to(s["dtype"])


def _ffn(s):
    c = s["case"]
    E, F, K, T, k = c["E"], c["N"], c["K"], c["M"], c["top_k"]
    W = _weight_values(s, s["codes"], s["scales"], F, K).reshape(E, 2 * F, K)
    up = _by_expert(s, _inputs(s), W, s["rows"].long())
    act = up[:, :F] / (1.0 + (-up[:, :F]).exp()) * up[:, F:]
    W = _weight_values(s, s["codes2"], s["scales2"], K, F)
    down = _by_expert(s, _values(*_mx(act, "e4m3")), W, torch.arange(T * k, device="cuda"))
    out = (down[s["pos"].long()] * s["weight"][..., None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(_BF16)


# ---- the definition in 64 bits -------------------------------------------------------------------


def _elements64(kind):
    """The element type's values that are not negative, in the order of their codes."""
    if kind == "e2m1":
        return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    v = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _power64(e):
    """2^e of whole numbers, exact (a power function need not be)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _held64(x, kind):
    """The values that blocks of 32 hold for x [M, K], by the borders between neighbouring elements."""
    el = _elements64(kind)
    y = x.double().reshape(x.shape[0], -1, 32)
    most = y.abs().amax(-1, keepdim=True)
    at = torch.ceil(torch.log2(torch.where(most > 0, most, 1.0) / el[-1])).clamp(min=-127)
    p = _power64(at)
    p = torch.where(most > el[-1] * p, 2 * p, torch.where((most <= el[-1] * p / 2) & (at > -127), p / 2, p))
    p = torch.where(most > 0, p, 2.0 ** -127)
    border = (el[1:] + el[:-1]) / 2
    size = y.abs() / p
    lo, hi = torch.searchsorted(border, size), torch.searchsorted(border, size, right=True)
    return (torch.copysign(el[torch.where(lo % 2 == 0, lo, hi)], y) * p).reshape(x.shape)


def _weight64(codes, scales, N, K):
    el = _elements64("e2m1")
    el = torch.cat([el, -el])
    v = torch.empty((codes.shape[0], K), dtype=torch.float64, device="cuda")
    v[:, 0::2], v[:, 1::2] = el[(codes % 16).long()], el[(codes // 16).long()]
    return (v.reshape(-1, K // 32, 32) * _power64(scales[:, :K // 32, None].long() - 127)).reshape(-1, N, K)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op, N, K, E, k = c["op"], c["N"], c["K"], c["E"], c["top_k"]
    if op == "quantize":
        return _held64(s["x"], c["kind"])
    if op == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        if s["residual"] is None:
            held = h
        else:
            held = h.to(s["dtype"]).double()             # the residual stream is held in its own type
        y = held / torch.sqrt(held.square().sum(-1, keepdim=True) / K + 1e-5) * s["w"].double()
        return h, _held64(y, "e4m3")
    if op == "product":
        return _held64(s["x"], "e4m3") @ _weight64(s["codes"], s["scales"], N, K)[0].T

    def routed():
        """The chosen experts' weights, by masking the best one top_k times."""
        z = s["logits"].double()
        p = torch.softmax(z, -1) if c["score"] == "softmax" else torch.sigmoid(z)
        left = p.clone() if s["bias"] is None else p + s["bias"].double()
        T, E = z.shape
        if c["top_groups"] < c["groups"]:
            g = left.reshape(T, c["groups"], -1)
            value = g.topk(min(c["best"], g.shape[-1]), -1).values.sum(-1)
            keep = torch.zeros_like(value, dtype=torch.bool)
            for _ in range(c["top_groups"]):
                at = value.masked_fill(keep, -math.inf).max(-1, keepdim=True).values == value.masked_fill(keep, -math.inf)
                keep |= at & (at.cumsum(-1) == 1)
            left[~keep.repeat_interleave(E // c["groups"], -1)] = -math.inf
        w = torch.zeros((T, c["top_k"]), dtype=torch.float64, device="cuda")
        for j in range(c["top_k"]):
            at = (left == left.max(-1, keepdim=True).values)
            at &= at.cumsum(-1) == 1
            w[:, j] = p[at]
            left[at] = -math.inf
        return (w / w.sum(-1, keepdim=True) if c["renorm"] else w) * c["factor"]

    if op == "route":
        return None, routed(), None, None, None
    x = _elements64("e4m3")[(s["xq"] & 127).long()] * torch.where(s["xq"] >= 128, -1.0, 1.0)
    x = (x.reshape(-1, K // 32, 32) * _power64(s["xb"][:, :K // 32, None].long() - 127)).reshape(-1, K)
    off, parts, res = s["offsets"].tolist(), 2 if op == "ffn" else 1, []
    for e in range(E):
        r = s["rows"][off[e]:off[e + 1]].long()
        if len(r) == 0:
            continue
        n = slice(e * parts * N, (e + 1) * parts * N)
        y = x[r] @ _weight64(s["codes"][n], s["scales"][n], parts * N, K)[0].T
        if op == "ffn":
            y = _held64(torch.nn.functional.silu(y[:, :N]) * y[:, N:], "e4m3")
            n = slice(e * K, (e + 1) * K)
            y = y @ _weight64(s["codes2"][n], s["scales2"][n], K, N)[0].T
        res.append(y)
    y = torch.cat(res)
    if op == "experts":
        return y
    out = torch.zeros((c["M"], K), dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
    for j in range(k):
        out = out + s["weight"][:, j, None].double() * y[s["pos"][:, j].long()]
    return out


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    c = case
    op, M, N, K, E, k = c["op"], c["M"], c["N"], c["K"], c["E"], c["top_k"]
    size = 2 if c["bf16"] else 4
    block = K * 33 // 32                                             # a row in e4m3 blocks
    if op == "quantize":
        # rows in, blocks out; blocks in, values out
        held = K * 17 // 32 if c["kind"] == "e2m1" else block
        return {"bytes": M * (size * K + 2 * held + 2 * K), "flops": 0}
    if op == "norm":
        return {"bytes": M * (size * K * (3 if c["residual"] else 1) + 2 * block + 2 * K) + 4 * K, "flops": 0}
    if op == "product":
        return {"bytes": N * K * 17 // 32 + size * M * (K + N), "flops": 2 * M * N * K}
    if op == "route":
        return {"bytes": size * M * E + 16 * M * k + 4 * E, "flops": 0}
    # the experts that are reached: each of the R rows finds one at random
    R = M * k
    seen = E * (1.0 - (1.0 - k / E) ** M) if k < E else E
    if op == "experts":
        return {"bytes": int(seen * N * K * 17 // 32) + M * block + 4 * R + size * R * N, "flops": 2 * R * N * K}
    res = size * M * K if c["residual"] else 0
    return {"bytes": int(seen * 3 * N * K * 17 // 32) + M * block + 12 * R + res + 2 * M * K, "flops": 6 * R * N * K}
