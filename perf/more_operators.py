"""4-bit operands on both sides of the layer's products, and what is measured of them.

Three groups of operators, each in its plain form (elementary torch operations)
and as the calls a user makes of the framework (`own`):

quant    rows to MXFP4 (e2m1 codes, a power-of-two scale per 32 values) and back
gemm     x W^T with both operands in MXFP4: the activations quantised, then the
         product with weights kept in that form
experts  the products of the routed experts on rows sorted by expert, ragged:
         gate and up with SiTU-GLU (`glu`), down with a weight per pair
         (`down`), and both in a row with 4-bit rows in between (`mlp`)
"""
import math

import torch

own = False

BETA, BETA_LIN = 4.0, 25.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)

K3 = {"latent": 3584, "inter": 3072}


def listed():
    return [
        # the input of a decoded token's dense products: a latency
        {"name": "quant 1", "op": "quant", "rows": 1, "k": 7168, "x": "bf16", "out": "f32", "rule": "fit"},
        # the latent rows of several prompts, to the format's own scale rule
        {"name": "quant 16384 ocp", "op": "quant", "rows": 16384, "k": 3584, "x": "f32", "out": "bf16", "rule": "ocp"},
        # the latent projection of one decoded token
        {"name": "gemm 1 latent", "op": "gemm", "tokens": 1, "n": 3584, "k": 7168, "out": "f32"},
        # the down product of the first layer's dense FFN for a decode batch: a weight stream
        {"name": "gemm 16 ffn down", "op": "gemm", "tokens": 16, "n": 7168, "k": 33792, "out": "bf16"},
        # the router's rows over a short prompt: ragged on every side
        {"name": "gemm 301 router", "op": "gemm", "tokens": 301, "n": 895, "k": 7168, "out": "f32"},
        # the shared experts' gate rows over a prompt
        {"name": "gemm 4096 gate", "op": "gemm", "tokens": 4096, "n": 6144, "k": 7168, "out": "bf16"},
        # one decoded token's gate and up products at full size, hidden rows in fp32
        {"name": "glu 1", "op": "glu", "tokens": 1, "experts": 896, "top_k": 16, **K3, "skew": 0.0, "out": "f32"},
        # the down products of a batch whose load sits on a few experts, with the routing weights
        {"name": "down 256 skewed", "op": "down", "tokens": 256, "experts": 64, "top_k": 4, **K3, "skew": 2.0,
         "out": "f32"},
        # three tokens through experts of the test suite's small shape: a latency
        {"name": "mlp 3 small", "op": "mlp", "tokens": 3, "experts": 32, "top_k": 4, "latent": 128, "inter": 128,
         "skew": 0.0, "out": "bf16"},
        # a decode batch through the routed experts at full size
        {"name": "mlp 16", "op": "mlp", "tokens": 16, "experts": 896, "top_k": 16, **K3, "skew": 0.0, "out": "bf16"},
        # a prompt on one GPU's share of the experts (112 of 896, two of a token's 16 on average)
        {"name": "mlp 4096 share", "op": "mlp", "tokens": 4096, "experts": 112, "top_k": 2, **K3, "skew": 0.3,
         "out": "bf16"},
        # several prompts on that share
        {"name": "mlp 16384 share", "op": "mlp", "tokens": 16384, "experts": 112, "top_k": 2, **K3, "skew": 0.0,
         "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "glu", "down", "mlp", "mlp"])
    if op == "quant":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "k": _log_int(rng, 1, 3584), "x": rng.choice(["bf16", "f32"]),
                "out": rng.choice(["bf16", "f32"]), "rule": rng.choice(["fit", "ocp"])}
    if op == "gemm":
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "n": _log_int(rng, 100, 6144), "k": 32 * _log_int(rng, 3, 224),
                "out": rng.choice(["bf16", "f32"])}
    e = _log_int(rng, 4, 112)
    return {"op": op, "tokens": _log_int(rng, 1, 4096), "experts": e, "top_k": rng.randint(1, min(6, e)),
            "latent": 32 * _log_int(rng, 4, 112), "inter": 32 * _log_int(rng, 2, 96), "skew": rng.choice([0.0, 0.5, 2.0]),
            "out": "bf16" if op == "mlp" else rng.choice(["bf16", "f32"])}


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def empty(*shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    def weights(name, *rows_k):
        # codes have a mean square of about 7.6: scales that keep a row's product near 1
        *rows, k = rows_k
        e = 127 - round(math.log2(2.75 * math.sqrt(k)))
        s[name] = torch.randint(0, 256, (*rows, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        s[name + "_scale"] = torch.randint(e - 1, e + 2, (*rows, k // 32), generator=g, device="cuda", dtype=torch.uint8)

    if c["op"] == "quant":
        T, K = c["rows"], c["k"]
        # rows near 1 with a few channels much larger than the rest
        s["x"] = (normal(T, K) * torch.exp(normal(K, std=0.7))).to(_dtype(c["x"]))
        s["q"], s["qs"] = empty(T, -(-K // 2)), empty(T, -(-K // 32))
        s["out"] = empty(T, K, dtype=_dtype(c["out"]))
        return s
    if c["op"] == "gemm":
        T, N, K = c["tokens"], c["n"], c["k"]
        s["x"] = (normal(T, K) * torch.exp(normal(K, std=0.5))).to(torch.bfloat16)
        weights("w", N, K)
        s["q"], s["qs"] = empty(T, K // 2), empty(T, K // 32)
        s["out"] = empty(T, N, dtype=_dtype(c["out"]))
        if own:
            import mxfp4_latent_moe_amd as mx
            s["ws"] = empty(max(16, mx.mxfp4_gemm_workspace_bytes(T, N, K)))
        return s
    T, E, k, L, I = c["tokens"], c["experts"], c["top_k"], c["latent"], c["inter"]
    P = T * k
    # the routing, as moe_permute leaves it: a token's experts ascend, pairs sorted by expert
    score = normal(T, E) + c["skew"] * normal(E)
    ids = torch.topk(score, k, dim=1).indices.sort(1).values.flatten()
    s["pair"] = torch.sort(ids, stable=True).indices.int()
    s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    count = torch.bincount(ids, minlength=E)
    s["offsets"][1:] = torch.cumsum(count, 0)
    s["most"] = int(count.max())
    if c["op"] == "down":
        s["x"] = normal(P, I, std=0.5)
        s["pair_weight"] = torch.softmax(normal(T, k), 1).flatten()
        weights("w2", E, L, I)
        s["q"], s["qs"] = empty(P, I // 2), empty(P, I // 32)
        s["out"] = empty(P, L, dtype=_dtype(c["out"]))
    else:
        s["x"] = normal(T, L)
        weights("w1", E, I, L)
        weights("w3", E, I, L)
        s["q"], s["qs"] = empty(T, L // 2), empty(T, L // 32)
        if c["op"] == "glu":
            s["out"] = empty(P, I, dtype=_dtype(c["out"]))
        else:
            weights("w2", E, L, I)
            s["h"], s["hs"] = empty(P, I // 2), empty(P, I // 32)
            s["out"] = empty(P, L, dtype=_dtype(c["out"]))
    if own:
        import mxfp4_latent_moe_amd as mx
        s["ws"] = empty(max(16, mx.mxfp4_expert_gemm_workspace_bytes(E, P, L, I), mx.mxfp4_expert_gemm_workspace_bytes(E, P, I, L)))
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import mxfp4_latent_moe_amd as mx
    c = s["case"]
    mx.mxfp4_quantize(s["x"], s["q"], s["qs"], rule=c.get("rule", "fit"))
    if c["op"] == "quant":
        mx.mxfp4_dequantize(s["q"], s["qs"], s["out"])
        return s["out"]
    if c["op"] == "gemm":
        mx.mxfp4_gemm(s["q"], s["qs"], s["w"], s["w_scale"], s["out"], s["ws"])
        return s["out"]
    if c["op"] == "down":
        mx.mxfp4_expert_gemm(s["q"], s["qs"], s["w2"], s["w2_scale"], s["offsets"], s["out"], s["ws"],
                             sorted_pair=s["pair"], pair_weight=s["pair_weight"])
        return s["out"]
    glu = {"w3": s["w3"], "w3_scale": s["w3_scale"], "sorted_pair": s["pair"], "top_k": c["top_k"], "beta": BETA,
           "beta_lin": BETA_LIN}
    if c["op"] == "glu":
        mx.mxfp4_expert_gemm(s["q"], s["qs"], s["w1"], s["w1_scale"], s["offsets"], s["out"], s["ws"], **glu)
        return s["out"]
    mx.mxfp4_expert_gemm(s["q"], s["qs"], s["w1"], s["w1_scale"], s["offsets"], s["h"], s["ws"], out_scale=s["hs"], **glu)
    mx.mxfp4_expert_gemm(s["h"], s["hs"], s["w2"], s["w2_scale"], s["offsets"], s["out"], s["ws"])
    return s["out"]


# ---- plain forms


def _four(x, rule):
    """Rows of x rounded to MXFP4, as the values that the codes and scales stand for (fp32)."""
    T, K = x.shape
    kb = -(-K // 32)
    b = torch.nn.functional.pad(x.float(), (0, 32 * kb - K)).view(T, kb, 32)
    m, p = torch.frexp(b.abs().amax(2, keepdim=True))  # amax = m 2^p, m in [0.5, 1); 6 = 0.75 2^3
    e = torch.where((m > 0.75) & (rule == "fit"), p - 2, p - 3)
    e = torch.where(m == 0, torch.full_like(e, -125), e).clamp(-125, 126)
    a = torch.ldexp(b.abs(), -e)
    # how many of the midpoints between codes lie below; a tie goes to the even code
    n = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    v = torch.tensor(E2M1[:8], device=x.device)[n]
    return torch.ldexp(torch.copysign(v, b), e).view(T, 32 * kb)[:, :K]


def _weights(packed, scale):
    table = torch.tensor(E2M1, device=packed.device)
    v = table[torch.stack([packed & 15, packed >> 4], -1).flatten(-2).int()]
    s = torch.ldexp(torch.ones((), device=packed.device), scale.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _situ(g, u):
    return BETA * torch.tanh(g / BETA) * torch.sigmoid(g) * BETA_LIN * torch.tanh(u / BETA_LIN)


def _plain(s):
    c = s["case"]
    x = _four(s["x"], c.get("rule", "fit"))
    if c["op"] == "quant":
        return x.to(_dtype(c["out"]))
    if c["op"] == "gemm":
        return (x @ _weights(s["w"], s["w_scale"]).T).to(_dtype(c["out"]))
    E, k, off, pair = c["experts"], c["top_k"], s["offsets"].long(), s["pair"].long()
    at = torch.arange(len(pair), device=off.device)
    expert = torch.searchsorted(off, at, right=True) - 1
    few = 2 * len(pair) < E  # a matrix for each row, or rows padded to the longest expert's

    def product(rows, name):
        w, ws = s[name], s[name + "_scale"]
        if few:
            return torch.bmm(_weights(w[expert], ws[expert]), rows[:, :, None])[:, :, 0]
        place = at - off[expert]
        padded = torch.zeros((E, s["most"], rows.shape[1]), device=rows.device)
        padded[expert, place] = rows
        return torch.bmm(_weights(w, ws), padded.transpose(1, 2).contiguous())[expert, :, place]

    if c["op"] == "down":
        return (product(x, "w2") * s["pair_weight"][pair][:, None]).to(_dtype(c["out"]))
    rows = x[pair // k]
    h = _situ(product(rows, "w1"), product(rows, "w3"))
    if c["op"] == "mlp":
        h = product(_four(h, "fit"), "w2")
    return h.to(_dtype(c["out"]))


# ---- 64-bit values from the definitions


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, d = s["case"], torch.float64

    def rounded(v, rule):
        """v on the grid of e2m1 over each block's scale"""
        r = torch.empty_like(v)
        for j in range(0, v.shape[1], 32):
            b = v[:, j:j + 32]
            top = b.abs().amax(1, keepdim=True)
            e = torch.floor(torch.log2(top.clamp_min(2.0 ** -140)))
            e = torch.where(top < torch.exp2(e), e - 1, torch.where(top >= torch.exp2(e + 1), e + 1, e)) - 2
            if rule == "fit":
                e = torch.where(top > 6 * torch.exp2(e), e + 1, e)
            scale = torch.exp2(e.clamp(-125, 126))
            t = b / scale
            # spacing of the grid at t: a half up to 2, 1 up to 4, 2 above; 6 is the last
            step = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0))
            r[:, j:j + 32] = (torch.round(t / step) * step).clamp(-6, 6) * scale
        return r

    def matrix(name, at=None):
        p, e = (s[name], s[name + "_scale"]) if at is None else (s[name][at], s[name + "_scale"][at])
        v = torch.empty((p.shape[0], 2 * p.shape[1]), dtype=d, device=p.device)
        for half, code in ((0, p % 16), (1, p // 16)):
            n = (code % 8).to(d)
            mag = torch.where(n < 4, n / 2, torch.where(n < 6, n - 2, 2 * n - 8))
            v[:, half::2] = torch.where(code >= 8, -mag, mag)
        return v * torch.exp2(e.to(d) - 127).repeat_interleave(32, 1)

    def situ(g, u):
        return BETA * torch.tanh(g / BETA) / (1 + torch.exp(-g)) * BETA_LIN * torch.tanh(u / BETA_LIN)

    x = rounded(s["x"].to(d), c.get("rule", "fit"))
    if c["op"] == "quant":
        return x
    if c["op"] == "gemm":
        return torch.matmul(x, matrix("w").T)
    off, pair = s["offsets"].tolist(), s["pair"].long()
    out = torch.zeros(s["out"].shape, dtype=d, device=x.device)
    for e in range(c["experts"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        if c["op"] == "down":
            out[lo:hi] = torch.matmul(x[lo:hi], matrix("w2", e).T) * s["pair_weight"][pair[lo:hi]].to(d)[:, None]
            continue
        rows = x[torch.div(pair[lo:hi], c["top_k"], rounding_mode="floor")]
        h = situ(torch.matmul(rows, matrix("w1", e).T), torch.matmul(rows, matrix("w3", e).T))
        out[lo:hi] = torch.matmul(rounded(h, "fit"), matrix("w2", e).T) if c["op"] == "mlp" else h
    return out


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "quant":
        T, K = c["rows"], c["k"]
        # codes and scales are written by the one call and read by the other
        return {"bytes": T * K * (size[c["x"]] + size[c["out"]]) + 2 * T * (-(-K // 2) + -(-K // 32)), "flops": 4 * T * K}
    if c["op"] == "gemm":
        T, N, K = c["tokens"], c["n"], c["k"]
        return {"bytes": 2 * T * K + N * K * 17 / 32 + T * N * size[c["out"]], "flops": 2 * T * N * K}
    T, E, k, L, I = c["tokens"], c["experts"], c["top_k"], c["latent"], c["inter"]
    P = T * k
    # distinct experts of T tokens with k of E each, every choice alike
    n = E * (1 - (1 - k / E) ** T)
    mats = {"down": 1, "glu": 2, "mlp": 3}[c["op"]]
    rows = 4 * P * I + 4 * P if c["op"] == "down" else 4 * T * L
    return {"bytes": mats * n * I * L * 17 / 32 + rows + 4 * (P + E) + P * (I if c["op"] == "glu" else L) * size[c["out"]],
            "flops": 2 * mats * P * I * L}
