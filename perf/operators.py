"""The operators of the decoder's MoE block and what is measured of them.

Three operators around and in the Stable LatentMoE layer, each in its plain
form (elementary torch operations) and as the calls a user makes of the
framework (`own`):

norm   RMSNorm before the block (bf16 operand, and its 8-bit form) and after
       it, fused with the block's gate, its residual scale, the residual and
       the next block's pre-norm
fp8    x W^T with e4m3 operands: activations quantised per token and 128
       inputs with a power-of-two scale, weights with one scale per 128 x 128
few    the whole layer (router, latent, MXFP4 experts, combine, shared
       experts) for a few tokens
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
EPS = 1e-6
BETA, BETA_LIN = 4.0, 25.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)

K3 = {"hidden": 7168, "latent": 3584, "experts": 896, "top_k": 16, "inter": 3072, "shared": 2, "shared_inter": 3072}


def listed():
    return [
        # the norm in front of the layer for one decoded token: a latency
        {"name": "pre 1", "op": "pre", "tokens": 1, "hidden": 7168, "x": "bf16", "q": True},
        # in front of a prompt's layer, residual stream in fp32, operand in bf16 alone
        {"name": "pre 4096 f32", "op": "pre", "tokens": 4096, "hidden": 7168, "x": "f32", "q": False},
        # after the layer for a decode batch, with the next block's norm and a gate per token
        {"name": "post 16 next", "op": "post", "tokens": 16, "hidden": 7168, "x": "bf16", "gate": "token",
         "sigmoid": True, "next": True, "q": True},
        # after a prompt's layer, gate per channel; a ragged prompt length
        {"name": "post 4001 channel", "op": "post", "tokens": 4001, "hidden": 7168, "x": "f32", "gate": "channel",
         "sigmoid": False, "next": False, "q": False},
        # the latent projection of a decode step in 8 bits
        {"name": "fp8 16 latent", "op": "fp8", "tokens": 16, "n": 3584, "k": 7168, "scale": "f32", "out": "f32"},
        # the down product of the first layer's dense FFN for one token: a weight stream
        {"name": "fp8 1 ffn down", "op": "fp8", "tokens": 1, "n": 7168, "k": 33792, "scale": "f32", "out": "f32"},
        # the router's rows over a short prompt: ragged tokens, rows that end inside a scale block
        {"name": "fp8 301 router", "op": "fp8", "tokens": 301, "n": 895, "k": 7168, "scale": "e8m0", "out": "f32"},
        # the shared experts' gate rows over a prompt, checkpoint scales
        {"name": "fp8 4096 gate", "op": "fp8", "tokens": 4096, "n": 6144, "k": 7168, "scale": "f32", "out": "bf16"},
        # the same product with power-of-two weight scales
        {"name": "fp8 4096 gate e8m0", "op": "fp8", "tokens": 4096, "n": 6144, "k": 7168, "scale": "e8m0",
         "out": "bf16"},
        # three tokens through a layer of the test suite's small shape: a latency
        {"name": "few 3 small", "op": "few", "tokens": 3, "hidden": 256, "latent": 128, "experts": 32, "top_k": 4,
         "inter": 128, "shared": 1, "shared_inter": 128},
        # one decoded token through the full layer
        {"name": "few 1", "op": "few", "tokens": 1, **K3},
        # one token and three drafted ones
        {"name": "few 4", "op": "few", "tokens": 4, **K3},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pre", "post", "fp8", "fp8", "few", "few"])
    if op in ("pre", "post"):
        c = {"op": op, "tokens": _log_int(rng, 1, 4096), "hidden": 128 * _log_int(rng, 2, 56),
             "x": rng.choice(["bf16", "f32"])}
        if op == "post":
            c["gate"] = rng.choice(["none", "token", "channel", "full"])
            c["sigmoid"] = c["gate"] != "none" and rng.random() < 0.5
            c["next"] = rng.random() < 0.5
        c["q"] = (op == "pre" or c["next"]) and rng.random() < 0.5
        return c
    if op == "fp8":
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "n": _log_int(rng, 100, 6144),
                "k": 16 * _log_int(rng, 8, 448), "scale": rng.choice(["f32", "e8m0"]),
                "out": rng.choice(["f32", "bf16"])}
    e = _log_int(rng, 16, 896)
    return {"op": op, "tokens": rng.randint(1, 4), "hidden": 128 * _log_int(rng, 2, 56),
            "latent": 128 * _log_int(rng, 1, 28), "experts": e, "top_k": rng.randint(1, min(16, e)),
            "inter": 128 * _log_int(rng, 1, 24), "shared": rng.randint(0, 2), "shared_inter": 128 * rng.randint(1, 24)}


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def empty(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    T = c["tokens"]
    bf = torch.bfloat16
    if c["op"] in ("pre", "post"):
        H = c["hidden"]
        xd = bf if c["x"] == "bf16" else torch.float32
        # residual rows of a deep layer: a few channels much larger than the rest
        s["x"] = (normal(T, H, std=2.0) * torch.exp(normal(H, std=0.7))).to(xd)
        s["gamma"] = (1.0 + normal(H, std=0.1)).to(bf)
        if c["op"] == "post":
            s["y"] = normal(T, H, std=0.5)
            s["scale"] = 0.22
            shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[c["gate"]]
            s["gate"] = None if shape is None else normal(*shape)
            s["out"] = empty(T, H, dtype=xd)
            s["next_gamma"] = (1.0 + normal(H, std=0.1)).to(bf) if c["next"] else None
        if c["op"] == "pre" or c["next"]:
            s["n"] = empty(T, H, dtype=bf)
            if c["q"]:
                s["q"] = empty(T, H, dtype=torch.uint8)
                s["qs"] = empty(T, -(-H // 128), dtype=torch.uint8)
    elif c["op"] == "fp8":
        N, K = c["n"], c["k"]
        kb, nb = -(-K // 128), -(-N // 128)
        # a pre-norm's output: near 1, a few large channels
        s["x"] = (normal(T, K) * torch.exp(normal(K, std=0.5))).to(bf)
        s["w"] = (normal(N, K) * 100.0).clamp(-448.0, 448.0).to(F8)
        if c["scale"] == "e8m0":
            s["w_scale"] = torch.randint(112, 116, (nb, kb), generator=g, device="cuda").to(torch.uint8)
        else:
            s["w_scale"] = torch.exp(normal(nb, kb, std=0.3)) * (0.01 / math.sqrt(K))
        s["q"] = empty(T, K, dtype=torch.uint8)
        s["qs"] = empty(T, kb, dtype=torch.uint8)
        s["out"] = empty(T, N, dtype=bf if c["out"] == "bf16" else torch.float32)
        if own:
            import mxfp4_latent_moe_amd as mx
            s["ws"] = torch.empty(max(16, mx.fp8_gemm_workspace_bytes(T, N, K)), dtype=torch.uint8, device="cuda")
    else:
        H, L, E, I = c["hidden"], c["latent"], c["experts"], c["inter"]
        S = c["shared"] * c["shared_inter"]
        s["x"] = normal(T, H, dtype=bf)
        w = s["w"] = {
            "w_router": normal(E, H, std=0.85 / math.sqrt(H), dtype=bf),
            "bias": normal(E, std=0.05),
            "w_down": normal(L, H, std=1 / math.sqrt(H), dtype=bf),
            "w_up": normal(H, L, std=1 / math.sqrt(L), dtype=bf),
            "gamma": (1.0 + normal(L, std=0.1)).to(bf),
            "sh_gate": normal(S, H, std=1 / math.sqrt(H), dtype=bf),
            "sh_up": normal(S, H, std=1 / math.sqrt(H), dtype=bf),
            "sh_down": normal(H, S, std=1 / math.sqrt(max(S, 1)), dtype=bf),
        }

        def codes(*shape):
            return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)

        for m, rows, cols in (("w1", I, L), ("w3", I, L), ("w2", L, I)):
            # scales that keep a row's product near 1: codes have a mean square of about 7.6
            e = 127 - round(math.log2(2.75 * math.sqrt(cols)))
            w[m + "_packed"] = codes(E, rows, cols // 2)
            w[m + "_scale"] = torch.randint(e - 1, e + 2, (E, rows, cols // 32), generator=g, device="cuda",
                                            dtype=torch.uint8)
        if own:
            import mxfp4_latent_moe_amd as mx
            shape = mx.make_shape(H, L, E, c["top_k"], I, c["shared"], c["shared_inter"], BETA, BETA_LIN, EPS)
            s["moe"] = mx.LatentMoE(shape, w, "cuda")
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import mxfp4_latent_moe_amd as mx
    c = s["case"]
    if c["op"] == "pre":
        mx.block_pre_norm(s["x"], s["gamma"], EPS, n=s["n"], q=s.get("q"), q_scale=s.get("qs"))
        return _normed(s)
    if c["op"] == "post":
        mx.block_post_norm(s["y"], s["x"], s["out"], gamma=s["gamma"], gate=s["gate"], gate_sigmoid=c["sigmoid"],
                           scale=s["scale"], eps=EPS, next_gamma=s["next_gamma"], n=s.get("n"), q=s.get("q"),
                           q_scale=s.get("qs"))
        return {"out": s["out"], **_normed(s)}
    if c["op"] == "fp8":
        mx.fp8_quantize(s["x"], s["q"], s["qs"])
        mx.fp8_gemm(s["q"], s["qs"], s["w"], s["w_scale"], s["out"], s["ws"])
        return s["out"]
    b = s["moe"].forward_few(s["x"])
    return {"out": b["out"], "ids": b["topk_ids"], "weights": b["topk_w"]}


def _normed(s):
    r = {"n": s["n"]} if "n" in s else {}
    if "q" in s:
        r["q"], r["qs"] = s["q"].view(F8), s["qs"].view(torch.float8_e8m0fnu)
    return r


# ---- plain forms


def _quantize(v):
    """Rows of v in e4m3 with the smallest power-of-two scale per 128 that keeps them within 448: (codes, exponents)."""
    T, K = v.shape
    kb = -(-K // 128)
    b = torch.nn.functional.pad(v, (0, kb * 128 - K)).view(T, kb, 128)
    m, p = torch.frexp(b.abs().amax(2))  # amax = m 2^p, m in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp(-126, 127)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    q = torch.ldexp(b, -e[:, :, None]).to(F8)
    return q.view(T, kb * 128)[:, :K].contiguous(), e


def _rms(v, gamma):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS) * gamma.float()


def _operand(s, v):
    r = {"n": v.to(torch.bfloat16)}
    if s["case"]["q"]:
        q, e = _quantize(v)
        r["q"], r["qs"] = q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return r


def _situ(g, u):
    return BETA * torch.tanh(g / BETA) * torch.sigmoid(g) * BETA_LIN * torch.tanh(u / BETA_LIN)


def _mxfp4(packed, scale):
    table = torch.tensor(E2M1, device=packed.device)
    v = table[torch.stack([packed & 15, packed >> 4], -1).int()].flatten(-2)
    s = torch.ldexp(torch.ones((), device=packed.device), scale.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _plain(s):
    c, x = s["case"], s["x"]
    if c["op"] == "pre":
        return _operand(s, _rms(x.float(), s["gamma"]))
    if c["op"] == "post":
        b = _rms(s["y"], s["gamma"]) * s["scale"]
        if s["gate"] is not None:
            b = b * (torch.sigmoid(s["gate"]) if c["sigmoid"] else s["gate"])
        out = (x.float() + b).to(x.dtype)
        return {"out": out, **(_operand(s, _rms(out.float(), s["next_gamma"])) if c["next"] else {})}
    if c["op"] == "fp8":
        q, e = _quantize(x.float())
        K, N = c["k"], c["n"]
        a = q.float() * torch.exp2(e.float()).repeat_interleave(128, 1)[:, :K]
        ws = torch.exp2(s["w_scale"].float() - 127) if c["scale"] == "e8m0" else s["w_scale"]
        w = s["w"].float() * ws.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        return (a @ w.T).to(s["out"].dtype)
    w, k, x = s["w"], c["top_k"], x.float()
    # the choice is made on 32-bit scores of logits summed in 64 bits: values next to a border
    score = torch.sigmoid((x.double() @ w["w_router"].double().T)).float()
    ids = torch.sort(score + w["bias"], dim=1, descending=True, stable=True).indices[:, :k].sort(1).values
    sel = score.gather(1, ids)
    wts = sel / sel.sum(1, keepdim=True)
    z = x @ w["w_down"].float().T
    y = torch.zeros_like(z)
    flat = ids.flatten()
    zt = z[:, None].expand(-1, k, -1).reshape(len(flat), -1, 1)
    h = _situ(torch.bmm(_mxfp4(w["w1_packed"][flat], w["w1_scale"][flat]), zt),
              torch.bmm(_mxfp4(w["w3_packed"][flat], w["w3_scale"][flat]), zt))
    y = torch.bmm(_mxfp4(w["w2_packed"][flat], w["w2_scale"][flat]), h).view(*ids.shape, -1)
    y = (y * wts[:, :, None]).sum(1)
    out = _rms(y, w["gamma"]) @ w["w_up"].float().T
    if c["shared"]:
        out = out + _situ(x @ w["sh_gate"].float().T, x @ w["sh_up"].float().T) @ w["sh_down"].float().T
    return {"out": out, "ids": ids.int(), "weights": wts}


# ---- 64-bit values from the definitions


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, d = s["case"], torch.float64
    x = s["x"].to(d)

    def norm(v, gamma):
        return v * gamma.to(d) * torch.rsqrt(torch.sum(v * v, -1, keepdim=True) / v.shape[-1] + EPS)

    def eight(v):
        """(values on the e4m3 grid over the block's scale, the scale)"""
        q, sc = torch.empty_like(v), torch.empty((v.shape[0], -(-v.shape[1] // 128)), dtype=d, device=v.device)
        for j in range(sc.shape[1]):
            b = v[:, 128 * j:128 * j + 128]
            top = b.abs().amax(1, keepdim=True)
            e = torch.ceil(torch.log2(top / 448.0)).clamp_min(-126)
            e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
            e = torch.where((e > -126) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e)
            t = b / torch.exp2(e)
            # spacing of the grid at t: 2^(floor(log2 |t|) - 3), never below 2^-9
            step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
            q[:, 128 * j:128 * j + 128] = torch.round(t / step) * step
            sc[:, j:j + 1] = torch.exp2(e)
        return q, sc

    def operand(v):
        r = {"n": v}
        if c["q"]:
            r["q"], r["qs"] = eight(v)
        return r

    if c["op"] == "pre":
        return operand(norm(x, s["gamma"]))
    if c["op"] == "post":
        gate = 1.0 if s["gate"] is None else s["gate"].to(d)
        if c["sigmoid"]:
            gate = 1.0 / (1.0 + torch.exp(-gate))
        out = x + s["scale"] * gate * norm(s["y"].to(d), s["gamma"])
        if not c["next"]:
            return {"out": out}
        # the next norm reads the residual as it is stored
        return {"out": out, **operand(norm(out.to(s["out"].dtype).to(d), s["next_gamma"]))}
    if c["op"] == "fp8":
        q, sc = eight(x)
        ws = torch.exp2(s["w_scale"].to(d) - 127) if c["scale"] == "e8m0" else s["w_scale"].to(d)
        out = torch.zeros((x.shape[0], c["n"]), dtype=d, device=x.device)
        rows = torch.arange(c["n"], device=x.device) // 128
        for j in range(sc.shape[1]):
            part = q[:, 128 * j:128 * j + 128] @ s["w"][:, 128 * j:128 * j + 128].to(d).T
            out += part * sc[:, j:j + 1] * ws[rows, j]
        return out
    w, k = s["w"], c["top_k"]
    table = torch.from_numpy(np.array([0, 1, 2, 3, 4, 6, 8, 12], dtype=np.float64) / 2).to(x.device)

    def matrix(name, e):
        p = w[name + "_packed"][e]
        v = torch.empty((p.shape[0], 2 * p.shape[1]), dtype=d, device=x.device)
        for half, code in ((0, p % 16), (1, p // 16)):
            v[:, half::2] = torch.where(code >= 8, -table[(code % 8).long()], table[(code % 8).long()])
        return v * torch.exp2(w[name + "_scale"][e].to(d) - 127).repeat_interleave(32, 1)

    def situ(g, u):
        return BETA * torch.tanh(g / BETA) / (1 + torch.exp(-g)) * BETA_LIN * torch.tanh(u / BETA_LIN)

    out, all_ids, all_w = [], [], []
    z = torch.matmul(x, w["w_down"].to(d).T)
    sigma = 1 / (1 + torch.exp(-torch.matmul(x, w["w_router"].to(d).T)))
    biased = (sigma.float() + w["bias"]).cpu().numpy()
    for t in range(x.shape[0]):
        ids = sorted(np.lexsort((np.arange(biased.shape[1]), -biased[t]))[:k].tolist())
        g = sigma[t, ids] / sigma[t, ids].sum()
        y = torch.zeros_like(z[0])
        for j, e in enumerate(ids):
            y += g[j] * torch.mv(matrix("w2", e), situ(torch.mv(matrix("w1", e), z[t]), torch.mv(matrix("w3", e), z[t])))
        o = torch.mv(w["w_up"].to(d), norm(y[None], w["gamma"])[0])
        if c["shared"]:
            o += torch.mv(w["sh_down"].to(d), situ(torch.mv(w["sh_gate"].to(d), x[t]), torch.mv(w["sh_up"].to(d), x[t])))
        out.append(o)
        all_ids.append(ids)
        all_w.append(g)
    return {"out": torch.stack(out), "ids": torch.tensor(all_ids, dtype=torch.int32), "weights": torch.stack(all_w)}


def work(case):
    c = case
    T = c["tokens"]
    if c["op"] in ("pre", "post"):
        H = c["hidden"]
        xb = 2 if c["x"] == "bf16" else 4
        b = T * H * xb + 2 * H
        f = 4 * T * H
        normed = c["op"] == "pre"
        if c["op"] == "post":
            b += T * H * (4 + xb) + 4 * {"none": 0, "token": T, "channel": H, "full": T * H}[c["gate"]]
            f += 4 * T * H
            normed = c["next"]
        if normed:
            b += 2 * T * H + (2 * H if c["op"] == "post" else 0) + (T * H + T * -(-H // 128) if c["q"] else 0)
        return {"bytes": b, "flops": f}
    if c["op"] == "fp8":
        N, K = c["n"], c["k"]
        kb = -(-K // 128)
        return {"bytes": 2 * T * K + N * K + -(-N // 128) * kb * (4 if c["scale"] == "f32" else 1)
                + T * N * (4 if c["out"] == "f32" else 2), "flops": 2 * T * N * K}
    H, L, E, I, k = c["hidden"], c["latent"], c["experts"], c["inter"], c["top_k"]
    S = c["shared"] * c["shared_inter"]
    # distinct experts of T tokens with k of E each, every choice alike
    n = E * (1 - (1 - k / E) ** T)
    dense = E * H + 2 * L * H + 3 * S * H
    return {"bytes": 2 * dense + 4 * E + 2 * L + n * 3 * I * L * 17 / 32 + T * H * 6 + 8 * T * k,
            "flops": 2 * T * (dense + k * 3 * I * L)}
