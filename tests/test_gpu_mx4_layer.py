"""The layer with its routed experts on MXFP4 rows: quantisation, gate and up, down and combine together.

Every step against float64 from the step before's own output, with the bounds
of test_gpu_mx4.py: a product is off by (128 + K / 64 + 16) 2^-23 of its sum of
magnitudes, and SiTU-GLU by (32 + |g|) 2^-23 of its value and what the two
products' errors make of it, 1.2 |u| and |g| times theirs (the derivative of
beta tanh(g / beta) sigmoid(g) is below 1.1).
"""
import numpy as np
import pytest
import torch

import synth
from synth.device import to_dev_bf16, upload_weights
from gpu_common import say
from oracle import mx4

pytestmark = pytest.mark.gpu
DEV = "cuda"
MID = synth.LayerShape(1024, 512, 64, 4, 768, 1, 256)
TINY = synth.TINY_SHAPE


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as m
    m.load()
    return m


def setup(mx, shape, T):
    wl = synth.Workload(f"rows4_{T}", 29, shape, T, 29, 0.02, 0.1, "normal", 119, 121)
    w = upload_weights(wl, DEV)
    return mx.shape_of(shape), w, to_dev_bf16(synth.gen_tokens(wl), DEV)


def numpy_of(b):
    return {k: v.cpu().numpy() for k, v in b.items() if not k.startswith("ws")}


@pytest.mark.parametrize("shape,T", [(TINY, 1), (TINY, 8), (TINY, 301), (MID, 1), (MID, 16), (MID, 200), (MID, 1200)])
def test_layer(mx, shape, T):
    from mxfp4_latent_moe_amd import ops
    say(f"case: layer on MXFP4 rows, {shape.n_experts} experts, T={T}")
    s, w, x = setup(mx, shape, T)
    b = mx.LatentMoE(s, w, DEV, mxfp4_rows=True).forward(x)
    torch.cuda.synchronize()
    plain = mx.LatentMoE(s, w, DEV).forward(x)
    out = torch.empty_like(b["out"])
    ops.shared_ffn(s, x, w["sh_gate"], w["sh_up"], w["sh_down"], out, 0, b["ws_shared"])
    ops.combine_norm_up(s, T, b["Y"], b["pair_pos"], b["topk_w"], w["gamma"], w["w_up"], out, 1, b["ws"])
    torch.cuda.synchronize()
    for k in ("topk_ids", "topk_w", "z", "offsets", "sorted_pair", "pair_pos"):
        assert torch.equal(b[k], plain[k]), k
    assert torch.equal(b["out"], out)
    g, L, I, k = numpy_of(b), s.latent, s.inter, s.top_k  # noqa: E741
    zq, zs = mx4.quantize(g["z"].astype(np.float64), "fit")
    assert (g["zq"] == zq).all() and (g["zq_scale"] == zs).all()
    host = {n: w[n].cpu().numpy() for n in w if n[:2] in ("w1", "w3", "w2")}
    deq = lambda n, K: mx4.dequantize(host[n + "_packed"], host[n + "_scale"], K)  # noqa: E731
    w1, w3, w2, z, src = deq("w1", L), deq("w3", L), deq("w2", I), mx4.dequantize(zq, zs, L), g["sorted_pair"] // k
    gate, _, mg = mx4.expert_product(z, w1, g["offsets"], rows=src)
    up, _, mu = mx4.expert_product(z, w3, g["offsets"], rows=src)
    eps = (128 + L // 64 + 16) * 2.0 ** -23
    ref = mx4.situ_glu(gate, up)
    tol = np.abs(ref) * (32 + np.abs(gate)) * 2.0 ** -23 + eps * (1.2 * mg * np.abs(up) + mu * np.abs(gate)) + 1e-37
    lo, hi = (mx4.scale_exponent(np.maximum(np.abs(ref) + d * tol, 0).reshape(len(ref), -1, 32).max(2), "fit") + 127
              for d in (-1, 1))
    assert ((lo <= g["H_scale"]) & (g["H_scale"] <= hi)).all()
    unit = np.repeat(2.0 ** (g["H_scale"].astype(np.float64) - 127), 32, 1)
    h = mx4.dequantize(g["H"], g["H_scale"], I)
    assert ((mx4.grid((ref - tol) / unit) <= h / unit) & (h / unit <= mx4.grid((ref + tol) / unit))).all()
    y, _, my = mx4.expert_product(h, w2, g["offsets"], rows=np.arange(len(h)))
    assert (np.abs(g["Y"] - y) <= (128 + I // 64 + 16) * 2.0 ** -23 * my).all()


@pytest.mark.parametrize("T", [3, 300])
def test_layer_replayed(mx, T):
    say(f"case: layer on MXFP4 rows, captured and replayed, T={T}")
    s, w, x = setup(mx, MID, T)
    moe = mx.LatentMoE(s, w, DEV, mxfp4_rows=True)
    want = {k: v.clone() for k, v in moe.forward(x).items()}
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    b = moe.forward(x, stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        moe.forward(x, stream)
    for _ in range(3):
        for k in ("out", "Y", "H", "zq"):
            b[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b[k], want[k]) for k in ("out", "Y", "H", "H_scale", "zq", "zq_scale"))
        moe.forward(x)
        torch.cuda.synchronize()
        assert torch.equal(b["out"], want["out"])


def test_refusals(mx):
    s, w, x = setup(mx, TINY, 4)
    bank_b = {"format": 0, "n_experts": 8, **{k: w[k][24:] for k in w if k[:2] in ("w1", "w3", "w2")}}
    with pytest.raises(ValueError):
        mx.LatentMoE(s, w, DEV, bank_b=bank_b, mxfp4_rows=True)
    with pytest.raises(ValueError):
        mx.LatentMoE(s, w, DEV, mxfp4_rows=True).forward_few(x)
