"""The layer on MXFP4 rows where its experts' products go through lists of chunks: gate and up by tiles and by streamed
experts into MXFP4 hidden rows, which the down product takes through its own list.

Every step against float64 from the step before's own output, with the bounds of test_gpu_mx4_layer.py.
"""
import numpy as np
import pytest
import torch

import synth
from gpu_common import say
from synth.device import to_dev_bf16, upload_weights
from test_gpu_mx4_direct import fit_byte, grid, values

pytestmark = pytest.mark.gpu
DEV = "cuda"
# test_mx4_expert_plan_host.py: both products through lists; below 32 rows an expert on average experts of up to 16
# rows are streamed, from there tiles take all
WIDE = synth.LayerShape(512, 1024, 128, 4, 1024, 1, 256)
BOTH, TILES = 900, 1200


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as m
    m.load()
    return m


@pytest.mark.parametrize("T", [BOTH, TILES])
def test_layer(mx, T):
    say(f"case: layer on MXFP4 rows through lists, T={T}")
    # experts of none, of few and of many rows
    wl = synth.Workload(f"rows4_lists_{T}", 29, WIDE, T, 29, 0.02, 0.05, "normal", 119, 121)
    w, x, s = upload_weights(wl, DEV), to_dev_bf16(synth.gen_tokens(wl), DEV), mx.shape_of(WIDE)
    moe = mx.LatentMoE(s, w, DEV, mxfp4_rows=True)
    b = {k: v.clone() for k, v in moe.forward(x).items()}
    again = moe.forward(x)
    torch.cuda.synchronize()
    assert all(torch.equal(b[k], again[k]) for k in ("zq", "zq_scale", "H", "H_scale", "Y", "out"))
    counts = np.diff(b["offsets"].cpu().numpy())
    assert ((0 < counts) & (counts <= 16)).any() and counts.min() == 0 and counts.max() > 128 and counts.sum() == 4 * T
    L, I = s.latent, s.inter  # noqa: E741
    z, h = values(b["zq"], b["zq_scale"]), values(b["H"], b["H_scale"])
    eps = (128 + L // 64 + 16) * 2.0 ** -23
    at = 0
    for e, n in enumerate(counts.tolist()):
        r = slice(at, at + n)
        at += n
        w1, w3, w2 = (values(w[m + "_packed"][e], w[m + "_scale"][e]).T.contiguous() for m in ("w1", "w3", "w2"))
        a = z[b["sorted_pair"][r].long() // s.top_k]
        gate, up, mg, mu = a @ w1, a @ w3, a.abs() @ w1.abs(), a.abs() @ w3.abs()
        ref = 4 * torch.tanh(gate / 4) * torch.sigmoid(gate) * 25 * torch.tanh(up / 25)
        tol = ref.abs() * (32 + gate.abs()) * 2.0 ** -23 + eps * (1.2 * mg * up.abs() + mu * gate.abs()) + 1e-37
        hs = b["H_scale"][r]
        lo, hi = (fit_byte((ref.abs() + d * tol).clamp_min(0).unflatten(1, (-1, 32)).amax(2)) for d in (-1, 1))
        assert ((lo <= hs) & (hs <= hi)).all(), e
        unit = torch.exp2(hs.double() - 127).repeat_interleave(32, 1)
        assert ((grid((ref - tol) / unit) <= h[r] / unit) & (h[r] / unit <= grid((ref + tol) / unit))).all(), e
        y, my = h[r] @ w2, h[r].abs() @ w2.abs()
        assert ((b["Y"][r].double() - y).abs() <= (128 + I // 64 + 16) * 2.0 ** -23 * my).all(), e
