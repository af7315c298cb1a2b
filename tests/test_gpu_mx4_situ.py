"""SiTU-GLU of the expert products on MXFP4 rows over the whole range of its betas, against float64.

The bound is test_gpu_mx4.py's, (32 + |g|) 2^-23 of the value, and what is lost where g / beta or the numerator of its
tanh, 2^-9 of it, is below fp32's normal numbers: each is rounded by at most 2^-150 there, together 1.01 2^-150 of a
numerator whose denominator is at least 2^-9, so beta tanh(g / beta) is off by beta 1.01 2^-141, of u's alike.
"""
import numpy as np
import pytest
import torch

from gpu_common import say
from oracle import mx4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as mx
    mx.load()
    return mx


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def glu(mx, x, xs, w, ws, w3, ws3, beta, beta_lin):
    """One expert's gate and up in fp32."""
    P, N, K = len(x), w.shape[0], 2 * w.shape[1]
    out = torch.empty((P, N), device=DEV)
    scratch = torch.empty(mx.mxfp4_expert_gemm_workspace_bytes(1, P, N, K), dtype=torch.uint8, device=DEV)
    mx.mxfp4_expert_gemm(dev(x), dev(xs), dev(w[None]), dev(ws[None]), dev(np.array([0, P], np.int32)), out, scratch,
                         w3=dev(w3[None]), w3_scale=dev(ws3[None]), beta=beta, beta_lin=beta_lin)
    return out.cpu().numpy().astype(np.float64)


# by waves that stream, and wide enough for tiles
SIZES = [(5, 64), (260, 16384)]
BETAS = [(4.0, 25.0), (1e20, 1e20), (2.0 ** 100, 2.0 ** 100), (1e30, 25.0), (4.0, 1e30), (2.0 ** -100, 2.0 ** -100),
         (2.0 ** -100, 2.0 ** 100), (1e-20, 1e-20)]


@pytest.mark.parametrize("P,N", SIZES)
@pytest.mark.parametrize("beta,beta_lin", BETAS)
def test_betas(mx, P, N, beta, beta_lin):
    say(f"case: SiTU-GLU, {P} rows, {N} columns, betas {beta} and {beta_lin}")
    K = 64
    rng = np.random.default_rng(N)
    x, xs = rng.integers(0, 256, (P, K // 2)).astype(np.uint8), rng.integers(126, 128, (P, K // 32)).astype(np.uint8)
    w, w3 = (rng.integers(0, 256, (N, K // 2)).astype(np.uint8) for _ in range(2))
    ws, ws3 = (rng.integers(121, 123, (N, K // 32)).astype(np.uint8) for _ in range(2))
    got = glu(mx, x, xs, w, ws, w3, ws3, beta, beta_lin)
    a = mx4.dequantize(x, xs, K)
    g, u = a @ mx4.dequantize(w, ws, K).T, a @ mx4.dequantize(w3, ws3, K).T
    b, bl = float(np.float32(beta)), float(np.float32(beta_lin))
    ref = mx4.situ_glu(g, u, b, bl)
    lost = 2.0 ** -140 * (b * np.minimum(np.abs(u), bl) + bl * np.minimum(1.1 * np.abs(g), b))
    assert (np.abs(got - ref) <= np.abs(ref) * (32 + np.abs(g)) * 2.0 ** -23 + lost + 1e-37).all()


@pytest.mark.parametrize("P,N", SIZES)
def test_large_products_with_large_betas(mx, P, N):
    """g u past fp32's range: 0 where the gate is far below zero, infinite where it is far above."""
    say(f"case: SiTU-GLU of products of 2^70, {P} rows, {N} columns")
    K = 32
    x, xs = np.full((P, K // 2), 0x22, np.uint8), np.full((P, 1), 127, np.uint8)  # ones
    sign = np.where(np.arange(N) % 2, 0x22, 0xAA).astype(np.uint8)[:, None]  # -1 in even columns
    w, ws = np.repeat(sign, K // 2, 1), np.full((N, 1), 127 + 65, np.uint8)
    w3 = np.full((N, K // 2), 0x22, np.uint8)
    got = glu(mx, x, xs, w, ws, w3, ws, 2.0 ** 100, 2.0 ** 100)
    assert (got[:, 0::2] == 0).all() and (got[:, 1::2] == np.inf).all()
