"""MXFP4 rows and the products with both operands in MXFP4, against float64 (oracle/mx4.py).

Quantisation is exact arithmetic and one rounding: codes and scale bytes are
the oracle's.  Products: with scales of two neighbouring binades on each side
every product is a multiple of 2^-3 times a common factor and magnitudes stay
below 36 * 4 K / 2^-3 = 1152 K < 2^24 of them (K <= 14000), so every sum is
exact in fp32 in any order, and results are the exact ones, rounded once to
bf16 where asked.  With scales far apart a sum is off by at most 2^-23 of the
sum of magnitudes (twice a rounding, as the matrix units may truncate) for each
addition: 128 in an instruction, K / 64 instructions, 16 joins.

SiTU-GLU of exact products g, u: each tanh's argument, its 2.4e-7 and its share
of the one division are under 6 * 2^-23 relative; sigmoid's exponential errs by
|g| / 2 * 2^-23 through its argument and 3 * 2^-23 else; four products and a
reciprocal 5 * 2^-23: together under (32 + |g|) 2^-23 of the value.
"""
import numpy as np
import pytest
import torch

from gpu_common import say
from oracle import mx4

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BF = 2.0 ** -8


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as mx
    mx.load()
    return mx


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ---- quantisation

@pytest.mark.parametrize("rule", ["fit", "ocp"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,pad", [(1, 1, 0), (1, 32, 0), (3, 33, 0), (2, 45, 3), (5, 64, 8), (7, 1000, 0),
                                     (70, 257, 1), (33, 3584, 0), (16, 7168, 16), (1, 33792, 0), (300, 96, 32)])
def test_quantize(mx, T, K, pad, kind, rule):
    say(f"case: quantise T={T} K={K} pad {pad} {kind} {rule}")
    g = torch.Generator().manual_seed(T + K)
    x = (torch.randn(T, K + pad, generator=g) * torch.exp(2 * torch.randn(K + pad, generator=g))).to(DT[kind])
    x[0, :K:3] = 0.0
    q = torch.full((T, -(-K // 2) + pad), 0xEE, dtype=torch.uint8, device=DEV)
    s = torch.full((T, -(-K // 32) + pad), 0xEE, dtype=torch.uint8, device=DEV)
    nq, ns = -(-K // 2), -(-K // 32)
    mx.mxfp4_quantize(x.to(DEV)[:, :K], q[:, :nq], s[:, :ns], rule=rule)
    wq, ws = mx4.quantize(f64(x)[:, :K], rule)
    assert (s[:, :ns].cpu().numpy() == ws).all() and (q[:, :nq].cpu().numpy() == wq).all()
    assert (q[:, nq:] == 0xEE).all() and (s[:, ns:] == 0xEE).all()
    for dt in DT.values():
        out = torch.full((T, K + pad), 3.0, dtype=dt, device=DEV)
        mx.mxfp4_dequantize(q[:, :nq], s[:, :ns], out[:, :K])
        assert (f64(out)[:, :K] == mx4.dequantize(wq, ws, K)).all() and (out[:, K:] == 3.0).all()


def test_quantize_every_border(mx):
    """Values at, just below and just above every border between codes, in blocks of every scale byte."""
    say("case: quantise at the borders of every scale")
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    v = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9))])
    v = np.concatenate([v, -v]).astype(np.float32)  # 48 values: two blocks of 24, their maxima above 6 and at 6
    rows = []
    for e in range(-125, 126):
        a = np.zeros((2, 32), np.float32)
        a[0, :24], a[1, :24] = v[:24], v[24:]
        a[0, 24], a[1, 24] = 6.0, 4.0
        with np.errstate(all="ignore"):
            rows.append(np.ldexp(np.clip(a, -6, 6), e).astype(np.float32))
    x = np.stack(rows).reshape(-1, 32)
    x = np.concatenate([x, np.ldexp(x[:2], 0) * 1.3, np.full((1, 32), 3.0e38, np.float32), np.zeros((1, 32), np.float32)])
    for rule in ("fit", "ocp"):
        q = torch.empty((len(x), 16), dtype=torch.uint8, device=DEV)
        s = torch.empty((len(x), 1), dtype=torch.uint8, device=DEV)
        mx.mxfp4_quantize(dev(x), q, s, rule=rule)
        wq, ws = mx4.quantize(x.astype(np.float64), rule)
        assert (s.cpu().numpy() == ws).all()
        assert (q.cpu().numpy() == wq).all()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("K", [64, 70])
def test_quantize_not_finite(mx, K, bad):
    """Such a value spoils its own block and no other; the row's results in a product are NaN."""
    x = np.random.default_rng(0).normal(size=(4, K)).astype(np.float32)
    x[1, 33] = bad
    q = torch.empty((4, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((4, -(-K // 32)), dtype=torch.uint8, device=DEV)
    mx.mxfp4_quantize(dev(x), q, s)
    wq, ws = mx4.quantize(x.astype(np.float64))
    assert ws[1, 1] == 255 and (s.cpu().numpy() == ws).all() and (q.cpu().numpy() == wq).all()
    out = torch.empty((4, K), device=DEV)
    mx.mxfp4_dequantize(q, s, out)
    nan = np.zeros((4, K), bool)
    nan[1, 32:64] = True
    assert (np.isnan(f64(out)) == nan).all()


def test_dequantize_every_byte(mx):
    """Every pair of codes under every scale byte, exact in fp32 and bf16 where they hold it."""
    q = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1))
    s = np.repeat(np.arange(256, dtype=np.uint8), 16)[:, None]
    want = mx4.dequantize(q, s, 32)
    for dt in DT.values():
        out = torch.empty((4096, 32), dtype=dt, device=DEV)
        mx.mxfp4_dequantize(dev(q), dev(s), out)
        got = f64(out)
        with np.errstate(over="ignore"):
            w = torch.from_numpy(want).to(dt).double().numpy()
        assert ((got == w) | (np.isnan(got) & np.isnan(w))).all()


# ---- products

def operands(rng, rows, N, K, E=1, spread=2, pad=0, mats=1):
    """Random codes; scales of `spread` binades around 1 (rows) and 2^-4 (weights).  Rows strided by K / 2 + pad, their
    scales by K / 32 + 3, with NaN scales beside them."""
    x = rng.integers(0, 256, (rows, K // 2 + pad)).astype(np.uint8)
    xs = rng.integers(127, 127 + spread, (rows, K // 32 + 3)).astype(np.uint8)
    xs[:, K // 32:] = 255
    w = [(rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8),
          rng.integers(123, 123 + spread, (E, N, K // 32)).astype(np.uint8)) for _ in range(mats)]
    return x, xs, w


def product(mx, T, N, K, out_kind, seed=0, pad=0, opad=0, accumulate=False, spread=2):
    rng = np.random.default_rng(seed)
    x, xs, [(w, ws)] = operands(rng, T, N, K, spread=spread, pad=pad)
    dx, dxs = dev(x)[:, :K // 2], dev(xs)[:, :K // 32]
    out = torch.full((T, N + opad), 3.0, dtype=DT[out_kind], device=DEV)
    scratch = torch.full((mx.mxfp4_gemm_workspace_bytes(T, N, K),), 0xFF, dtype=torch.uint8, device=DEV)
    dw, dws = dev(w[0]), dev(ws[0])
    mx.mxfp4_gemm(dx, dxs, dw, dws, out[:, :N], scratch, accumulate=accumulate)
    again = torch.full_like(out, 3.0)
    mx.mxfp4_gemm(dx, dxs, dw, dws, again[:, :N], scratch, accumulate=accumulate)
    assert torch.equal(out, again) and (out[:, N:] == 3.0).all()
    a, b = mx4.dequantize(x[:, :K // 2], xs[:, :K // 32], K), mx4.dequantize(w[0], ws[0], K)
    ref = a @ b.T + (3.0 if accumulate else 0.0)
    got = f64(out)[:, :N]
    if spread == 2:
        assert torch.equal(out[:, :N].cpu(), torch.from_numpy(ref).to(DT[out_kind]))
        return
    tol = (128 + K // 64 + 16) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T + 3.0)
    assert (np.abs(got - ref) <= tol + (BF * (np.abs(ref) + tol) if out_kind == "bf16" else 0)).all()
    if out_kind == "f32" and T * N >= 1000 and not accumulate:
        # as fp32 sums in the mean, not only at worst: twice what adding in order in fp32 measured
        assert np.sqrt(np.mean((got - ref) ** 2) / np.mean(ref ** 2)) < 2e-6


# rows on both sides of every tile, columns and K that end inside one, K of one block to long
SIZES = [(1, 1, 32), (1, 16, 128), (2, 17, 160), (15, 130, 1056), (16, 128, 2048), (17, 257, 256), (31, 64, 4128),
         (33, 100, 384), (64, 255, 640), (65, 384, 416), (97, 129, 288), (129, 513, 1152), (255, 895, 1024),
         (257, 256, 128), (300, 640, 3616), (700, 1100, 544), (70, 130, 13984), (7, 6150, 416), (16, 6145, 4128),
         (9, 50, 4128), (1, 300, 5024), (50, 900, 4128), (41, 4200, 4128), (513, 33, 96), (1, 3584, 7168),
         (301, 895, 7168), (1500, 2100, 256), (5, 31, 512), (260, 40, 544)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_product(mx, T, N, K):
    out = "bf16" if (T + N) % 2 else "f32"
    say(f"case: 4-bit product T={T} N={N} K={K} out {out}")
    product(mx, T, N, K, out, seed=T + N + K)


@pytest.mark.parametrize("T,N,K", [(3, 100, 416), (40, 129, 288), (200, 200, 512), (520, 384, 1152), (130, 257, 4096)])
def test_strides_and_accumulate(mx, T, N, K):
    for opad in (1, 4):
        say(f"case: 4-bit product, strided rows, added to: T={T} N={N} K={K} out pad {opad}")
        product(mx, T, N, K, "f32", seed=1, pad=16, opad=opad, accumulate=True)
        product(mx, T, N, K, "bf16", seed=2, pad=32, opad=opad)


@pytest.mark.parametrize("T,N,K", [(1, 1000, 7168), (16, 200, 7168), (60, 300, 1056), (130, 257, 544), (301, 895, 7168)])
def test_scales_far_apart(mx, T, N, K):
    for out in DT:
        say(f"case: 4-bit product, scales far apart, T={T} N={N} K={K} out {out}")
        product(mx, T, N, K, out, seed=3, spread=20)


@pytest.mark.parametrize("T,N,K", [(5, 260, 672), (300, 260, 672), (130, 700, 4096)])
def test_nan_stays_in_its_row_and_column(mx, T, N, K):
    say(f"case: 4-bit product with NaN scales, T={T} N={N} K={K}")
    rng = np.random.default_rng(3)
    x, xs, [(w, ws)] = operands(rng, T, N, K)
    d = [dev(v) for v in (x, xs[:, :K // 32], w[0], ws[0])]
    scratch = torch.empty(mx.mxfp4_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    clean, out = torch.empty((T, N), device=DEV), torch.empty((T, N), device=DEV)
    mx.mxfp4_gemm(*d, clean, scratch)
    d[1][2, K // 32 - 1] = 255
    d[3][255, 3] = 255
    mx.mxfp4_gemm(*d, out, scratch)
    bad = torch.zeros((T, N), dtype=torch.bool, device=DEV)
    bad[2] = True
    bad[:, 255] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("T", [3, 300])
def test_scale_bytes_at_their_ends(mx, T):
    """Row scale bytes 0 and 254 against weight scales that bring them back: as the formula has them."""
    N, K = 64, 256
    x, xs, [(w, ws)] = operands(np.random.default_rng(5), T, N, K)
    xs, ws = xs[:, :K // 32].copy(), ws[0]
    for lo, hi in ((0, 250), (254, 4), (2, 250), (253, 4)):
        say(f"case: 4-bit product, scale bytes {lo} and {hi}, T={T}")
        xs[:], ws[:] = lo, hi
        out = torch.empty((T, N), device=DEV)
        scratch = torch.empty(mx.mxfp4_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
        mx.mxfp4_gemm(dev(x), dev(xs), dev(w[0]), dev(ws), out, scratch)
        ref = mx4.dequantize(x, xs, K) @ mx4.dequantize(w[0], ws, K).T
        assert (f64(out) == ref).all()


@pytest.mark.parametrize("T", [1, 16, 64, 384, 1024])
def test_full_sizes(mx, T):
    """Sizes of the layer's dense products; a sample of the outputs, exact."""
    N, K = 3584, 7168
    say(f"case: 4-bit product at T={T} N={N} K={K}")
    x, xs, [(w, ws)] = operands(np.random.default_rng(T), T, N, K)
    out = torch.empty((T, N), device=DEV)
    scratch = torch.empty(mx.mxfp4_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    mx.mxfp4_gemm(dev(x), dev(xs)[:, :K // 32], dev(w[0]), dev(ws[0]), out, scratch)
    ts = np.unique(np.concatenate([[0, T - 1], np.random.default_rng(0).integers(0, T, 6)]))
    ref = mx4.dequantize(x[ts], xs[ts, :K // 32], K) @ mx4.dequantize(w[0], ws[0], K).T
    assert (f64(out)[ts] == ref).all()


# whole tiles of every height, a round of the largest with lower ones behind it, K in parts: test_mx4_plan_host.py
# holds the plan to that
LARGE = [(301, 895, 7168), (512, 3584, 7168), (1500, 2100, 256), (2900, 4400, 1056), (4100, 6200, 768),
         (3000, 6600, 1536), (4096, 4096, 4096)]


@pytest.mark.parametrize("T,N,K", LARGE)
def test_tiles(mx, T, N, K):
    """Every result, against the same product in float64 on the GPU (exact there as here)."""
    for out_kind, opad in (("f32", 0), ("bf16", 8), ("bf16", 4), ("bf16", 1)):
        say(f"case: 4-bit product by tiles T={T} N={N} K={K} out {out_kind} pad {opad}")
        x, xs, [(w, ws)] = operands(np.random.default_rng(T), T, N, K)
        out = torch.full((T, N + opad), 3.0, dtype=DT[out_kind], device=DEV)
        scratch = torch.full((mx.mxfp4_gemm_workspace_bytes(T, N, K),), 0xFF, dtype=torch.uint8, device=DEV)
        mx.mxfp4_gemm(dev(x), dev(xs)[:, :K // 32], dev(w[0]), dev(ws[0]), out[:, :N], scratch)
        a, b = dev(mx4.dequantize(x, xs[:, :K // 32], K)), dev(mx4.dequantize(w[0], ws[0], K).T)
        assert torch.equal(out[:, :N], (a @ b).to(DT[out_kind])) and (out[:, N:] == 3.0).all()


# ---- expert products

def routing(rng, counts, tokens, top_k, spare):
    """Offsets of the given rows an expert, and a pair for each sorted row: P = sum(counts) + spare rows."""
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    P = int(offsets[-1]) + spare
    return offsets, rng.integers(0, tokens * top_k, P).astype(np.int32), P


def expert(mx, counts, N, K, glu, out_kind, tokens=0, top_k=0, weights=False, spare=0, pad=0, opad=0, seed=0):
    """One call against the oracle: gathered rows with top_k > 0, sorted ones else."""
    rng = np.random.default_rng(seed)
    E, pairs = len(counts), max(1, tokens) * max(1, top_k)
    offsets, pair, P = routing(rng, counts, max(1, tokens), max(1, top_k), spare)
    rows = tokens if top_k else P
    x, xs, mats = operands(rng, max(1, rows), N, K, E=E, pad=pad, mats=2 if glu else 1)
    x, xs = x[:rows], xs[:rows]
    if glu:  # products of a few units, where SiTU-GLU bends
        for _, s in mats:
            s -= 6
    pw = rng.random(pairs).astype(np.float32) if weights else None
    kw = dict(sorted_pair=dev(pair), top_k=top_k) if top_k or weights else {}
    if glu:
        kw |= dict(w3=dev(mats[1][0]), w3_scale=dev(mats[1][1]))
    if weights:
        kw["pair_weight"] = dev(pw)
    four = out_kind == "mx4"
    cols = N // 2 if four else N
    out = torch.full((P, cols + opad), 0xEE if four else 3.0, dtype=torch.uint8 if four else DT[out_kind], device=DEV)
    sc = torch.full((P, N // 32 + opad), 0xEE, dtype=torch.uint8, device=DEV) if four else None
    scratch = torch.full((mx.mxfp4_expert_gemm_workspace_bytes(E, P, N, K),), 0xFF, dtype=torch.uint8, device=DEV)
    if four:
        kw["out_scale"] = sc[:, :N // 32]
    mx.mxfp4_expert_gemm(dev(x)[:, :K // 2], dev(xs)[:, :K // 32], dev(mats[0][0]), dev(mats[0][1]), dev(offsets),
                         out[:, :cols], scratch, **kw)
    src = pair // top_k if top_k else np.arange(P)
    a = mx4.dequantize(x[:, :K // 2], xs[:, :K // 32], K)
    w = [mx4.dequantize(q, s, K) for q, s in mats]
    ref, gate, _ = mx4.expert_product(a, w[0], offsets, w[1] if glu else None, src,
                                      None if pw is None else pw[pair].astype(np.float64))
    end = offsets[-1]
    untouched = (out[end:] == (0xEE if four else 3.0)).all() and (out[:, cols:] == (0xEE if four else 3.0)).all()
    assert untouched and (not four or ((sc[end:] == 0xEE).all() and (sc[:, N // 32:] == 0xEE).all()))
    ref, gate = ref[:end], gate[:end]
    if not end:
        return
    tol = np.abs(ref) * (32 + np.abs(gate)) * 2.0 ** -23 + 1e-37 if glu else np.abs(ref) * (2.0 ** -24 if weights else 0)
    if four:
        q, s = out[:end, :cols].cpu().numpy(), sc[:end, :N // 32].cpu().numpy()
        lo, hi = (mx4.scale_exponent(np.maximum(np.abs(ref) + d * tol, 0).reshape(end, -1, 32).max(2), "fit") + 127
                  for d in (-1, 1))
        assert ((lo <= s) & (s <= hi)).all()
        unit = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, 1)
        v = mx4.dequantize(q, s, N) / unit
        assert ((mx4.grid((ref - tol) / unit) <= v) & (v <= mx4.grid((ref + tol) / unit))).all()
        return
    got = f64(out)[:end, :N]
    assert (np.abs(got - ref) <= tol + (BF * (np.abs(ref) + tol) if out_kind == "bf16" else 0)).all()
    if not glu and not weights:
        assert torch.equal(out[:end, :N].cpu(), torch.from_numpy(ref).to(DT[out_kind]))


COUNTS = [[1], [0, 3, 0], [5, 0, 1, 17, 0, 2], [0, 0, 0], [64, 65, 1, 0, 33], [130, 0, 257, 16], [300], [1] * 70 + [40],
          [31, 32, 33, 0, 96, 97, 128, 129, 160, 161]]


@pytest.mark.parametrize("N,K", [(32, 32), (128, 128), (96, 416), (288, 1056), (160, 576)])
@pytest.mark.parametrize("counts", COUNTS, ids=[str(i) for i in range(len(COUNTS))])
def test_expert_glu(mx, counts, N, K):
    for out in ("f32", "bf16", "mx4"):
        say(f"case: expert gate and up, rows {counts[:8]} N={N} K={K} out {out}")
        expert(mx, counts, N, K, True, out, tokens=37, top_k=3, spare=2, seed=N + K)
    expert(mx, counts, N, K, True, "mx4", pad=16, opad=16, spare=1, seed=K)  # sorted rows


@pytest.mark.parametrize("N,K", [(1, 32), (130, 128), (257, 416), (64, 1056)])
@pytest.mark.parametrize("counts", COUNTS, ids=[str(i) for i in range(len(COUNTS))])
def test_expert_down(mx, counts, N, K):
    for out in DT:
        say(f"case: expert down, rows {counts[:8]} N={N} K={K} out {out}")
        expert(mx, counts, N, K, False, out, spare=3, pad=16, opad=1, seed=N + K)
        expert(mx, counts, N, K, False, out, tokens=50, top_k=2, weights=True, spare=1, seed=N)
        expert(mx, counts, N, K, False, out, tokens=50, weights=True, opad=4, seed=N)


def test_expert_odd_columns(mx):
    say("case: expert gate and up, odd columns")
    for out in DT:
        expert(mx, [5, 0, 70], 77, 160, True, out, tokens=9, top_k=2, opad=3)


@pytest.mark.parametrize("counts", [[1, 400, 0, 17, 2, 300], [1] * 12 + [0, 200, 16, 65, 17, 3, 0, 129, 2, 33, 0, 1]])
def test_expert_lists(mx, counts):
    """Wide enough for lists of chunks: tiles alone, and both kernels."""
    expert(mx, counts, 4160, 64, True, "mx4", tokens=50, top_k=3, seed=3)
    expert(mx, counts, 4161, 64, True, "f32", tokens=50, top_k=3, seed=4, spare=5)
    expert(mx, counts, 8323, 96, False, "bf16", seed=5, opad=5)
    expert(mx, counts, 8320, 544, False, "f32", weights=True, seed=6, spare=70)


def test_expert_many_experts(mx):
    rng = np.random.default_rng(8)
    counts = rng.permutation(np.concatenate([np.zeros(800, int), rng.integers(1, 5, 200), [70] * 24]))
    say("case: expert products, 1024 experts")
    expert(mx, counts.tolist(), 64, 128, True, "mx4", tokens=100, top_k=4, seed=1)
    expert(mx, counts.tolist(), 96, 64, False, "f32", seed=2)


@pytest.mark.parametrize("counts", [[1, 0, 2, 0, 1, 1], [74, 0, 73, 75], [292, 290]])
def test_expert_full_sizes(mx, counts):
    """The routed experts' own sizes; sampled rows."""
    L, I, k = 3584, 3072, 4  # noqa: E741
    rng = np.random.default_rng(2)
    E = len(counts)
    offsets, pair, P = routing(rng, counts, 20, k, 0)
    say(f"case: expert gate and up, then down, at full size, rows {counts}")
    z, zs, mats = operands(rng, 20, I, L, E=E, mats=2)
    for _, s in mats:
        s -= 7
    h, hs = (torch.empty((P, n), dtype=torch.uint8, device=DEV) for n in (I // 2, I // 32))
    scratch = torch.empty(max(mx.mxfp4_expert_gemm_workspace_bytes(E, P, I, L),
                              mx.mxfp4_expert_gemm_workspace_bytes(E, P, L, I)), dtype=torch.uint8, device=DEV)
    f = torch.empty((P, I), device=DEV)
    d = [dev(v) for q in mats for v in q]
    args = dict(w3=d[2], w3_scale=d[3], sorted_pair=dev(pair), top_k=k)
    for out, more in ((f, {}), (h, {"out_scale": hs})):
        mx.mxfp4_expert_gemm(dev(z), dev(zs)[:, :L // 32], d[0], d[1], dev(offsets), out, scratch, **args, **more)
    ps = np.unique(np.concatenate([[0, P - 1], rng.integers(0, P, 10)]))
    a = mx4.dequantize(z, zs[:, :L // 32], L)[pair[ps] // k]
    e = np.searchsorted(offsets, ps, side="right") - 1
    g, u = (np.stack([a[i] @ mx4.dequantize(q[e[i]], s[e[i]], L).T for i in range(len(ps))]) for q, s in mats)
    ref = mx4.situ_glu(g, u)
    assert (np.abs(f64(f)[ps] - ref) <= np.abs(ref) * (32 + np.abs(g)) * 2.0 ** -23 + 1e-37).all()
    # the 4-bit rows are those of the fp32 ones
    wq, wsc = torch.empty_like(h), torch.empty_like(hs)
    mx.mxfp4_quantize(f, wq, wsc)
    assert torch.equal(h, wq) and torch.equal(hs, wsc)
    _, _, [(w2, s2)] = operands(rng, 1, L, I, E=E)
    y = torch.empty((P, L), device=DEV)
    mx.mxfp4_expert_gemm(h, hs, dev(w2), dev(s2), dev(offsets), y, scratch)
    hv = mx4.dequantize(h.cpu().numpy()[ps], hs.cpu().numpy()[ps], I)
    w = [mx4.dequantize(w2[i], s2[i], I) for i in e]
    ref = np.stack([hv[i] @ w[i].T for i in range(len(ps))])
    mag = np.stack([np.abs(hv[i]) @ np.abs(w[i]).T for i in range(len(ps))])
    assert (np.abs(f64(y)[ps] - ref) <= (128 + I // 64 + 16) * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("rows,N", [(3, 64), (70, 64), (300, 16384)])
def test_expert_glu_not_finite(mx, rows, N):
    """Products that are infinite or NaN, by waves that stream and by tiles: SiTU-GLU's limits."""
    say(f"case: SiTU-GLU of infinite products, {rows} rows, {N} columns")
    K, T = 32, rows
    x, xs = np.full((T, K // 2), 0x22, np.uint8), np.full((T, 1), 127, np.uint8)  # ones
    # value and scale byte of a row's codes: 32 * 6 * 2^127 and NaN, else 16 and 2
    kinds = {"inf": (0x77, 254), "-inf": (0xFF, 254), "nan": (0x22, 255), "16": (0x11, 127), "-2": (0x99, 124)}
    pairs = [(a, b) for a in kinds for b in kinds]
    at = np.arange(N) % len(pairs)
    w = [np.stack([np.full(K // 2, kinds[pairs[i][m]][0], np.uint8) for i in at])[None] for m in range(2)]
    s = [np.array([[kinds[pairs[i][m]][1]] for i in at], np.uint8)[None] for m in range(2)]
    with np.errstate(invalid="ignore"):
        value = [np.array([float(pairs[i][m]) for i in at]) for m in range(2)]
        g, u = value
        ref = 4 * np.tanh(g / 4) * 25 * np.tanh(u / 25) * np.where(g == -np.inf, 0, 1 / (1 + np.exp(-np.maximum(g, -700))))
    out = torch.empty((T, N), device=DEV)
    scratch = torch.empty(mx.mxfp4_expert_gemm_workspace_bytes(1, T, N, K), dtype=torch.uint8, device=DEV)
    mx.mxfp4_expert_gemm(dev(x), dev(xs), dev(w[0]), dev(s[0]), dev(np.array([0, T], np.int32)), out, scratch,
                         w3=dev(w[1]), w3_scale=dev(s[1]), sorted_pair=dev(np.arange(T, dtype=np.int32)), top_k=1)
    got = f64(out)
    assert (np.isnan(got) == np.isnan(ref)).all()
    ok = ~np.isnan(ref)
    assert (np.abs(got[:, ok] - ref[ok]) <= np.abs(ref[ok]) * (32 + 16) * 2.0 ** -23).all()


def test_streams_and_replays(mx):
    """Two calls at once with a workspace each; two captured calls that share one, replayed in turn with eager work in
    between, every replay the eager result."""
    for counts in ([2, 0, 1, 3], [200, 0, 90, 300]):
        say(f"case: 4-bit products on two streams and replayed, rows {counts}")
        N, K = 256, 640
        calls, want, out, scratch = [], [], [], []
        for seed in (1, 2):
            rng = np.random.default_rng(seed)
            offsets, pair, P = routing(rng, counts, 60, 3, 0)
            x, xs, mats = operands(rng, 60, N, K, E=len(counts), mats=2)
            d = [dev(v) for v in (x, xs[:, :K // 32], mats[0][0], mats[0][1], offsets, mats[1][0], mats[1][1], pair)]
            out.append((torch.empty((P, N), device=DEV), torch.empty((60, N), device=DEV)))
            want.append(tuple(torch.empty_like(o) for o in out[-1]))
            scratch.append(torch.empty(max(mx.mxfp4_expert_gemm_workspace_bytes(len(counts), P, N, K),
                                           mx.mxfp4_gemm_workspace_bytes(60, N, K)), dtype=torch.uint8, device=DEV))

            def call(o, ws, stream=None, d=d):
                mx.mxfp4_expert_gemm(*d[:5], o[0], ws, w3=d[5], w3_scale=d[6], sorted_pair=d[7], top_k=3, stream=stream)
                mx.mxfp4_gemm(d[0], d[1], d[2][0], d[3][0], o[1], ws, stream=stream)
            calls.append(call)
            call(want[-1], scratch[-1])
        torch.cuda.synchronize()
        same = lambda: all(torch.equal(a, b) for o, w in zip(out, want) for a, b in zip(o, w))  # noqa: E731
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(10):
            for i in range(2):
                calls[i](out[i], scratch[i], streams[i])
        torch.cuda.synchronize()
        assert same()
        graphs = []
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                calls[i](out[i], scratch[0])
            graphs.append(g)
        for _ in range(3):
            for i in range(2):
                for o in out[i]:
                    o.zero_()
                graphs[i].replay()
                calls[1](want[1], scratch[0])
            torch.cuda.synchronize()
            assert same()


def test_refusals(mx):
    T, N, K, E = 4, 64, 128, 3
    x, xs, [(w, ws), (w3, ws3)] = operands(np.random.default_rng(0), T, N, K, E=E, mats=2)
    dx, dxs, dw, dws, dw3, dws3 = (dev(v) for v in (x, xs[:, :K // 32], w, ws, w3, ws3))
    out, off = torch.empty((T, N), device=DEV), dev(np.array([0, 1, 2, 4], np.int32))
    q, s = torch.empty((T, N // 2), dtype=torch.uint8, device=DEV), torch.empty((T, N // 32), dtype=torch.uint8, device=DEV)
    sp = dev(np.arange(T, dtype=np.int32))
    big = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    f = torch.zeros((T, K), device=DEV)
    mx.mxfp4_quantize(f[:0], dx[:0], dxs[:0])
    mx.mxfp4_dequantize(dx[:0], dxs[:0], f[:0])
    mx.mxfp4_gemm(dx[:0], dxs[:0], dw[0], dws[0], out[:0], big)
    mx.mxfp4_expert_gemm(dx[:0], dxs[:0], dw, dws, off, out[:0], big)
    bad = [
        lambda: mx.mxfp4_quantize(f, dx, dxs, rule="best"),
        lambda: mx.mxfp4_quantize(f.half(), dx, dxs),
        lambda: mx.mxfp4_quantize(f, dx[:, :63], dxs),
        lambda: mx.mxfp4_quantize(f, dx, dxs[:, :3]),
        lambda: mx.mxfp4_quantize(f.cpu(), dx, dxs),
        lambda: mx.mxfp4_dequantize(dx, dxs, f.half()),
        lambda: mx.mxfp4_dequantize(dx, dxs[:3], f),
        lambda: mx.mxfp4_gemm(dx, dxs, dw[0], dws[0], out.half(), big),
        lambda: mx.mxfp4_gemm(dx, dxs, dw[0], dws[0], out.bfloat16(), big, accumulate=True),
        lambda: mx.mxfp4_gemm(dx, dxs, dw[0], dws[0], out[:, :63], big),
        lambda: mx.mxfp4_gemm(dx, dxs, dw[0], dws[0], out, big[:16]),
        lambda: mx.mxfp4_gemm(dx[:, 1:], dxs, dw[0], dws[0], out, big),
        lambda: mx.mxfp4_gemm(dx[:, :40], dxs[:, :2], dw[0, :, :40].contiguous(), dws[0, :, :2].contiguous(), out, big),
        lambda: mx.mxfp4_gemm(dx, dxs, dw[0].t(), dws[0], out, big),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw[0], dws, off, out, big),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off.long(), out, big),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off[:3], out, big),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, out, big, w3=dw3),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, out, big, top_k=2),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, out, big, top_k=-1, sorted_pair=sp),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, out, big, pair_weight=f[0]),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, out, big, w3=dw3, w3_scale=dws3, sorted_pair=sp,
                                     pair_weight=f[0]),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, q, big, out_scale=s),
        lambda: mx.mxfp4_expert_gemm(dx[:2], dxs[:2], dw, dws, off, out, big),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, out, big[:16]),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, q, big, w3=dw3, w3_scale=dws3),
        lambda: mx.mxfp4_expert_gemm(dx, dxs, dw, dws, off, out, big, w3=dw3, w3_scale=dws3, beta=0.0),
    ]
    for i, b in enumerate(bad):
        with pytest.raises((ValueError, KeyError, mx.MoeError)):
            b()
            say(f"refusal {i} did not come")
