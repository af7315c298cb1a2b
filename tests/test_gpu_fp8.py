"""The 8-bit product against fp64 on the dequantised operands.

Tolerance, fp32 out.  Products of e4m3 codes are exact in fp32.  A block's sum
has at most 128 additions and is scaled once; the sums of kb blocks are added,
some of them in separate parts.  Each of these 128 + 2 kb + 8 steps is off by
at most 2^-23 of the sum of magnitudes (twice a rounding, as the matrix units
may truncate), so |err| <= (128 + 2 kb + 8) 2^-23 sum |x w|.  bf16 out adds half
a step, and what the 8-bit matrix instructions drop: each of a block's 128
products loses at most 2^-14 of the largest.  Codes that stay inside the
instructions' window give exact sums, which pins the indexing without any of
this (test_exact_sums).
"""
import numpy as np
import pytest
import torch

from gpu_common import say
from test_gpu_block import e4m3

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as mx
    mx.load()
    return mx


def operands(T, N, K, kind, seed, pad=0):
    """Random codes without NaN, scales of a few binades; rows of x strided by K + pad."""
    rng = np.random.default_rng(seed)
    kb, nb = -(-K // 128), -(-N // 128)

    def codes(*shape):
        c = rng.integers(0, 256, shape).astype(np.uint8)
        return np.where((c & 0x7F) == 0x7F, 0x3A, c).astype(np.uint8)

    x, w = codes(T, K + pad), codes(N, K)
    x[:, K:] = 0x7F  # NaN beside the rows
    xs = rng.integers(118, 126, (T, kb + 1)).astype(np.uint8)
    ws = (rng.integers(115, 122, (nb, kb)).astype(np.uint8) if kind == "e8m0"
          else (np.exp(rng.normal(size=(nb, kb))) * 0.01).astype(np.float32))
    return x, xs, w, ws


def reference(x, xs, w, ws, K, kind):
    """(value, sum of magnitudes) in fp64."""
    kb = -(-K // 128)
    N = w.shape[0]
    a = e4m3(x[:, :K]) * np.repeat(2.0 ** (xs[:, :kb].astype(np.float64) - 127), 128, 1)[:, :K]
    s = 2.0 ** (ws.astype(np.float64) - 127) if kind == "e8m0" else ws.astype(np.float64)
    b = e4m3(w) * np.repeat(np.repeat(s, 128, 0)[:N], 128, 1)[:, :K]
    top = [[np.abs(v[:, 128 * j:128 * j + 128]).max(1) for j in range(kb)] for v in (a, b)]
    # an upper bound of each block's largest product, summed over the blocks
    return a @ b.T, np.abs(a) @ np.abs(b).T, sum(np.outer(p, q) for p, q in zip(*top))


def bound(mag, top, K, out, ref):
    kb = -(-K // 128)
    t = (128 + 2 * kb + 8) * 2.0 ** -23 * mag
    if out == "bf16":
        t = t + 128 * 2.0 ** -14 * top
        t = t + 2.0 ** -8 * (np.abs(ref) + t)
    return t + 1e-37


def run(mx, T, N, K, kind, out_kind, seed=0, pad=0, opad=0, accumulate=False):
    x, xs, w, ws = operands(T, N, K, kind, seed, pad)
    kb = -(-K // 128)
    dx, dxs, dw, dws = (torch.from_numpy(v).to(DEV) for v in (x, xs, w, ws))
    dt = torch.bfloat16 if out_kind == "bf16" else torch.float32
    out = torch.full((T, N + opad), 3.0, dtype=dt, device=DEV)
    scratch = torch.full((mx.fp8_gemm_workspace_bytes(T, N, K),), 0xFF, dtype=torch.uint8, device=DEV)
    mx.fp8_gemm(dx[:, :K], dxs[:, :kb], dw, dws, out[:, :N], scratch, accumulate=accumulate)
    again = torch.full_like(out, 3.0)
    mx.fp8_gemm(dx[:, :K], dxs[:, :kb], dw, dws, again[:, :N], scratch, accumulate=accumulate)
    assert torch.equal(out.nan_to_num(0.0), again.nan_to_num(0.0))  # the same twice
    assert (out[:, N:] == 3.0).all()
    ref, mag, top = reference(x, xs, w, ws, K, kind)
    got = out[:, :N].float().cpu().numpy().astype(np.float64)
    if accumulate:
        got = got - 3.0
        mag = mag + 3.0
    assert (np.abs(got - ref) <= bound(mag, top, K, out_kind, ref)).all()


# tokens on both sides of every column tile, rows and K that end inside a block
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 16, 128), (2, 17, 144), (15, 130, 1040), (16, 128, 2048),
                                   (17, 257, 256), (31, 64, 4112), (33, 100, 384), (64, 255, 640), (65, 384, 400),
                                   (127, 129, 272), (129, 513, 1152), (255, 895, 1024), (257, 256, 128),
                                   (300, 640, 3600), (700, 1100, 528), (70, 130, 16400),
                                   (7, 6150, 400), (16, 6145, 4128), (9, 50, 4112), (1, 300, 5008), (50, 900, 4112),
                                   (41, 4200, 4112)])
def test_product(mx, T, N, K, kind):
    out = "bf16" if (T + N) % 2 else "f32"
    say(f"case: 8-bit product T={T} N={N} K={K} scales {kind} out {out}")
    run(mx, T, N, K, kind, out, seed=T + N + K)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,N,K", [(1, 40, 272), (16, 130, 400), (60, 300, 1040), (130, 257, 528), (513, 640, 1168)])
def test_exact_sums(mx, T, N, K, kind):
    """Codes of magnitude 1 to 1.875: products are multiples of 1/64 below 4, every sum is exact in fp32 and in the
    8-bit instructions, scales are powers of two: the results are exact."""
    say(f"case: 8-bit product, exact sums, T={T} N={N} K={K} scales {kind}")
    rng = np.random.default_rng(T)
    kb, nb = -(-K // 128), -(-N // 128)
    x, w = ((0x38 + rng.integers(0, 8, s) + 0x80 * rng.integers(0, 2, s)).astype(np.uint8) for s in ((T, K), (N, K)))
    xs = rng.integers(125, 130, (T, kb)).astype(np.uint8)
    e = rng.integers(125, 130, (nb, kb))
    ws = e.astype(np.uint8) if kind == "e8m0" else (2.0 ** (e - 127.0)).astype(np.float32)
    d = [torch.from_numpy(v).to(DEV) for v in (x, xs, w, ws)]
    scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    ref, _, _ = reference(x, xs, w, ws, K, kind)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty((T, N), dtype=dt, device=DEV)
        mx.fp8_gemm(*d, out, scratch)
        want = torch.from_numpy(ref).to(dt)  # sums of under 2^24 steps of 2^-10: exact, then rounded once
        assert torch.equal(out.cpu(), want)


# K in parts; tiles of 128 tokens in one turn; of 256 in one turn; first of 256, then of 128; long K
TILES = [(130, 3000, 4112), (1500, 3000, 272), (3000, 3000, 144), (4100, 4500, 272), (100, 6144, 7168)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,N,K", TILES)
def test_tiles(mx, T, N, K, kind, out):
    say(f"case: 8-bit product by tiles T={T} N={N} K={K} scales {kind} out {out}")
    run(mx, T, N, K, kind, out, seed=T + K, pad=16, opad=4 if N < 4000 else 1)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,N,K", TILES[:4])
def test_tiles_exact_and_nan(mx, T, N, K, kind):
    """As test_exact_sums, in both outputs; then one NaN code in each operand, which stays in its row and column."""
    say(f"case: 8-bit product by tiles, exact sums, T={T} N={N} K={K} scales {kind}")
    rng = np.random.default_rng(N)
    kb, nb = -(-K // 128), -(-N // 128)
    x, w = ((0x38 + rng.integers(0, 8, s) + 0x80 * rng.integers(0, 2, s)).astype(np.uint8) for s in ((T, K), (N, K)))
    xs = rng.integers(125, 130, (T, kb)).astype(np.uint8)
    e = rng.integers(125, 130, (nb, kb))
    ws = e.astype(np.uint8) if kind == "e8m0" else (2.0 ** (e - 127.0)).astype(np.float32)
    d = [torch.from_numpy(v).to(DEV) for v in (x, xs, w, ws)]
    scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    a = e4m3(x).astype(np.float32) * np.repeat(2.0 ** (xs.astype(np.float32) - 127), 128, 1)[:, :K]
    b = e4m3(w).astype(np.float32) * np.repeat(np.repeat(2.0 ** (e - 127.0), 128, 0)[:N], 128, 1)[:, :K].astype(np.float32)
    want = torch.from_numpy(a @ b.T)  # sums of under 2^24 steps of 2^-10: exact in fp32 in any order
    bad = torch.zeros((T, N), dtype=torch.bool, device=DEV)
    bad[T - 2] = True
    bad[:, N - 1] = True
    for dt in (torch.float32, torch.bfloat16):
        d[0][T - 2, K - 1], d[2][N - 1, 0] = int(x[T - 2, K - 1]), int(w[N - 1, 0])
        out = torch.empty((T, N), dtype=dt, device=DEV)
        mx.fp8_gemm(*d, out, scratch)
        assert torch.equal(out.cpu(), want.to(dt))
        d[0][T - 2, K - 1], d[2][N - 1, 0] = 0x7F, 0xFF
        got = torch.empty((T, N), dtype=dt, device=DEV)
        mx.fp8_gemm(*d, got, scratch)
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], out[~bad])


@pytest.mark.parametrize("T,N,K", [TILES[0], TILES[1], (100, 3002, 7168)])
def test_tiles_accumulate(mx, T, N, K):
    for opad in (1, 4):
        say(f"case: 8-bit product by tiles, added to: T={T} N={N} K={K} out pad {opad}")
        run(mx, T, N, K, "f32", "f32", seed=1, pad=16, opad=opad, accumulate=True)


# K in parts in both outputs, with rows that are not whole groups of four: test_fp8_plan_host.py holds the plan to that
PARTS_ODD = [(301, 895, 7168), (301, 893, 7168), (130, 3002, 4112)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,N,K", PARTS_ODD)
def test_parts_of_odd_rows(mx, T, N, K, kind):
    """The parts' padded rows and the last, shorter group of the pass that joins them."""
    for out, acc in (("f32", False), ("f32", True), ("bf16", False)):
        for opad in (0, 1, -N % 4):
            say(f"case: 8-bit product, K in parts, T={T} N={N} K={K} scales {kind} out {out} pad {opad} added {acc}")
            run(mx, T, N, K, kind, out, seed=N, pad=16, opad=opad, accumulate=acc)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_what_the_8_bit_instruction_drops(mx, kind):
    """bf16 results by the 8-bit instructions, normally distributed operands: the documented loss is 1.5e-5 of the
    results' rms.  A result within 2^-10 of the rms of zero is rounded to bf16 by less than 2^-18 = 3.8e-6 of it, so
    there the loss stands almost alone; about one in 1300 of the results is that small, some 1200 here, which gives their
    mean square to 5 per cent.  A third more than the documented figure is allowed for that and its digits."""
    T, N, K = 512, 2944, 4096
    say(f"case: 8-bit product, what is dropped, T={T} N={N} K={K} scales {kind}")
    g = torch.Generator().manual_seed(3)
    x, w = (torch.randn(n, K, generator=g) for n in (T, N))
    q, s = (torch.empty((T, n), dtype=torch.uint8, device=DEV) for n in (K, K // 128))
    mx.fp8_quantize(x.to(DEV), q, s)
    wq = (w * 100.0).clamp(-448, 448).to(torch.float8_e4m3fn).to(DEV)
    ws = torch.full((N // 128, K // 128), 120, dtype=torch.uint8) if kind == "e8m0" else torch.full((N // 128, K // 128),
                                                                                                 2.0 ** -7 * 1.1)
    out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    mx.fp8_gemm(q, s, wq, ws.to(DEV), out, scratch)
    scale = 2.0 ** -7 if kind == "e8m0" else float(np.float32(2.0 ** -7 * 1.1))
    a = e4m3(q.cpu().numpy()) * np.repeat(2.0 ** (s.cpu().numpy() - 127.0), 128, 1)
    ref = a @ (e4m3(wq.view(torch.uint8).cpu().numpy()) * scale).T
    err = out.float().cpu().numpy() - ref
    rms = np.sqrt(np.mean(ref ** 2))
    near = np.abs(ref) < 2.0 ** -10 * rms
    lost = np.sqrt(np.mean(err[near] ** 2)) / rms
    say(f"  {near.sum()} results near zero, lost {lost:.2e} of the rms")
    assert near.sum() > 500 and lost < 2e-5


def test_many_tokens_of_one_short_row(mx):
    """The most tokens a call may have: 65536 groups of them in one grid."""
    T, N, K = 1 << 22, 1, 16
    say(f"case: 8-bit product T={T} N={N} K={K}")
    x = torch.full((T, K), 0x38, dtype=torch.uint8, device=DEV)  # ones
    x[:, 0] = torch.where(torch.arange(T, device=DEV) % 5 == 0, 0x40, 0x38).to(torch.uint8)  # twos among them
    out = torch.zeros((T, N), device=DEV)
    mx.fp8_gemm(x, torch.full((T, 1), 128, dtype=torch.uint8, device=DEV),
                torch.full((N, K), 0x38, dtype=torch.uint8, device=DEV), torch.full((1, 1), 0.5, device=DEV), out,
                torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV))
    assert torch.equal(out[:, 0], 16.0 + (torch.arange(T, device=DEV) % 5 == 0).float())


def test_tiles_on_streams_and_replayed(mx):
    """K in parts: the parts' sums in a workspace of the call's own."""
    T, N, K = 130, 3000, 4112
    say("case: 8-bit product by tiles on two streams and replayed")
    nb = mx.fp8_gemm_workspace_bytes(T, N, K)
    assert nb > T * N * 8
    ops, want, out, scratch = [], [], [], []
    for seed in (1, 2):
        x, xs, w, ws = operands(T, N, K, "f32", seed)
        ops.append([torch.from_numpy(v.copy()).to(DEV) for v in (x, xs[:, :-1], w, ws)])
        scratch.append(torch.empty(nb, dtype=torch.uint8, device=DEV))
        want.append(torch.empty((T, N), dtype=torch.bfloat16, device=DEV))
        out.append(torch.empty((T, N), dtype=torch.bfloat16, device=DEV))
        mx.fp8_gemm(*ops[-1], want[-1], scratch[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            mx.fp8_gemm(*ops[i], out[i], scratch[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    # two graphs that share a workspace, one after the other, with eager calls between
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mx.fp8_gemm(*ops[i], out[i], scratch[0])
        graphs.append(g)
    for _ in range(3):
        for i in range(2):
            out[i].zero_()
            graphs[i].replay()
            mx.fp8_gemm(*ops[1], want[1], scratch[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("T,N,K", [(3, 100, 400), (40, 129, 272), (200, 200, 512), (520, 384, 1152)])
def test_strides_and_accumulate(mx, T, N, K):
    for opad in (1, 4):
        say(f"case: 8-bit product, strided rows, added to: T={T} N={N} K={K} out pad {opad}")
        run(mx, T, N, K, "f32", "f32", seed=1, pad=16, opad=opad, accumulate=True)
        run(mx, T, N, K, "e8m0", "bf16", seed=2, pad=32, opad=opad)


@pytest.mark.parametrize("T", [1, 16, 64, 384, 1024])
def test_full_sizes(mx, T):
    """Sizes of the layer's dense products; a sample of the outputs against fp64."""
    N, K = 3584, 7168
    say(f"case: 8-bit product at T={T} N={N} K={K}")
    x, xs, w, ws = operands(T, N, K, "f32", T)
    d = [torch.from_numpy(v).to(DEV) for v in (x, xs[:, :K // 128].copy(), w, ws)]
    out = torch.empty((T, N), device=DEV)
    scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    mx.fp8_gemm(*d, out, scratch)
    ts = np.unique(np.concatenate([[0, T - 1], np.random.default_rng(0).integers(0, T, 6)]))
    ref, mag, top = reference(x[ts], xs[ts], w, ws, K, "f32")
    got = out.cpu().numpy().astype(np.float64)[ts]
    assert (np.abs(got - ref) <= bound(mag, top, K, "f32", ref)).all()


def test_nan_stays_in_its_row_and_column(mx):
    for T in (5, 300):
        say(f"case: 8-bit product with a NaN code, T={T}")
        N, K = 260, 656
        x, xs, w, ws = operands(T, N, K, "f32", 3)
        d = [torch.from_numpy(v.copy()).to(DEV) for v in (x, xs[:, :-1], w, ws)]
        scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
        clean, out = torch.empty((T, N), device=DEV), torch.empty((T, N), device=DEV)
        mx.fp8_gemm(*d, clean, scratch)
        d[0][2, 650] = 0x7F
        d[2][255, 3] = 0xFF
        mx.fp8_gemm(*d, out, scratch)
        bad = torch.zeros((T, N), dtype=torch.bool, device=DEV)
        bad[2] = True
        bad[:, 255] = True
        assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("T,N,K", [(5, 900, 400), (60, 900, 400), TILES[0], TILES[1], TILES[3]])
def test_scale_bytes_at_their_ends(mx, T, N, K):
    """Weight scale bytes 255 (NaN) and 0 (2^-127), activation bytes 1 and 247: NaN in the block's rows, nothing
    elsewhere; the small and the large values as the formula has them."""
    say(f"case: 8-bit product, scale bytes at their ends, T={T} N={N} K={K}")
    x, xs, w, ws = operands(T, N, K, "e8m0", 4)
    xs = xs[:, :-1].copy()
    xs[1], xs[3] = 247, 1
    ws[2, 0], ws[5] = 255, 0
    d = [torch.from_numpy(v).to(DEV) for v in (x, xs, w, ws)]
    scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    bad = np.zeros(N, bool)
    bad[256:384] = True
    ts = np.unique([0, 1, 2, 3, 4, T - 1])
    ws[2, 0] = 120
    ref, mag, top = reference(x[ts], xs[ts], w, ws, K, "e8m0")
    for out_kind, dt in (("f32", torch.float32), ("bf16", torch.bfloat16)):
        out = torch.empty((T, N), dtype=dt, device=DEV)
        mx.fp8_gemm(*d, out, scratch)
        got = out.float().cpu().numpy().astype(np.float64)
        assert np.isnan(got[:, bad]).all() and not np.isnan(np.delete(got, 1, 0)[:, ~bad]).any()
        # token 1's sums of magnitudes pass 2^128: its partial sums may be infinite, and their sum NaN
        with np.errstate(all="ignore"):
            ok = (np.abs(got[ts] - ref) <= bound(mag, top, K, out_kind, ref)) | (mag >= 2.0 ** 127)
        assert ok[:, ~bad].all() and (mag < 2.0 ** 127)[ts != 1][:, ~bad].all()


def test_quantize_then_product(mx):
    """As used: bf16 rows, quantised, then the product, against the bf16 rows' own product in fp64 with the
    rounding of each operand value (2^-4, or half the grid's smallest step) counted."""
    T, N, K = 37, 300, 1040
    say("case: quantize then product")
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(DEV)
    _, _, w, ws = operands(T, N, K, "f32", 9)
    q = torch.empty((T, K), dtype=torch.uint8, device=DEV)
    s = torch.empty((T, -(-K // 128)), dtype=torch.uint8, device=DEV)
    mx.fp8_quantize(x, q, s)
    out = torch.empty((T, N), device=DEV)
    scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    mx.fp8_gemm(q, s, torch.from_numpy(w).to(DEV), torch.from_numpy(ws).to(DEV), out, scratch)
    xv = x.float().cpu().numpy().astype(np.float64)
    wv = e4m3(w) * np.repeat(np.repeat(ws.astype(np.float64), 128, 0)[:N], 128, 1)[:, :K]
    sc = np.repeat(2.0 ** (s.cpu().numpy().astype(np.float64) - 127), 128, 1)[:, :K]
    off = np.maximum(np.abs(xv) * 2.0 ** -4, sc * 2.0 ** -10)
    ref = xv @ wv.T
    tol = off @ np.abs(wv).T + bound((np.abs(xv) + off) @ np.abs(wv).T, 0, K, "f32", ref)
    assert (np.abs(out.cpu().numpy() - ref) <= tol).all()


def test_graph_replays_and_streams(mx):
    for T in (4, 300):
        say(f"case: 8-bit product on two streams and replayed, T={T}")
        N, K = 640, 2048
        ops = []
        for seed in (1, 2):
            x, xs, w, ws = operands(T, N, K, "f32", seed)
            ops.append([torch.from_numpy(v.copy()).to(DEV) for v in (x, xs[:, :-1], w, ws)])
        nb = mx.fp8_gemm_workspace_bytes(T, N, K)
        scratch = [torch.empty(nb, dtype=torch.uint8, device=DEV) for _ in range(2)]
        want = [torch.empty((T, N), device=DEV) for _ in range(2)]
        out = [torch.empty((T, N), device=DEV) for _ in range(2)]
        for i in range(2):
            mx.fp8_gemm(*ops[i], want[i], scratch[0])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(20):
            for i in range(2):
                mx.fp8_gemm(*ops[i], out[i], scratch[i], stream=streams[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mx.fp8_gemm(*ops[0], out[0], scratch[0])
        for _ in range(3):
            out[0].zero_()
            g.replay()
            mx.fp8_gemm(*ops[1], out[1], scratch[1])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals(mx):
    T, N, K = 2, 32, 64
    x, xs, w, ws = operands(T, N, K, "f32", 1)
    d = [torch.from_numpy(v.copy()).to(DEV) for v in (x, xs[:, :1], w, ws)]
    out = torch.empty((T, N), device=DEV)
    scratch = torch.empty(mx.fp8_gemm_workspace_bytes(T, N, K), dtype=torch.uint8, device=DEV)
    assert mx.fp8_gemm_workspace_bytes(T, N, 40) == 0
    mx.fp8_gemm(d[0][:0], d[1][:0], d[2], d[3], out[:0], scratch)  # no rows
    for bad in (lambda: mx.fp8_gemm(d[0], d[1], d[2][:, :40], d[3], out, scratch),
                lambda: mx.fp8_gemm(d[0][:, :40].contiguous(), d[1], d[2][:, :40].contiguous(), d[3], out, scratch),
                lambda: mx.fp8_gemm(*d, out.half(), scratch),
                lambda: mx.fp8_gemm(*d, out.bfloat16(), scratch, accumulate=True),
                lambda: mx.fp8_gemm(*d, out, scratch[:16]),
                lambda: mx.fp8_gemm(d[0], d[1][:1], d[2], d[3], out, scratch),
                lambda: mx.fp8_gemm(d[0], d[1], d[2], d[3].half(), out, scratch),
                lambda: mx.fp8_gemm(d[0], d[1], d[2], d[3], out[:, :31], scratch)):
        with pytest.raises((ValueError, mx.MoeError)):
            bad()
