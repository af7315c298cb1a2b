"""The products on MXFP4 rows with scale rows that go straight into LDS: whole dwords apart and aligned, which is how the
layer's own calls have them (contiguous rows, K a multiple of 128).

Scales of two neighbouring binades on each side make every sum exact in fp32 (see test_gpu_mx4.py), so results are those
of float64, rounded once.  Behind a row's scales stand NaN bytes: of other rows, or in a pitch of four more than a row
needs.  A few rows and columns have NaN scales of their own and are NaN alone.  SiTU-GLU is off by at most
(32 + |g|) 2^-23 of its value (derived there).  test_mx4_expert_plan_host.py holds these sizes to every kernel and cut.
"""
import numpy as np
import pytest
import torch

from gpu_common import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
PITCH = {"contiguous": 0, "a pitch": 4}


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as mx
    mx.load()
    return mx


def values(q, s):
    """float64 values of codes and scale bytes."""
    table = torch.tensor(E2M1, dtype=torch.float64, device=q.device)
    v = table[torch.stack([q & 15, q >> 4], -1).flatten(-2).int()]
    e = torch.exp2(s.double() - 127)
    return (v.unflatten(-1, (-1, 32)) * torch.where(s == 255, torch.nan, e)[..., None]).flatten(-2)


def codes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device=DEV)


def scales(g, lo, *shape, pad=0):
    """Scale bytes lo and lo + 1; with a pad, NaN in `pad` bytes behind each row."""
    s = torch.randint(lo, lo + 2, (*shape[:-1], shape[-1] + pad), generator=g, dtype=torch.uint8, device=DEV)
    s[..., shape[-1]:] = 255
    return s[..., :shape[-1]]


def seeded(n):
    return torch.Generator(device=DEV).manual_seed(n)


def direct(s, K):
    """The condition for scales to be loaded straight into LDS."""
    return s.data_ptr() % 4 == 0 and (len(s) < 2 or s.stride(0) % 4 == 0) and K // 32 % 4 == 0


def workspace(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)


# test_mx4_expert_plan_host.py: streams by 16, 32 and 64 rows; tiles of 64, 128, 192 and 256 rows, whole, in parts of K and
# behind rounds of larger ones.  K ends inside a stage of 256 and inside a pair of stages.
DENSE = [(16, 100, 128), (9, 300, 1152), (3, 260, 7168), (20, 260, 640), (31, 257, 2432), (40, 512, 1152), (300, 64, 896),
         (130, 257, 3968), (200, 2100, 128), (100, 4400, 2432), (200, 2100, 6784), (700, 6200, 1152), (700, 1800, 6784),
         (1500, 6200, 1408), (4000, 6200, 640), (2900, 6200, 1152), (2000, 6200, 2432), (200, 6200, 6784)]


LONG = (200, 4400, 131072)


@pytest.mark.parametrize("pitch", PITCH)
@pytest.mark.parametrize("T,N,K", DENSE)
def test_dense(mx, T, N, K, pitch):
    g = seeded(T + N + K)
    x, xs, w, ws = codes(g, T, K // 2), scales(g, 127, T, K // 32, pad=PITCH[pitch]), codes(g, N, K // 2), scales(g, 123, N, K // 32)
    row, col = T // 2, N // 3
    xs[row, K // 64] = 255
    ws[col] = 255
    assert direct(xs, K) and direct(ws, K)
    ref = values(x, xs) @ values(w, ws).T.contiguous()
    scratch = workspace(mx.mxfp4_gemm_workspace_bytes(T, N, K))
    for out_kind, opad, accumulate in (("f32", 0, False), ("f32", 1, True), ("f32", 4, True), ("bf16", 8, False),
                                       ("bf16", 4, False), ("bf16", 1, False)):
        say(f"case: 4-bit product, direct scales ({pitch}), T={T} N={N} K={K} out {out_kind} pad {opad} added {accumulate}")
        out = torch.full((T, N + opad), 3.0, dtype=DT[out_kind], device=DEV)
        mx.mxfp4_gemm(x, xs, w, ws, out[:, :N], scratch, accumulate=accumulate)
        want = (ref + 3.0 if accumulate else ref).to(DT[out_kind])
        nan = torch.isnan(want)
        assert nan[row].all() and nan[:, col].all() and int(nan.sum()) == T + N - 1
        assert torch.equal(torch.isnan(out[:, :N]), nan) and torch.equal(out[:, :N][~nan], want[~nan])
        assert (out[:, N:] == 3.0).all()


def test_dense_parts_of_the_largest_tiles(mx):
    """K so long that tiles of 256 rows take parts of it: ones and minus ones, whose sums stay exact."""
    T, N, K = LONG
    say(f"case: 4-bit product, direct scales, T={T} N={N} K={K}")
    g = seeded(1)
    x, w = ((codes(g, n, K // 2) & 0x88) + 0x22 for n in (T, N))
    xs, ws = scales(g, 127, T, K // 32, pad=4), scales(g, 123, N, K // 32)
    xs[5, -1] = 255
    assert direct(xs, K) and direct(ws, K)
    out = torch.empty((T, N), device=DEV)
    mx.mxfp4_gemm(x, xs, w, ws, out, workspace(mx.mxfp4_gemm_workspace_bytes(T, N, K)))
    a = values(x, xs)
    for n in range(0, N, 500):
        want = (a @ values(w[n:n + 500], ws[n:n + 500]).T.contiguous()).float()
        assert torch.equal(torch.nan_to_num(out[:, n:n + 500], 0.3), torch.nan_to_num(want, 0.3))
    assert torch.isnan(out[5]).all() and int(torch.isnan(out).sum()) == N


def test_dense_both_ways(mx):
    """The same product with scale rows that cannot go straight into LDS: the same bits."""
    for T, N, K in ((9, 300, 1152), (31, 257, 2432), (130, 257, 3968), (700, 1800, 6784), (2000, 6200, 640)):
        say(f"case: 4-bit product, scales both ways, T={T} N={N} K={K}")
        g = seeded(T)
        x, xs, w, ws = codes(g, T, K // 2), scales(g, 110, T, K // 32), codes(g, N, K // 2), scales(g, 120, N, K // 32)
        xs[:, ::3] += 20  # sums that are not exact
        scratch = workspace(mx.mxfp4_gemm_workspace_bytes(T, N, K))
        other = torch.full((T, K // 32 + 3), 255, dtype=torch.uint8, device=DEV)
        moved = torch.full((T, K // 32 + 4), 255, dtype=torch.uint8, device=DEV)
        other[:, :K // 32], moved[:, 1:K // 32 + 1] = xs, xs
        outs = [torch.empty((T, N), device=DEV) for _ in range(3)]
        for s, out in zip((xs, other[:, :K // 32], moved[:, 1:K // 32 + 1]), outs):
            mx.mxfp4_gemm(x, s, w, ws, out, scratch)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# counts of rows an expert, gate and up's and down's columns.  test_mx4_expert_plan_host.py: chunks that work-groups find
# themselves; tiles alone, of every height; tiles and streamed experts; streamed experts with a tile launch that finds none
EXPERTS = {
    "found": ([5, 0, 1, 17, 0, 2, 40, 64, 65], 160, 257),
    "tiles": ([70, 400, 0, 17, 190, 300, 1, 129], 5120, 10000),
    "both": ([1] * 12 + [0, 200, 16, 65, 17, 3, 0, 129, 2, 33, 0, 256], 4160, 8325),
    "streamed": ([1, 2, 0, 5] * 24, 1024, 2049),
}


def routed(mx, counts, N, K, glu, out_kind, gathered, weights=False, pitch=0, opad=0, spare=3, seed=0):
    g = seeded(seed + N + K)
    E, P = len(counts), sum(counts) + spare
    end, tokens, k = P - spare, 50, 3
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device=DEV)
    rows = tokens if gathered else P
    pair = torch.randint(0, tokens * k, (P,), generator=g, dtype=torch.int32, device=DEV)
    x, xs = codes(g, rows, K // 2), scales(g, 127, rows, K // 32, pad=pitch)
    low = 117 if glu else 123  # gate and up products of a few units, where SiTU-GLU bends
    mats = [(codes(g, E, N, K // 2), scales(g, low, E, N, K // 32)) for _ in range(2 if glu else 1)]
    bad, col, spoilt_e = 7 % rows, N // 3, next(e for e in (*range(E // 2, E), 0) if counts[e])
    xs[bad, 1] = 255
    mats[0][1][spoilt_e, col] = 255
    assert direct(xs, K) and all(direct(s[0], K) for _, s in mats)
    pw = torch.rand(tokens * k, generator=g, device=DEV) if weights else None
    kw = dict(sorted_pair=pair, top_k=k) if gathered else dict(sorted_pair=pair) if weights else {}
    if glu:
        kw |= dict(w3=mats[1][0], w3_scale=mats[1][1])
    if weights:
        kw["pair_weight"] = pw
    four = out_kind == "mx4"
    cols, fill = (N // 2, 0xEE) if four else (N, 3.0)
    out = torch.full((P, cols + opad), fill, dtype=torch.uint8 if four else DT[out_kind], device=DEV)
    sc = torch.full((P, N // 32 + opad), 0xEE, dtype=torch.uint8, device=DEV)
    if four:
        kw["out_scale"] = sc[:, :N // 32]
    mx.mxfp4_expert_gemm(x, xs, mats[0][0], mats[0][1], off, out[:, :cols],
                         workspace(mx.mxfp4_expert_gemm_workspace_bytes(E, P, N, K)), **kw)
    assert (out[end:] == fill).all() and (out[:, cols:] == fill).all()
    assert (sc[end:] == 0xEE).all() and (sc[:, N // 32:] == 0xEE).all()
    a = values(x, xs)
    ends = np.cumsum(counts).tolist()
    for e in range(E):
        r = slice(ends[e] - counts[e], ends[e])
        if not counts[e]:
            continue
        at = a[(pair[r].long() // k) if gathered else r]
        p = [at @ values(q[e], s[e]).T.contiguous() for q, s in mats]
        if not glu:
            want = p[0].float()  # exact
            if weights:
                want = want * pw[pair[r].long()][:, None]
            assert torch.equal(torch.nan_to_num(out[r, :N], 77.0), torch.nan_to_num(want.to(DT[out_kind]), 77.0)), e
            continue
        gate, up = p
        ref = 4 * torch.tanh(gate / 4) * torch.sigmoid(gate) * 25 * torch.tanh(up / 25)
        nan = torch.isnan(ref)
        assert nan[:, col].all() or e != spoilt_e
        tol = ref.abs() * (32 + gate.abs()) * 2.0 ** -23 + 1e-37
        if four:
            b, t = ref.unflatten(1, (-1, 32)), tol.unflatten(1, (-1, 32))
            spoilt = torch.isnan(b).any(2)
            s = sc[r, :N // 32]
            assert torch.equal(s == 255, spoilt)
            lo, hi = (fit_byte((b.abs() + d * t).clamp_min(0).amax(2)) for d in (-1, 1))
            assert (((lo <= s) & (s <= hi)) | spoilt).all()
            v = values(out[r, :cols], torch.full_like(s, 127)).unflatten(1, (-1, 32))
            assert (v[spoilt] == 0).all()
            unit = torch.exp2(s.double() - 127)[..., None]
            ok = (grid((b - t) / unit) <= v) & (v <= grid((b + t) / unit))
            assert (ok | spoilt[..., None]).all(), e
            continue
        got = out[r, :N].double()
        if out_kind == "bf16":
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        assert torch.equal(torch.isnan(got), nan) and (((got - ref).abs() <= tol) | nan).all(), e


def fit_byte(top):
    """The scale byte of the smallest power of two with top <= 6 of it."""
    m, p = torch.frexp(top)  # top = m 2^p, 6 = 0.75 2^3
    e = p - 3 + (m > 0.75).int()
    return torch.where(top == 0, -125, e.clamp(-125, 126)) + 127


def grid(t):
    """t on e2m1's values: nearest, ties to even, at most 6."""
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp_max(6.0), t)


@pytest.mark.parametrize("K", [128, 640, 1152, 2176])
@pytest.mark.parametrize("form", EXPERTS)
def test_expert_glu(mx, form, K):
    counts, N, _ = EXPERTS[form]
    for out_kind, gathered, pitch in (("mx4", True, 0), ("mx4", False, 4), ("f32", True, 4), ("bf16", False, 0)):
        say(f"case: gate and up, direct scales, {form} K={K} out {out_kind} gathered {gathered} pitch {pitch}")
        routed(mx, counts, N, K, True, out_kind, gathered, pitch=pitch, opad=16 if gathered else 0)


@pytest.mark.parametrize("K", [128, 640, 1152, 2176])
@pytest.mark.parametrize("form", EXPERTS)
def test_expert_down(mx, form, K):
    counts, _, N = EXPERTS[form]
    for out_kind, gathered, weights, pitch, opad in (("f32", False, False, 0, 0), ("f32", False, True, 4, 3),
                                                     ("bf16", True, True, 0, 1), ("bf16", False, False, 4, 0),
                                                     ("f32", True, False, 4, 1)):
        say(f"case: down, direct scales, {form} K={K} out {out_kind} gathered {gathered} weights {weights} pitch {pitch}")
        routed(mx, counts, N, K, False, out_kind, gathered, weights, pitch=pitch, opad=opad)


def test_expert_many_experts(mx):
    """1024 experts, rows in order and gathered, through lists of both kinds."""
    rng = np.random.default_rng(8)
    counts = rng.permutation(np.concatenate([np.zeros(800, int), rng.integers(1, 5, 200), [70] * 24])).tolist()
    say("case: expert products, direct scales, 1024 experts")
    routed(mx, counts, 128, 384, True, "mx4", True)
    routed(mx, counts, 129, 384, False, "f32", False, True, pitch=4)


@pytest.mark.parametrize("T,N", [(16, 300), (20, 300), (300, 1300), (700, 6200)])
def test_blocks_of_zeros(mx, T, N):
    """Blocks of zeros add nothing, under scales whose product is far outside fp32's range too: quantised zeros have the
    least scale there is, 2^-125, and weights are below 1."""
    K = 512
    say(f"case: 4-bit product of blocks of zeros, T={T} N={N}")
    g = seeded(T)
    rows = torch.randn(T, K, generator=g, device=DEV)
    rows[:, :128] = 0
    rows[0] = 0
    x, xs = (torch.empty((T, n), dtype=torch.uint8, device=DEV) for n in (K // 2, K // 32))
    mx.mxfp4_quantize(rows, x, xs)
    assert (xs[:, :4] == 2).all() and (xs[0] == 2).all()
    w, ws = codes(g, N, K // 2), scales(g, 118, N, K // 32)
    # under the rows' zeros (blocks 0 to 3) weights of every scale; under zeros of both signs in the weights (4 to 7) rows
    ws[:, :4] = torch.randint(0, 255, (N, 4), generator=g, device=DEV).byte()
    w[:, 64:128] &= 0x88
    ws[:, 4:8] = torch.randint(0, 255, (N, 4), generator=g, device=DEV).byte()
    xs[1:, 4:8] = torch.randint(0, 255, (T - 1, 4), generator=g, device=DEV).byte()
    ws[0, :8], xs[1, 4:8], ws[1, :8], xs[2, 4:8] = 254, 254, 0, 0
    out = torch.empty((T, N), device=DEV)
    mx.mxfp4_gemm(x, xs, w, ws, out, workspace(mx.mxfp4_gemm_workspace_bytes(T, N, K)))
    a, b = values(x, xs), values(w, ws)
    ref, mag = a @ b.T.contiguous(), a.abs() @ b.abs().T.contiguous()
    assert torch.isfinite(out).all() and (out[0] == 0).all()
    # 128 additions in an instruction, K / 64 instructions, 16 joins, each off by 2^-23 of the sum of magnitudes at most
    assert ((out.double() - ref).abs() <= (128 + K // 64 + 16) * 2.0 ** -23 * mag).all()


def test_element_types(mx):
    """Codes and scales in torch's own types for them, where it has them, are the same bytes."""
    if not hasattr(torch, "float4_e2m1fn_x2") or not hasattr(torch, "float8_e8m0fnu"):
        pytest.skip("torch without 4-bit floats")
    say("case: 4-bit products of tensors of torch's 4-bit and scale types")
    four, e8 = (lambda t: t.view(torch.float4_e2m1fn_x2)), (lambda t: t.view(torch.float8_e8m0fnu))
    g = seeded(4)
    E, T, N, K = 3, 40, 96, 256
    x, xs = torch.empty((T, K // 2), dtype=torch.uint8, device=DEV), torch.empty((T, K // 32), dtype=torch.uint8, device=DEV)
    rows = torch.randn(T, K, generator=g, device=DEV)
    mx.mxfp4_quantize(rows, four(x), e8(xs))
    back, want = torch.empty_like(rows), values(x, xs)
    mx.mxfp4_dequantize(four(x), e8(xs), back)
    assert torch.equal(back.double(), want) and not torch.equal(want, torch.zeros_like(want))
    w, ws, w3, ws3 = codes(g, E, N, K // 2), scales(g, 117, E, N, K // 32), codes(g, E, N, K // 2), scales(g, 117, E, N, K // 32)
    scratch = workspace(1 << 16)
    outs = [torch.empty((T, N), device=DEV) for _ in range(2)]
    mx.mxfp4_gemm(x, xs, w[0], ws[0], outs[0], scratch)
    mx.mxfp4_gemm(four(x), e8(xs), four(w[0]), e8(ws[0]), outs[1], scratch)
    assert torch.equal(*outs)
    off = torch.tensor([0, 7, 7, T], dtype=torch.int32, device=DEV)
    h = [(torch.zeros((T, N // 2), dtype=torch.uint8, device=DEV), torch.zeros((T, N // 32), dtype=torch.uint8, device=DEV))
         for _ in range(2)]
    mx.mxfp4_expert_gemm(x, xs, w, ws, off, h[0][0], scratch, w3=w3, w3_scale=ws3, out_scale=h[0][1])
    mx.mxfp4_expert_gemm(four(x), e8(xs), four(w), e8(ws), off, four(h[1][0]), scratch, w3=four(w3), w3_scale=e8(ws3),
                         out_scale=e8(h[1][1]))
    assert torch.equal(h[0][0], h[1][0]) and torch.equal(h[0][1], h[1][1]) and h[0][0].any()
