"""The norms around the block and the 8-bit activations against fp64 on the CPU.

Tolerances.  A normed value goes through the row's fp32 sum of squares (at most
32 additions in a thread, 6 in the wave, 8 over the waves, each off by 2^-24 of
the sum, and half of it in the root), a division, a root and a few products:
under 64 roundings of 2^-24, so F32 = 2^-18 relative.  Storing rounds by at
most half a step: 2^-8 relative in bf16, 2^-24 in fp32.  e4m3 codes are off by
2^-4 of the value, or by half the smallest step, 2^-10 of the scale.
"""
import numpy as np
import pytest
import torch

from gpu_common import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32 = 2.0 ** -18
BF = 2.0 ** -8
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as mx
    mx.load()
    return mx


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rms(v, gamma, eps):
    return v / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps) * gamma


def e4m3(codes):
    """Values of e4m3 codes, from the bits."""
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 0x80, -v, v)


def grid(t):
    """t on the e4m3 grid, ties to even."""
    step = 2.0 ** (np.maximum(np.frexp(np.abs(t))[1] - 1, -6) - 3)
    return np.round(t / step) * step


def quantized(v):
    """(values, scale bytes) by the definition, in fp64: exact."""
    T, K = v.shape
    kb = -(-K // 128)
    q, sb = np.empty_like(v), np.empty((T, kb), np.int64)
    for b in range(kb):
        s = slice(128 * b, min(K, 128 * b + 128))
        blk = v[:, s]
        top = np.max(np.where(np.isfinite(blk), np.abs(blk), 0.0), axis=1)
        for t in range(T):
            e = -126
            if top[t] > 448 * 2.0 ** -126:
                e = int(np.ceil(np.log2(top[t] / 448.0))) - 1
                while top[t] > 448 * 2.0 ** e:
                    e += 1
            sb[t, b] = e + 127
        with np.errstate(invalid="ignore"):
            q[:, s] = np.where(np.isfinite(blk), grid(blk / 2.0 ** (sb[:, b:b + 1] - 127.0)), np.nan)
    return q, sb


def rows(T, H, dtype, pad, seed, std=1.0, special=False):
    """[T, H] values in a wider tensor (rows strided by H + pad)."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(T, H + pad, generator=g) * std * torch.exp(0.7 * torch.randn(H + pad, generator=g))
    if special and T > 2:
        v[1] = 0.0
        v[2] *= 1e-20
    return v.to(dtype).to(DEV)[:, :H]


def check_normed(n, q, qs, ref, H):
    """The written forms of a normed row against the fp64 one."""
    if n is not None:
        err = np.abs(f64(n) - ref)
        assert (err <= np.abs(ref) * (BF + F32) * (1 + BF) + 1e-38).all()
    if q is None:
        return
    sb = qs.cpu().numpy().astype(np.int64)
    s = np.repeat(2.0 ** (sb - 127.0), 128, axis=1)[:, :H]
    v = e4m3(q.cpu().numpy()) * s
    assert (np.abs(v - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s) + F32 * np.abs(ref)).all()
    for b in range(sb.shape[1]):
        top = np.abs(ref[:, 128 * b:128 * b + 128]).max(1)
        sc = 2.0 ** (sb[:, b] - 127.0)
        assert (top <= 448 * sc * (1 + F32)).all()  # large enough
        assert ((top * (1 + F32) > 224 * sc) | (sb[:, b] == 1)).all()  # and not larger


# widths: one lane's chunk, a block, not a multiple of 8 or 16, several rounds of threads
SHAPES = [(1, 7168, 0), (3, 1, 0), (2, 8, 8), (5, 127, 1), (4, 129, 3), (3, 136, 8), (7, 4096, 0), (3, 4104, 24),
          (2, 8200, 0), (2, 16384, 0), (300, 256, 0)]


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,pad", SHAPES)
def test_pre_norm(mx, T, H, pad, xd):
    say(f"case: pre norm T={T} H={H} pad={pad} {xd}")
    x = rows(T, H, DTYPES[xd], pad, seed=T + H, special=True)
    gamma = (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).to(DEV)
    kb = -(-H // 128)
    n = torch.full((T, H + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    q = torch.full((T, H + pad), 0x55, dtype=torch.uint8, device=DEV)
    qs = torch.full((T, kb + 1), 0x55, dtype=torch.uint8, device=DEV)
    mx.block_pre_norm(x, gamma, 1e-6, n=n[:, :H], q=q[:, :H], q_scale=qs[:, :kb])
    check_normed(n[:, :H], q[:, :H], qs[:, :kb], rms(f64(x), f64(gamma), 1e-6), H)
    # what lies beside the rows stays
    assert (n[:, H:] == 7.0).all() and (q[:, H:] == 0x55).all() and (qs[:, kb:] == 0x55).all()
    # each form alone is the same
    n1, q1, s1 = torch.empty_like(n), torch.empty_like(q), torch.empty_like(qs)
    mx.block_pre_norm(x, gamma, 1e-6, n=n1[:, :H])
    mx.block_pre_norm(x, gamma, 1e-6, q=q1[:, :H], q_scale=s1[:, :kb])
    assert torch.equal(n1[:, :H], n[:, :H]) and torch.equal(q1[:, :H], q[:, :H])
    assert torch.equal(s1[:, :kb], qs[:, :kb])


def test_pre_norm_not_finite_stays_in_its_row(mx):
    say("case: pre norm, NaN and infinity in a row")
    H = 512
    x = rows(4, H, torch.float32, 0, seed=3)
    clean = x.clone()
    x[1, 5] = float("nan")
    x[2, 300] = float("inf")
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    out = []
    for v in (x, clean):
        n = torch.empty((4, H), dtype=torch.bfloat16, device=DEV)
        q = torch.empty((4, H), dtype=torch.uint8, device=DEV)
        s = torch.empty((4, 4), dtype=torch.uint8, device=DEV)
        mx.block_pre_norm(v, gamma, 1e-6, n=n, q=q, q_scale=s)
        out.append((n, q, s))
    for a, b in zip(*out):
        assert torch.equal(a[[0, 3]], b[[0, 3]])
    n, q, s = (t.cpu() for t in out[0])
    assert torch.isnan(n[1]).all() and (q[1] == 0x7F).all() and (s[1] == 1).all()
    # an infinite value makes the root infinite: the others vanish, it is NaN
    assert torch.isnan(n[2, 300]) and (n[2].nan_to_num(0.0) == 0).all() and q[2, 300] == 0x7F


GATES = {"none": None, "token": "t", "channel": "c", "full": "f"}


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("yd,rd", [("f32", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("T,H,pad", [(1, 7168, 0), (5, 127, 1), (3, 8200, 8), (64, 384, 0)])
def test_post_norm(mx, T, H, pad, yd, rd, gate):
    sig = (T + H) % 2 == 0
    say(f"case: post norm T={T} H={H} pad={pad} y {yd} residual {rd} gate {gate} sigmoid {sig}")
    y = rows(T, H, DTYPES[yd], pad, seed=H, std=0.3, special=True)
    r = rows(T, H, DTYPES[rd], pad, seed=H + 1)
    gen = torch.Generator().manual_seed(5)
    gamma, nxt = ((1 + 0.1 * torch.randn(H, generator=gen)).to(torch.bfloat16).to(DEV) for _ in range(2))
    shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[gate]
    gd = torch.bfloat16 if rd == "f32" else torch.float32
    g = None if shape is None else torch.randn(*shape, generator=gen).to(gd).to(DEV)
    for norm in (True, False):
        out = torch.full((T, H + pad), 9.0, dtype=DTYPES[rd], device=DEV)
        n = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        q = torch.empty((T, H), dtype=torch.uint8, device=DEV)
        qs = torch.empty((T, -(-H // 128)), dtype=torch.uint8, device=DEV)
        kw = dict(gamma=gamma if norm else None, gate=g, gate_sigmoid=sig and g is not None, scale=0.22, eps=1e-6)
        mx.block_post_norm(y, r, out[:, :H], next_gamma=nxt, n=n, q=q, q_scale=qs, **kw)
        b = rms(f64(y), f64(gamma), 1e-6) if norm else f64(y)
        gv = 1.0 if g is None else (1 / (1 + np.exp(-f64(g))) if sig else f64(g))
        b = b * gv * np.float64(np.float32(0.22))
        ref = f64(r) + b
        half = BF if rd == "bf16" else 2.0 ** -24
        assert (np.abs(f64(out[:, :H]) - ref) <= (np.abs(ref) * half + np.abs(b) * F32) * (1 + BF) + 1e-37).all()
        assert (out[:, H:] == 9.0).all()
        # the next norm is that of the row as stored, bit for bit
        n1, q1, s1 = torch.empty_like(n), torch.empty_like(q), torch.empty_like(qs)
        mx.block_pre_norm(out[:, :H], nxt, 1e-6, n=n1, q=q1, q_scale=s1)
        assert torch.equal(n1, n) and torch.equal(q1, q) and torch.equal(s1, qs)
        check_normed(n, q, qs, rms(f64(out[:, :H]), f64(nxt), 1e-6), H)
        # in place
        r2 = r.clone() if pad == 0 else torch.nn.functional.pad(r, (0, pad))[:, :H]
        mx.block_post_norm(y, r2, r2, **kw)
        assert torch.equal(r2, out[:, :H])


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,pad", [(1, 1, 0), (1, 128, 0), (3, 127, 2), (5, 130, 0), (37, 7168, 16), (300, 272, 0)])
def test_quantize_exact(mx, T, K, pad, xd):
    say(f"case: quantize T={T} K={K} pad={pad} {xd}")
    x = rows(T, K, DTYPES[xd], pad, seed=K, special=True)
    if T > 4:
        x[3, 0] = float("nan")
        x[4, K - 1] = float("-inf")
        x[0, :] = torch.linspace(-448, 448, K).to(x.dtype).to(DEV)  # midpoints and borders among them
    kb = -(-K // 128)
    q = torch.full((T, K + pad), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((T, kb), 0, dtype=torch.uint8, device=DEV)
    mx.fp8_quantize(x, q[:, :K], s)
    ref, sb = quantized(f64(x))
    assert (s.cpu().numpy() == sb).all()
    got = e4m3(q[:, :K].cpu().numpy())
    np.testing.assert_array_equal(got, ref)
    assert (q[:, K:] == 0x55).all()


def test_quantize_every_border(mx):
    """Every e4m3 value, every midpoint of two neighbours and the fp32 values next to them, at several scales; a
    448 in each block fixes its scale."""
    v = e4m3(np.arange(0x7F))
    mid = (v[1:] + v[:-1]) / 2
    pts = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                          np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64)])
    pts = np.concatenate([pts, -pts])
    pts = np.pad(pts, (0, -len(pts) % 127)).reshape(-1, 127)
    pts = np.concatenate([pts, np.full((len(pts), 1), 448.0)], 1)
    for e in (-100, -3, 0, 5, 110):
        say(f"case: quantize every border at 2^{e}")
        x = torch.from_numpy((pts * 2.0 ** e).astype(np.float32)).to(DEV)
        q = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
        s = torch.empty((len(pts), 1), dtype=torch.uint8, device=DEV)
        mx.fp8_quantize(x, q, s)
        assert (s.cpu().numpy() == e + 127).all()
        np.testing.assert_array_equal(e4m3(q.cpu().numpy()), grid(pts))


def test_no_rows(mx):
    say("case: calls of no rows")
    z = lambda *s, d=torch.float32: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    gamma = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    mx.block_pre_norm(z(0, 64), gamma, n=z(0, 64, d=torch.bfloat16))
    mx.block_post_norm(z(0, 64), z(0, 64), z(0, 64), gamma=gamma)
    mx.fp8_quantize(z(0, 64), z(0, 64, d=torch.uint8), z(0, 1, d=torch.uint8))
    torch.cuda.synchronize()


def test_norms_on_a_side_stream_and_in_a_graph(mx):
    say("case: norms on a side stream and replayed")
    T, H = 6, 1024
    x, y = rows(T, H, torch.float32, 0, seed=1), rows(T, H, torch.float32, 0, seed=2)
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    want_o, want_n = torch.empty_like(x), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    out, n = torch.empty_like(want_o), torch.empty_like(want_n)
    run = lambda o, nn, **kw: mx.block_post_norm(y, x, o, gamma=gamma, next_gamma=gamma, n=nn, **kw)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(out, n, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    run(want_o, want_n)
    assert torch.equal(out, want_o) and torch.equal(n, want_n)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run(out, n)
    for k in range(3):
        x.add_(1.0)
        run(want_o, want_n)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_o) and torch.equal(n, want_n)


def test_rows_past_32_bit_offsets(mx):
    say("case: 300000 rows of 7168 values")
    T, H = 300_000, 7168  # 2.15e9 values
    x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    x.fill_(1.0)
    x[-1] = 3.0
    x[-1, ::2] = -1.0
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    n = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((T, H), dtype=torch.uint8, device=DEV)
    s = torch.zeros((T, H // 128), dtype=torch.uint8, device=DEV)
    mx.block_pre_norm(x, gamma, 0.0, n=n, q=q, q_scale=s)
    check_normed(n[-3:], q[-3:], s[-3:], rms(f64(x[-3:]), 1.0, 0.0), H)
    mx.fp8_quantize(x, q, s)
    ref, sb = quantized(f64(x[-3:]))
    np.testing.assert_array_equal(e4m3(q[-3:].cpu().numpy()), ref)
    assert (s[-3:].cpu().numpy() == sb).all()


def repeated(small, T):
    """Row t of the result is row t % 7 of small."""
    return small.repeat(-(-T // 7), *[1] * (small.dim() - 1))[:T]


# more rows than one launch of 128 (512) threads a row holds
@pytest.mark.parametrize("T,H", [(2 ** 25 + 5, 1), (2 ** 23 + 3, 1032)])
def test_pre_norm_of_many_rows(mx, T, H):
    """A row's result does not depend on the others: seven rows over and over against the seven alone, bit for bit."""
    say(f"case: pre norm T={T} H={H}")
    few = rows(7, H, torch.bfloat16, 0, seed=H)
    gamma = (1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).to(DEV)
    kb = -(-H // 128)
    got = []
    for x in (few.contiguous(), repeated(few, T)):
        t = x.shape[0]
        o = (torch.zeros((t, H), dtype=torch.bfloat16, device=DEV), torch.zeros((t, H), dtype=torch.uint8, device=DEV),
             torch.zeros((t, kb), dtype=torch.uint8, device=DEV))
        mx.block_pre_norm(x, gamma, 1.0, n=o[0], q=o[1], q_scale=o[2])
        got.append(o)
    del x
    for a, b in zip(*got):
        assert torch.equal(repeated(a, T), b)


def test_post_norm_of_many_rows(mx):
    T, H = 2 ** 25 + 5, 2
    say(f"case: post norm T={T} H={H}")
    few = [rows(7, H, torch.float32, 0, seed=i) for i in (1, 2)] + [rows(7, 1, torch.float32, 0, seed=3)]
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    got = []
    for y, r, g in (tuple(v.contiguous() for v in few), tuple(repeated(v, T) for v in few)):
        t = y.shape[0]
        n = torch.zeros((t, H), dtype=torch.bfloat16, device=DEV)
        mx.block_post_norm(y, r, r, gamma=gamma, gate=g, scale=0.5, eps=1.0, next_gamma=gamma, n=n)  # in place
        full = torch.zeros_like(r)
        mx.block_post_norm(y, r, full, gate=y, gate_sigmoid=True)
        got.append((r, n, full))
    for a, b in zip(*got):
        assert torch.equal(repeated(a, T), b)


@pytest.mark.parametrize("T,K", [(2 ** 28 + 17, 1), (2 ** 27 + 9, 130)])
def test_quantize_of_many_blocks(mx, T, K):
    say(f"case: quantize T={T} K={K}")
    few = rows(7, K, torch.bfloat16, 0, seed=K)
    kb = -(-K // 128)
    got = []
    for x in (few.contiguous(), repeated(few, T)):
        o = [torch.zeros((x.shape[0], n), dtype=torch.uint8, device=DEV) for n in (K, kb)]
        mx.fp8_quantize(x, *o)
        got.append(o)
    del x
    for a, b in zip(*got):
        assert torch.equal(repeated(a, T), b)


def test_python_refusals(mx):
    gamma = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((2, 64), device=DEV)
    n = torch.zeros((2, 64), dtype=torch.bfloat16, device=DEV)
    q, s = torch.zeros((2, 64), dtype=torch.uint8, device=DEV), torch.zeros((2, 1), dtype=torch.uint8, device=DEV)
    for bad in (lambda: mx.block_pre_norm(x, gamma),  # nothing asked for
                lambda: mx.block_pre_norm(x, gamma, n=n.float()),
                lambda: mx.block_pre_norm(x, gamma[:63], n=n),
                lambda: mx.block_pre_norm(x, gamma, q=q),
                lambda: mx.block_pre_norm(x.cpu(), gamma, n=n),
                lambda: mx.block_pre_norm(x[:1].expand(2, 64), gamma, n=n),  # rows on top of each other
                lambda: mx.block_pre_norm(x.t().contiguous().t(), gamma, n=n),
                lambda: mx.block_pre_norm(torch.zeros((1, 20000), device=DEV),
                                          torch.ones(20000, dtype=torch.bfloat16, device=DEV),
                                          n=torch.zeros((1, 20000), dtype=torch.bfloat16, device=DEV)),
                lambda: mx.block_post_norm(x, x, n),  # out of another type than the residual
                lambda: mx.block_post_norm(x, x, x, gate=torch.zeros((1, 1), device=DEV)),
                lambda: mx.block_post_norm(x, x, x, gate=torch.zeros((3, 1), device=DEV)),
                lambda: mx.block_post_norm(x, x, x, n=n),
                lambda: mx.fp8_quantize(x, q, s[:1]),
                lambda: mx.fp8_quantize(x.half(), q, s)):
        with pytest.raises((ValueError, mx.MoeError)):
            bad()
