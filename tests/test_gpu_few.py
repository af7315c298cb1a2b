"""The layer for a few tokens in one call, against the float64 oracle.

Tolerance.  Every product takes its operands at fp32 precision and sums in
fp32.  Along the longest path (z, gate or up, down, combine, norm, up_proj) a
value passes five sums; one of n terms of random signs that a wave adds in n /
32 steps and eight waves join is off by about sqrt(n / 32 + 8) 2^-24 of its
root mean square, at most 24 2^-24 here (n <= 7168), and five of them with the
elementwise steps between stay under 200 2^-24 = 1.2e-5 of the rms in the
mean square; the largest of some thousand values is within 4 of these.
"""
import numpy as np
import pytest
import torch

from synth.device import to_dev, to_dev_bf16
from synth.inputs import LayerShape
from oracle import layer
from gpu_common import GAP_EXCLUDE, rel_max_err, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 4 * 1.2e-5


@pytest.fixture(scope="module")
def mx():
    import mxfp4_latent_moe_amd as mx
    mx.load()
    return mx


def bits(a):
    """bf16 bit patterns, rounded to nearest even."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def make(sh, seed, bias_std=0.05):
    rng = np.random.default_rng(seed)
    S = sh.n_shared * sh.shared_inter
    n = lambda *s, std=1.0: rng.normal(size=s) * std  # noqa: E731
    dense = {"w_router": bits(n(sh.n_experts, sh.hidden, std=0.85 / sh.hidden ** 0.5)),
             "w_down": bits(n(sh.latent, sh.hidden, std=sh.hidden ** -0.5)),
             "w_up": bits(n(sh.hidden, sh.latent, std=sh.latent ** -0.5)),
             "gamma": bits(1 + 0.1 * n(sh.latent)),
             "sh_gate": bits(n(S, sh.hidden, std=sh.hidden ** -0.5)),
             "sh_up": bits(n(S, sh.hidden, std=sh.hidden ** -0.5)),
             "sh_down": bits(n(sh.hidden, S, std=max(S, 1) ** -0.5))}
    bias = (n(sh.n_experts) * bias_std).astype(np.float32)
    stack = {}
    for m, (N, K) in {"w1": (sh.inter, sh.latent), "w3": (sh.inter, sh.latent), "w2": (sh.latent, sh.inter)}.items():
        e = 127 - round(np.log2(2.75 * K ** 0.5))
        stack[m + "_packed"] = rng.integers(0, 256, (sh.n_experts, N, K // 2), dtype=np.uint8)
        stack[m + "_scale"] = rng.integers(e - 1, e + 2, (sh.n_experts, N, K // 32)).astype(np.uint8)
    return dense, bias, stack


def upload(dense, bias, stack):
    w = {k: to_dev_bf16(v, DEV) for k, v in dense.items()}
    w["bias"] = to_dev(bias, DEV)
    w.update({k: to_dev(v, DEV) for k, v in stack.items()})
    return w


def oracle(x_bits, dense, bias, stack, sh):
    cache = layer.ExpertCache(lambda e: {k: v[e] for k, v in stack.items()})
    return layer.layer_forward(x_bits, dense, bias, cache, sh)


def tokens(sh, T, seed):
    return bits(np.random.default_rng(seed).normal(size=(T, sh.hidden)))


def check(b, ref, x_bits, moe):
    ids, wts, out = (b[k].cpu().numpy() for k in ("topk_ids", "topk_w", "out"))
    ok = ref["gap"] >= GAP_EXCLUDE
    assert ok.any()
    assert (ids[ok] == ref["ids"][ok]).all()
    # a weight is a score over a sum of at most 32: its roundings, and those of its logit's sum
    np.testing.assert_allclose(wts[ok], ref["weights"][ok], rtol=2e-5, atol=1e-7)
    err = rel_max_err(out[ok], ref["out"][ok])
    say(f"  max|gpu-oracle|/rms = {err:.2e}")
    assert err <= TOL


SHAPES = [LayerShape(256, 128, 32, 4, 128, 1, 128),      # every expert product one K step
          LayerShape(384, 256, 62, 7, 384, 2, 192),      # E and k odd, K steps not shared evenly
          LayerShape(128, 128, 5, 5, 128, 0, 0),         # every expert, no shared ones
          LayerShape(1024, 640, 33, 1, 256, 1, 1152),    # one expert a token, latent no multiple of 256
          LayerShape(2048, 2048, 64, 4, 1536, 2, 384),
          LayerShape(512, 1152, 200, 32, 640, 1, 256),   # the most pairs
          LayerShape(256, 3200, 40, 2, 256, 0, 0),       # few long rows: K over a work-group's waves, gate/up
          LayerShape(128, 256, 24, 1, 2688, 1, 128)]     # and down


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("sh", SHAPES, ids=lambda s: f"H{s.hidden}L{s.latent}E{s.n_experts}k{s.top_k}")
def test_against_oracle(mx, sh, T):
    say(f"case: few tokens T={T} {sh}")
    dense, bias, stack = make(sh, seed=sh.hidden + sh.latent)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    x = tokens(sh, T, seed=T)
    xd = to_dev_bf16(x, DEV)
    b = moe.forward_few(xd)
    check(b, oracle(x, dense, bias, stack, sh), x, moe)
    # the same again, over a workspace of garbage
    first = b["out"].clone()
    b["ws"].fill_(0xFF)
    b["out"].fill_(float("nan"))
    moe.forward_few(xd)
    assert torch.equal(b["out"], first)


@pytest.mark.parametrize("sh", [LayerShape(128, 12288, 6, 2, 128, 1, 128), LayerShape(128, 128, 6, 3, 12288, 0, 0)],
                         ids=["latent", "inter"])
def test_longest_rows(mx, sh):
    """The longest rows whose columns stay in LDS: one work-group a CU."""
    say(f"case: few tokens {sh}")
    dense, bias, stack = make(sh, seed=3)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    for T in (1, 4):
        x = tokens(sh, T, seed=30 + T)
        check(moe.forward_few(to_dev_bf16(x, DEV)), oracle(x, dense, bias, stack, sh), x, moe)


# K over a work-group's waves, where the sums and the columns take more than 64 KB of LDS together, and more than 60
# for the columns alone; gate/up and down
SPLIT_LONG = [LayerShape(128, 4224, 10, 2, 256, 0, 0), LayerShape(128, 8192, 6, 2, 256, 1, 128),
              LayerShape(128, 256, 10, 1, 4224, 1, 128), LayerShape(128, 256, 6, 2, 8192, 0, 0)]


@pytest.mark.parametrize("sh", SPLIT_LONG + SHAPES[-2:], ids=lambda s: f"L{s.latent}I{s.inter}")
def test_split_rows(mx, sh):
    """Long rows split over the waves against the oracle; a token's result is the same alone and in company."""
    say(f"case: few tokens, rows split over the waves, {sh}")
    dense, bias, stack = make(sh, seed=17)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    x = tokens(sh, 4, 18)
    ref = oracle(x, dense, bias, stack, sh)
    alone = []
    for t in range(4):
        alone.append(moe.forward_few(to_dev_bf16(x[t:t + 1], DEV))["out"][0].clone())
    for T in (1, 2, 3, 4):
        b = moe.forward_few(to_dev_bf16(x[:T], DEV))
        check(b, {k: ref[k][:T] for k in ("ids", "weights", "out", "gap")}, x[:T], moe)
        for t in range(T):
            assert torch.equal(b["out"][t], alone[t])


@pytest.mark.parametrize("sh", [LayerShape(65536, 128, 6, 2, 128, 1, 128), LayerShape(128, 128, 6, 2, 128, 1, 65536),
                                LayerShape(128, 128, 1024, 32, 128, 0, 0)], ids=["hidden", "shared", "experts"])
def test_largest_sizes(mx, sh):
    """The widest hidden and shared layers (one or two sums of 65536 terms, 46 2^-24 each by the rule above, beside
    short ones of under 4: no more than five of 24), and the most experts and choices."""
    say(f"case: few tokens {sh}")
    dense, bias, stack = make(sh, seed=19)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    for T in (1, 4):
        x = tokens(sh, T, seed=60 + T)
        check(moe.forward_few(to_dev_bf16(x, DEV)), oracle(x, dense, bias, stack, sh), x, moe)


def test_without_the_routing(mx):
    """The call that does not ask for ids and weights."""
    sh = SHAPES[1]
    say("case: few tokens, ids and weights not asked for")
    w = upload(*make(sh, seed=23))
    shape = mx.shape_of(sh)
    x = to_dev_bf16(tokens(sh, 3, 2), DEV)
    want = mx.LatentMoE(shape, w, DEV).forward_few(x)["out"]
    out = torch.empty_like(want)
    ws = torch.full((mx.ops.layer_few_workspace_bytes(shape, 3),), 0xFF, dtype=torch.uint8, device=DEV)
    mx.ops.layer_few(shape, x, mx.ops.layer_weights(w), None, None, out, ws)
    assert torch.equal(out, want)


def test_first_call_in_a_capture(mx):
    """Buffers made while a graph is captured serve its replays and eager calls after it."""
    sh = SHAPES[1]
    say("case: few tokens, the first call captured")
    w = upload(*make(sh, seed=24))
    moe, eager = (mx.LatentMoE(mx.shape_of(sh), w, DEV) for _ in range(2))
    x = to_dev_bf16(tokens(sh, 2, 7), DEV)
    eager.forward_few(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = moe.forward_few(x)
    for k in range(3):
        x.copy_(to_dev_bf16(tokens(sh, 2, 200 + k), DEV))
        want = eager.forward_few(x)["out"].clone()
        b["out"].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["out"], want)
        b["out"].fill_(float("nan"))
        assert moe.forward_few(x)["out"] is b["out"]
        torch.cuda.synchronize()
        assert torch.equal(b["out"], want)


def test_matches_the_chain_of_calls(mx):
    sh = SHAPES[4]
    dense, bias, stack = make(sh, seed=11)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    for T in (1, 4):
        say(f"case: few tokens against forward(), T={T}")
        x = to_dev_bf16(tokens(sh, T, 20 + T), DEV)
        ref = {k: v.cpu() for k, v in moe.forward(x).items() if k in ("topk_ids", "topk_w", "out", "gap")}
        b = moe.forward_few(x)
        assert (ref["gap"] > GAP_EXCLUDE).all()
        assert torch.equal(b["topk_ids"].cpu(), ref["topk_ids"])
        torch.testing.assert_close(b["topk_w"].cpu(), ref["topk_w"], rtol=2e-5, atol=1e-7)
        # forward() rounds z, h and the normed latent to two bf16 terms, 2^-17 each
        assert rel_max_err(b["out"].cpu().numpy(), ref["out"].numpy().astype(np.float64)) <= TOL + 1e-4


def test_tokens_that_share_experts(mx):
    """Tokens alike: a chosen expert serves several columns, in one entry of the list or two; rows are equal bit for
    bit."""
    sh = SHAPES[1]
    say("case: few tokens, all alike")
    dense, bias, stack = make(sh, seed=5)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    one = tokens(sh, 1, 9)
    x = np.repeat(one, 4, 0)
    x[2] = tokens(sh, 1, 10)[0]
    b = moe.forward_few(to_dev_bf16(x, DEV))
    check(b, oracle(x, dense, bias, stack, sh), x, moe)
    assert torch.equal(b["out"][0], b["out"][1]) and torch.equal(b["out"][0], b["out"][3])
    # a token's result does not depend on its company
    alone = moe.forward_few(to_dev_bf16(one, DEV))["out"]
    assert torch.equal(alone[0], b["out"][0])


def test_exact_ties_and_masked_experts(mx):
    """Scores exact on both sides (logits -120, 0, 20; biases from -inf to 1/2): ids and weights equal the oracle's."""
    sh = LayerShape(256, 128, 200, 16, 128, 0, 0)
    say("case: few tokens, exact ties and -inf biases")
    dense, bias, stack = make(sh, seed=6)
    rng = np.random.default_rng(8)
    dense["w_router"] = bits(rng.choice([-120.0, 0.0, 20.0], size=(200, 256), p=[0.3, 0.5, 0.2]))
    bias = rng.choice(np.array([-np.inf, -1, -0.5, 0, 0.5], np.float32), size=200, p=[0.1, 0.2, 0.2, 0.3, 0.2])
    x = np.zeros((4, 256), np.float32)
    x[np.arange(4), rng.integers(0, 256, 4)] = 1.0
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias.astype(np.float32), stack), DEV)
    b = moe.forward_few(to_dev_bf16(bits(x), DEV))
    ref = oracle(bits(x), dense, bias, stack, sh)
    assert (b["topk_ids"].cpu().numpy() == ref["ids"]).all()
    np.testing.assert_allclose(b["topk_w"].cpu().numpy(), ref["weights"], rtol=1e-6)
    assert rel_max_err(b["out"].cpu().numpy(), ref["out"]) <= TOL


def test_zero_and_nan_tokens(mx):
    sh = SHAPES[0]
    say("case: few tokens, a row of zeros and a row with NaN")
    dense, bias, stack = make(sh, seed=7)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    x = tokens(sh, 4, 3)
    clean = moe.forward_few(to_dev_bf16(x, DEV))["out"].clone()
    x[1] = 0
    x[2, 7] = 0x7FC0
    b = moe.forward_few(to_dev_bf16(x, DEV))
    out = b["out"]
    # z = 0 gives h = 0 and y = 0; 0 / sqrt(0 + eps) = 0
    assert (out[1] == 0).all()
    assert torch.isnan(out[2]).all()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    ids = b["topk_ids"].cpu().numpy()
    assert ((ids >= 0) & (ids < sh.n_experts)).all()


def test_streams_at_once(mx):
    """Calls of several layer objects on several streams at once, beside other work: more work-groups than the card
    holds, so that some of each kernel start late."""
    sh = SHAPES[4]
    n = 4
    say(f"case: few tokens, {n} calls at once")
    made = [make(sh, seed=30 + i) for i in range(n)]
    moes = [mx.LatentMoE(mx.shape_of(sh), upload(*m), DEV) for m in made]
    xs = [to_dev_bf16(tokens(sh, 1 + i, 40 + i), DEV) for i in range(n)]
    want = [m.forward_few(x)["out"].clone() for m, x in zip(moes, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(n)]
    busy = torch.randn(2048, 2048, device=DEV)
    for rep in range(10):
        for m, x, s in zip(moes, xs, streams):
            m.forward_few(x, stream=s)
        busy = busy @ busy * 1e-3
    torch.cuda.synchronize()
    for m, x, w in zip(moes, xs, want):
        assert torch.equal(m.forward_few(x)["out"], w)
    for m, x, w, s in zip(moes, xs, want, streams):
        b = m.forward_few(x, stream=s)
        s.synchronize()
        assert torch.equal(b["out"], w)


def test_graph_replays(mx):
    sh = SHAPES[1]
    say("case: few tokens, captured and replayed")
    dense, bias, stack = make(sh, seed=12)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    eager = mx.LatentMoE(mx.shape_of(sh), moe.w, DEV)
    x = to_dev_bf16(tokens(sh, 3, 1), DEV)
    b = moe.forward_few(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.forward_few(x)
    for k in range(4):
        x.copy_(to_dev_bf16(tokens(sh, 3, 100 + k), DEV))
        want = eager.forward_few(x)["out"].clone()
        b["out"].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["out"], want)


def test_block_around_the_layer(mx):
    """As a decoder runs it: pre-norm, the layer, post-norm with gate and residual scale and the next pre-norm."""
    sh = SHAPES[1]
    say("case: pre-norm, few-token layer, post-norm")
    T, H = 3, sh.hidden
    dense, bias, stack = make(sh, seed=13)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    g = torch.Generator().manual_seed(4)
    resid = torch.randn(T, H, generator=g).to(DEV)
    g1, g2, g3 = ((1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(3))
    gate = torch.randn(T, 1, generator=g).to(DEV)
    n, nn = (torch.empty((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.empty_like(resid)
    mx.block_pre_norm(resid, g1, 1e-6, n=n)
    y = moe.forward_few(n)["out"]
    mx.block_post_norm(y, resid, out, gamma=g2, gate=gate, gate_sigmoid=True, scale=0.5, next_gamma=g3, n=nn)
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    rms = lambda v, gm: v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * f(gm)  # noqa: E731
    nb = n.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.abs(f(n) - rms(f(resid), g1)).max() <= 2.0 ** -8 * np.abs(f(n)).max() * 1.01
    ref = oracle(nb, dense, bias, stack, sh)
    assert (ref["gap"] >= GAP_EXCLUDE).all()
    want = f(resid) + 0.5 / (1 + np.exp(-f(gate))) * rms(ref["out"], g2)
    # the branch has an rms of about half: the layer's tolerance through the norm
    assert np.abs(f(out) - want).max() <= 2 * TOL
    assert np.abs(f(nn) - rms(want, g3)).max() <= (2.0 ** -8 + 4 * TOL) * np.abs(f(nn)).max() * 1.01


def test_python_refusals(mx):
    sh = SHAPES[0]
    dense, bias, stack = make(sh, seed=1)
    moe = mx.LatentMoE(mx.shape_of(sh), upload(dense, bias, stack), DEV)
    x = to_dev_bf16(tokens(sh, 5, 1), DEV)
    for bad in (x, x[:0], x[:2, :128], x[:2].float(), x[:2].cpu(), x[::2][:2]):
        with pytest.raises(ValueError):
            moe.forward_few(bad)


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def apart(a, b):
    return all(hi <= lo2 or hi2 <= lo for lo, hi in a for lo2, hi2 in b)


def test_buffers_follow_the_streams_of_the_calls(mx):
    """The first call for a token count on a side stream takes no memory whose last use may be pending on the current
    stream; buffers of a dropped layer object are not handed out while a stream that a call ran on still uses them."""
    sh = SHAPES[1]
    say("case: few tokens, buffers and streams")
    made = make(sh, seed=21)
    w = upload(*made)
    x = to_dev_bf16(tokens(sh, 2, 5), DEV)
    want = mx.LatentMoE(mx.shape_of(sh), w, DEV).forward_few(x)["out"].clone()
    ws = mx.ops.layer_few_workspace_bytes(mx.shape_of(sh), 2)
    sizes = [2 * sh.top_k * 4] * 2 + [2 * sh.hidden * 4, ws]
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()

    def blocks():
        return [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]

    free = blocks()
    at = spans(free)
    del free  # the current stream's to use again
    moe = mx.LatentMoE(mx.shape_of(sh), w, DEV)
    b = moe.forward_few(x, stream=one)
    assert apart(spans(b.values()), at)
    one.synchronize()
    assert torch.equal(b["out"], want)
    # a call on a second stream, behind other work there; the layer object goes while that is pending
    with torch.cuda.stream(two):
        torch.cuda._sleep(200_000_000)
    moe.forward_few(x, stream=two)
    at = spans(b.values())
    del moe, b
    with torch.cuda.stream(one):
        new = blocks()
    pending = not two.query()
    assert pending and apart(spans(new), at)
    torch.cuda.synchronize()
    # without a stream: the one that is current, as it changes
    moe = mx.LatentMoE(mx.shape_of(sh), w, DEV)
    for s in (one, two, one):
        with torch.cuda.stream(s):
            b = moe.forward_few(x)
        s.synchronize()
        assert torch.equal(b["out"], want)


@pytest.mark.parametrize("T", [2, 96])
def test_buffers_of_the_chain_of_calls(mx, T):
    """As test_buffers_follow_the_streams_of_the_calls, for forward()."""
    sh = SHAPES[1]
    say(f"case: forward(), buffers and streams, T={T}")
    w = upload(*make(sh, seed=22))
    x = to_dev_bf16(tokens(sh, T, 6), DEV)
    first = mx.LatentMoE(mx.shape_of(sh), w, DEV).forward(x)
    want = first["out"].clone()
    sizes = [t.numel() * t.element_size() for t in first.values()]
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    del first
    torch.cuda.empty_cache()

    def blocks():
        return [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]

    free = blocks()
    at = spans(free)
    del free
    moe = mx.LatentMoE(mx.shape_of(sh), w, DEV)
    b = moe.forward(x, stream=one)
    assert apart(spans(b.values()), at)
    one.synchronize()
    assert torch.equal(b["out"], want)
    with torch.cuda.stream(two):
        torch.cuda._sleep(200_000_000)
    moe.forward(x, stream=two)
    at = spans(b.values())
    del moe, b
    with torch.cuda.stream(one):
        new = blocks()
    pending = not two.query()
    assert pending and apart(spans(new), at)
    torch.cuda.synchronize()


@pytest.mark.slow
@pytest.mark.parametrize("T", [1, 4])
def test_full_shape(mx, T):
    import synth
    from synth.device import upload_weights
    from gpu_common import raw_expert
    wl = synth.workload("decode")
    say(f"case: few tokens at full shape, T={T}")
    w = upload_weights(wl, DEV)
    moe = mx.LatentMoE(mx.shape_of(wl.shape), w, DEV)
    x = synth.gen_tokens(wl)[:T]
    b = moe.forward_few(to_dev_bf16(x, DEV))
    torch.cuda.synchronize()
    from gpu_common import oracle_layer_threaded
    ref = oracle_layer_threaded(wl, x, synth.gen_dense(wl), synth.gen_bias(wl))
    check(b, ref, x, moe)
