"""Host-side refusals of the block norms, the 8-bit calls and the few-token layer (no GPU needed): every bad
argument gives the documented code before the device is touched."""
import ctypes
import os

import pytest

import synth
from mxfp4_latent_moe_amd import _lib

FAKE = 0x10000  # 16-byte aligned, never dereferenced
F32, BF16 = _lib.MOE_DT_F32, _lib.MOE_DT_BF16
EINVAL, ENOTSUP, EWS = _lib.MOE_EINVAL, _lib.MOE_ENOTSUP, _lib.MOE_EWORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def norm_out(**kw):
    o = _lib.MoeNormOut(FAKE, FAKE, 256, FAKE, 256, FAKE, 2)
    for k, v in kw.items():
        setattr(o, k, v)
    return o


BAD_OUT = [dict(gamma=None), dict(gamma=FAKE + 1), dict(n=None, q=None, q_scale=None), dict(q_scale=None),
           dict(q=None), dict(n=FAKE + 1), dict(ldn=255), dict(ldq=255), dict(ldqs=1)]


def test_pre_norm(lib):
    def call(T=2, H=256, x=FAKE, dt=F32, ldx=256, eps=1e-6, o=None, **kw):
        return lib.moe_block_pre_norm(T, H, x, dt, ldx, eps, norm_out(**kw) if o is None else o, None)

    for bad in (dict(T=-1), dict(H=0), dict(x=None), dict(x=FAKE + 2), dict(dt=BF16, x=FAKE + 1), dict(dt=2),
                dict(ldx=255), dict(eps=-1.0), dict(eps=float("nan")), *BAD_OUT):
        assert call(**bad) == EINVAL, bad
    assert lib.moe_block_pre_norm(2, 256, FAKE, F32, 256, 1e-6, None, None) == EINVAL
    assert call(H=16385, ldx=16385, ldn=16385, ldq=16385, ldqs=129) == ENOTSUP


def test_post_norm(lib):
    def call(next_=None, **kw):
        a = _lib.MoePostNormArgs(2, 256, FAKE, 256, FAKE, 256, FAKE, 256, F32, BF16, FAKE, FAKE, 256,
                                 _lib.MOE_GATE_FULL, F32, 0, 1.0, 1e-6, None)
        for k, v in kw.items():
            setattr(a, k, v)
        if next_ is not None:
            a.next = ctypes.pointer(norm_out(**next_))
        return lib.moe_block_post_norm(a, None)

    assert lib.moe_block_post_norm(None, None) == EINVAL
    for bad in (dict(T=-1), dict(H=0), dict(y=None), dict(resid=None), dict(out=None), dict(y=FAKE + 2),
                dict(resid=FAKE + 1), dict(out=FAKE + 1), dict(gamma=FAKE + 1), dict(ldy=255), dict(ldr=255),
                dict(ldo=255), dict(ldr=512), dict(y_dtype=2), dict(dtype=2), dict(gate_kind=4), dict(gate_kind=-1),
                dict(gate_kind=_lib.MOE_GATE_NONE), dict(gate=None), dict(gate=FAKE + 2), dict(ldg=255),
                dict(gate_kind=_lib.MOE_GATE_TOKEN, ldg=0), dict(gate_dtype=2), dict(gate_sigmoid=2),
                dict(eps=-1.0)):
        assert call(**bad) == EINVAL, bad
    for bad in BAD_OUT:
        assert call(next_=bad) == EINVAL, bad
    big = dict.fromkeys(("H", "ldy", "ldr", "ldo", "ldg"), 16385)
    assert call(**big) == ENOTSUP


def test_fp8_quantize(lib):
    def call(T=2, K=200, x=FAKE, dt=F32, ldx=200, q=FAKE, ldq=200, s=FAKE, lds=2):
        return lib.moe_fp8_quantize(T, K, x, dt, ldx, q, ldq, s, lds, None)

    for bad in (dict(T=-1), dict(K=0), dict(x=None), dict(q=None), dict(s=None), dict(dt=3), dict(ldx=199),
                dict(ldq=199), dict(lds=1), dict(x=FAKE + 2), dict(dt=BF16, x=FAKE + 1)):
        assert call(**bad) == EINVAL, bad
    for k in ((1 << 30) + 1, 2 ** 31 - 1):
        assert call(K=k, ldx=k, ldq=k, lds=k) == ENOTSUP, k


def test_fp8_gemm(lib):
    ws = lib.moe_fp8_gemm_workspace_bytes(2, 300, 400)
    assert ws > 0

    def call(T=2, N=300, K=400, x=FAKE, ldx=400, xs=FAKE, ldxs=4, w=FAKE, sw=FAKE, kind=_lib.MOE_SCALE_F32, out=FAKE,
             dt=F32, ldo=300, acc=0, wsp=FAKE, wsb=ws):
        return lib.moe_fp8_gemm(T, N, K, x, ldx, xs, ldxs, w, sw, kind, out, dt, ldo, acc, wsp, wsb, None)

    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(x=None), dict(xs=None), dict(w=None), dict(sw=None),
                dict(out=None), dict(wsp=None), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(out=FAKE + 2),
                dict(sw=FAKE + 2), dict(wsp=FAKE + 8), dict(ldx=408), dict(ldx=384), dict(ldxs=3), dict(ldo=299),
                dict(kind=2), dict(dt=2), dict(acc=2), dict(acc=1, dt=BF16), dict(dt=BF16, out=FAKE + 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(K=392, ldx=400), dict(K=(1 << 20) + 16, ldx=1 << 21, ldxs=1 << 14), dict(T=(1 << 22) + 1),
                dict(N=(1 << 22) + 1, ldo=1 << 23), dict(ldx=(1 << 22) + 16)):
        assert call(**bad) == ENOTSUP, bad
    assert call(wsb=ws - 1) == EWS
    for T, N, K in ((-1, 1, 16), (1, 0, 16), (1, 1, 0), (1, 1, 24), (1, 1, 1 << 21)):
        assert lib.moe_fp8_gemm_workspace_bytes(T, N, K) == 0
    assert lib.moe_fp8_gemm_workspace_bytes(0, 1, 16) > 0


@pytest.mark.parametrize("T", [1, 2, 64, 300])
def test_fp8_gemm_scale_rows_far_apart(lib, T):
    """A stride of x_scale with which offsets within a work-group's rows pass 32 bits is refused, as one of x is; the
    largest that is taken is looked at no further here (the workspace is too small)."""
    ws = lib.moe_fp8_gemm_workspace_bytes(T, 300, 400)

    def call(ldxs, wsb):
        return lib.moe_fp8_gemm(T, 300, 400, FAKE, 400, FAKE, ldxs, FAKE, FAKE, _lib.MOE_SCALE_F32, FAKE, F32, 300, 0,
                                FAKE, wsb, None)

    assert call(1 << 22, ws - 1) == EWS
    for ldxs in ((1 << 22) + 1, (1 << 32) // 63 + 1, 1 << 32, 1 << 40):
        assert call(ldxs, ws) == ENOTSUP, ldxs


def _shape(**kw):
    sh = synth.K3_SHAPE
    s = _lib.make_shape(sh.hidden, sh.latent, sh.n_experts, sh.top_k, sh.inter, sh.n_shared, sh.shared_inter)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_layer_few(lib):
    s = _shape()
    ws = lib.moe_layer_few_workspace_bytes(s, 4)
    assert ws > lib.moe_layer_few_workspace_bytes(s, 1) > 0

    def weights(**kw):
        lw = _lib.MoeLayerWeights(*[FAKE] * 14)
        for k, v in kw.items():
            setattr(lw, k, v)
        return lw

    def call(s=s, T=4, x=FAKE, lw=None, ids=FAKE, w=FAKE, out=FAKE, wsp=FAKE, wsb=ws, **kw):
        return lib.moe_layer_few(s, T, x, weights(**kw) if lw is None else lw, ids, w, out, wsp, wsb, None)

    for bad in (dict(T=0), dict(x=None), dict(out=None), dict(wsp=None), dict(ids=None), dict(w=None),
                dict(x=FAKE + 8), dict(out=FAKE + 4), dict(wsp=FAKE + 4), dict(ids=FAKE + 2), dict(w=FAKE + 2),
                dict(s=None), dict(s=_shape(top_k=900)), dict(s=_shape(operand_mode=9))):
        assert call(**bad) == EINVAL, bad
    assert lib.moe_layer_few(s, 4, FAKE, None, FAKE, FAKE, FAKE, FAKE, ws, None) == EINVAL
    for name, _ in _lib.MoeLayerWeights._fields_:
        assert call(**{name: None}) == EINVAL, name
        assert call(**{name: FAKE + 1}) == EINVAL, name
    for bad in (dict(T=_lib.MOE_FEW_MAX_T + 1), dict(s=_shape(hidden=7000)), dict(s=_shape(n_experts=2048)),
                dict(s=_shape(latent=128 * 97)), dict(s=_shape(inter=128 * 97)), dict(s=_shape(hidden=128 * 513)),
                dict(s=_shape(shared_inter=128 * 257))):
        assert call(**bad) == ENOTSUP, bad
    assert lib.moe_layer_few_workspace_bytes(_shape(latent=128 * 96, inter=128 * 96, hidden=128 * 512), 4) > 0
    assert call(wsb=ws - 1) == EWS
    assert lib.moe_layer_few_workspace_bytes(s, 0) == 0 and lib.moe_layer_few_workspace_bytes(s, 5) == 0
    # without shared experts their tensors are not looked at
    n = _shape(n_shared=0)
    need = lib.moe_layer_few_workspace_bytes(n, 4)
    assert call(s=n, wsb=need - 1, sh_gate=None, sh_up=None, sh_down=None) == EWS


def test_few_kernel_constants_agree(lib):
    """The binding's token limit is the library's."""
    s = _shape()
    assert lib.moe_layer_few_workspace_bytes(s, _lib.MOE_FEW_MAX_T) > 0
