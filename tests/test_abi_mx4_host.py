"""Host-side refusals of the MXFP4 calls (no GPU needed): every bad argument gives the documented code before the
device is touched."""
import ctypes
import os
import shutil
import subprocess

import pytest

from mxfp4_latent_moe_amd import _lib

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
FAKE = 0x10000  # 16-byte aligned, never dereferenced
F32, BF16, MX4 = _lib.MOE_DT_F32, _lib.MOE_DT_BF16, _lib.MOE_DT_MXFP4
EINVAL, ENOTSUP, EWS = _lib.MOE_EINVAL, _lib.MOE_ENOTSUP, _lib.MOE_EWORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def test_quantize(lib):
    def call(T=2, K=45, x=FAKE, dt=F32, ldx=45, rule=0, q=FAKE, ldq=23, s=FAKE, lds=2):
        return lib.moe_mxfp4_quantize(T, K, x, dt, ldx, rule, q, ldq, s, lds, None)

    for bad in (dict(T=-1), dict(K=0), dict(x=None), dict(q=None), dict(s=None), dict(dt=2), dict(dt=MX4), dict(ldx=44),
                dict(ldq=22), dict(lds=1), dict(rule=2), dict(rule=-1), dict(x=FAKE + 2), dict(dt=BF16, x=FAKE + 1)):
        assert call(**bad) == EINVAL, bad
    for k in ((1 << 30) + 1, 2 ** 31 - 1):
        assert call(K=k, ldx=k, ldq=k, lds=k) == ENOTSUP, k


def test_dequantize(lib):
    def call(T=2, K=45, q=FAKE, ldq=23, s=FAKE, lds=2, out=FAKE, dt=F32, ldo=45):
        return lib.moe_mxfp4_dequantize(T, K, q, ldq, s, lds, out, dt, ldo, None)

    for bad in (dict(T=-1), dict(K=0), dict(out=None), dict(q=None), dict(s=None), dict(dt=2), dict(ldo=44),
                dict(ldq=22), dict(lds=1), dict(out=FAKE + 2), dict(dt=BF16, out=FAKE + 1)):
        assert call(**bad) == EINVAL, bad
    k = (1 << 30) + 1
    assert call(K=k, ldo=k, ldq=k, lds=k) == ENOTSUP


def test_gemm(lib):
    ws = lib.moe_mxfp4_gemm_workspace_bytes(2, 300, 416)
    assert ws > 0

    def call(T=2, N=300, K=416, x=FAKE, ldx=208, xs=FAKE, ldxs=13, w=FAKE, sw=FAKE, out=FAKE, dt=F32, ldo=300, acc=0,
             wsp=FAKE, wsb=ws):
        return lib.moe_mxfp4_gemm(T, N, K, x, ldx, xs, ldxs, w, sw, out, dt, ldo, acc, wsp, wsb, None)

    for bad in (dict(T=-1), dict(N=0), dict(K=0), dict(x=None), dict(xs=None), dict(w=None), dict(sw=None),
                dict(out=None), dict(wsp=None), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(out=FAKE + 2),
                dict(wsp=FAKE + 8), dict(ldx=200), dict(ldx=216), dict(ldxs=12), dict(ldo=299), dict(dt=2), dict(dt=MX4),
                dict(acc=2), dict(acc=1, dt=BF16), dict(dt=BF16, out=FAKE + 1)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(K=400), dict(K=(1 << 20) + 32, ldx=1 << 20, ldxs=1 << 16), dict(T=(1 << 21) + 1),
                dict(N=(1 << 20) + 1, ldo=1 << 21), dict(ldx=(1 << 22) + 16), dict(ldxs=(1 << 22) + 1),
                dict(ldxs=1 << 32)):
        assert call(**bad) == ENOTSUP, bad
    assert call(wsb=ws - 1) == EWS
    for T, N, K in ((-1, 1, 32), (1, 0, 32), (1, 1, 0), (1, 1, 48), (1, 1, 1 << 21)):
        assert lib.moe_mxfp4_gemm_workspace_bytes(T, N, K) == 0
    assert lib.moe_mxfp4_gemm_workspace_bytes(0, 1, 32) > 0
    assert lib.moe_mxfp4_gemm_workspace_bytes(1 << 21, 1 << 12, 1 << 20) > 0
    assert lib.moe_mxfp4_gemm_workspace_bytes(1 << 21, (1 << 12) + 1, 1 << 20) == 0


def test_expert_gemm(lib):
    ws = lib.moe_mxfp4_expert_gemm_workspace_bytes(8, 100, 64, 160)
    assert ws > 0

    def call(wsp=FAKE, wsb=ws, **kw):
        a = _lib.MoeMxfp4ExpertArgs(8, 100, 64, 160, FAKE, FAKE, 80, FAKE, 5, 50, 2, FAKE, FAKE, FAKE, FAKE, FAKE, 4.0,
                                    25.0, None, FAKE, 64, F32, None, 0)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.moe_mxfp4_expert_gemm(a, wsp, wsb, None)

    assert lib.moe_mxfp4_expert_gemm(None, FAKE, ws, None) == EINVAL
    down = dict(w3=None, w3_scale=None, top_k=0, x_rows=100)
    four = dict(out_dtype=MX4, out_scale=FAKE, ldos=2, ldo=32)
    for bad in (dict(n_experts=0), dict(P=-1), dict(N=0), dict(K=0), dict(expert_offsets=None), dict(x=None),
                dict(x_scale=None), dict(w=None), dict(w_scale=None), dict(out=None), dict(wsp=None), dict(w3=None),
                dict(w3_scale=None), dict(out_dtype=2), dict(out_dtype=4), dict(out_scale=FAKE), dict(beta=0.0),
                dict(beta_lin=-1.0), dict(beta=float("nan")), dict(pair_weight=FAKE), dict(top_k=-1),
                dict(sorted_pair=None), dict(x_rows=0), dict(**{**down, "x_rows": 99}), dict(ldx=64), dict(ldx=88),
                dict(ldxs=4), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(w3=FAKE + 8), dict(wsp=FAKE + 8),
                dict(expert_offsets=FAKE + 2), dict(sorted_pair=FAKE + 1), dict(ldo=63), dict(out=FAKE + 2),
                dict(**down, pair_weight=FAKE + 2), dict(**down, pair_weight=FAKE, sorted_pair=None),
                dict(**down, **four), {**four, "out_scale": None}, {**four, "ldo": 24}, {**four, "ldo": 40},
                {**four, "ldos": 1}, {**four, "out": FAKE + 8}):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(n_experts=1025), dict(K=144), dict(P=(1 << 21) + 1), dict(N=(1 << 18) + 1, ldo=1 << 21),
                dict(ldx=(1 << 22) + 16), dict(ldxs=(1 << 22) + 1), dict(x_rows=1 << 30), dict(P=1 << 20, N=1 << 14, ldo=1 << 14),
                dict(x_rows=1 << 21, ldx=1 << 10), {**four, "N": 72, "ldo": 48, "ldos": 3}):
        assert call(**bad) == ENOTSUP, bad
    assert call(wsb=ws - 1) == EWS and call(**down, wsb=ws - 1) == EWS and call(**four, wsb=ws - 1) == EWS
    for E, P, N, K in ((0, 1, 1, 32), (1025, 1, 1, 32), (1, -1, 1, 32), (1, 1, 0, 32), (1, 1, 1, 40), (1, 1 << 22, 1, 32)):
        assert lib.moe_mxfp4_expert_gemm_workspace_bytes(E, P, N, K) == 0
    assert lib.moe_mxfp4_expert_gemm_workspace_bytes(1024, 1 << 15, 1 << 18, 1 << 20) > 0
    assert lib.moe_mxfp4_expert_gemm_workspace_bytes(1024, 1 << 21, 1 << 12, 1 << 20) > 0


def test_struct_layout(tmp_path):
    """The binding's argument block is the header's, field for field."""
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    names = [n for n, _ in _lib.MoeMxfp4ExpertArgs._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"moe_latent.h\"\nint main(void) {\n"
                   + "".join(f'  printf("%zu\\n", offsetof(moe_mxfp4_expert_args, {n}));\n' for n in names)
                   + '  printf("%zu\\n", sizeof(moe_mxfp4_expert_args));\n  return 0;\n}\n')
    subprocess.run([cc, "-I", INCLUDE, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    assert got == [getattr(_lib.MoeMxfp4ExpertArgs, n).offset for n in names] + [ctypes.sizeof(_lib.MoeMxfp4ExpertArgs)]
