"""Limits of the MXFP4 calls that are checked on the host (no GPU needed)."""
import os

import pytest

from mxfp4_latent_moe_amd import _lib

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built")
    return _lib.load()


def test_betas(lib):
    """Gate and up take betas of 2^-100 to 2^100; the down product has none."""
    ws = lib.moe_mxfp4_expert_gemm_workspace_bytes(8, 100, 64, 160)

    def call(wsb=ws, **kw):
        a = _lib.MoeMxfp4ExpertArgs(8, 100, 64, 160, FAKE, FAKE, 80, FAKE, 5, 50, 2, FAKE, FAKE, FAKE, FAKE, FAKE, 4.0,
                                    25.0, None, FAKE, 64, _lib.MOE_DT_F32, None, 0)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.moe_mxfp4_expert_gemm(a, FAKE, wsb, None)

    past = (2.0 ** 101, 2.0 ** 127, float("inf"), 2.0 ** -101, 2.0 ** -140)
    for name in ("beta", "beta_lin"):
        for b in past:
            assert call(**{name: b}) == _lib.MOE_ENOTSUP, (name, b)
        for b in (0.0, -1.0, float("nan")):
            assert call(**{name: b}) == _lib.MOE_EINVAL, (name, b)
        for b in (2.0 ** 100, 2.0 ** -100):  # past this check, to that of the workspace
            assert call(**{name: b}, wsb=ws - 1) == _lib.MOE_EWORKSPACE, (name, b)
    assert call(w3=None, w3_scale=None, beta=float("inf"), beta_lin=0.0, wsb=ws - 1) == _lib.MOE_EWORKSPACE
