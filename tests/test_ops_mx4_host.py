"""Checks that the Python calls on MXFP4 rows make before anything is launched (no GPU needed: tensors without memory,
which a call that passes these checks refuses as not on a GPU)."""
import pytest
import torch

import mxfp4_latent_moe_amd as mx

NOT_ON_GPU = "tensors must be on a GPU"


def meta(*shape, dtype=torch.uint8):
    return torch.empty(shape, dtype=dtype, device="meta")


def down(rows, P, pairs, top_k=0, **kw):
    E, N, K = 3, 64, 128
    mx.mxfp4_expert_gemm(meta(rows, K // 2), meta(rows, K // 32), meta(E, N, K // 2), meta(E, N, K // 32),
                         meta(E + 1, dtype=torch.int32), meta(P, N, dtype=torch.float32), meta(1 << 16),
                         sorted_pair=meta(P, dtype=torch.int32), top_k=top_k,
                         pair_weight=meta(*pairs, dtype=kw.get("dtype", torch.float32)))


def test_pair_weight():
    """Rows of x under top_k fix how many pairs there may be; a shorter vector would be read past its end."""
    for pairs in ((39,), (0,), (20,)):
        with pytest.raises(ValueError, match="pair_weight: .* at least 40 values"):
            down(20, 30, pairs, top_k=2)
    with pytest.raises(ValueError, match="pair_weight"):
        down(30, 30, (0,))
    with pytest.raises(ValueError, match="pair_weight"):
        down(20, 30, (40,), top_k=2, dtype=torch.float64)
    for args in ((20, 30, (40,), 2), (20, 30, (20, 2), 2), (20, 30, (41,), 2), (30, 30, (30,), 0), (30, 30, (7,), 0)):
        with pytest.raises(ValueError, match=NOT_ON_GPU):
            down(*args)
