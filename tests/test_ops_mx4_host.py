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


BIG = 2 ** 32 + 5  # five, to a call that keeps the low 32 bits


def test_sizes_past_32_bits():
    """Sizes that the library's ints cannot hold are refused, not cut to their low bits."""
    f32, bf16 = torch.float32, torch.bfloat16
    calls = [
        lambda: mx.block_pre_norm(meta(BIG, 1, dtype=f32), meta(1, dtype=bf16), n=meta(BIG, 1, dtype=bf16)),
        lambda: mx.block_post_norm(meta(BIG, 1, dtype=f32), meta(BIG, 1, dtype=f32), meta(BIG, 1, dtype=f32)),
        lambda: mx.fp8_quantize(meta(BIG, 1, dtype=f32), meta(BIG, 1), meta(BIG, 1)),
        lambda: mx.fp8_gemm(meta(BIG, 1), meta(BIG, 1), meta(1, 1), meta(1, 1), meta(BIG, 1, dtype=f32), meta(1024)),
        lambda: mx.mxfp4_quantize(meta(BIG, 1, dtype=f32), meta(BIG, 1), meta(BIG, 1)),
        lambda: mx.mxfp4_quantize(meta(1, BIG, dtype=f32), meta(1, BIG // 2 + 1), meta(1, BIG // 32 + 1)),
        lambda: mx.mxfp4_dequantize(meta(BIG, 1), meta(BIG, 1), meta(BIG, 1, dtype=f32)),
        lambda: mx.mxfp4_gemm(meta(BIG, 16), meta(BIG, 1), meta(1, 16), meta(1, 1), meta(BIG, 1, dtype=f32), meta(1024)),
        lambda: mx.mxfp4_gemm(meta(1, 16), meta(1, 1), meta(BIG, 16), meta(BIG, 1), meta(1, BIG, dtype=f32), meta(1024)),
        lambda: mx.mxfp4_gemm(meta(1, 2 ** 31 + 16), meta(1, 2 ** 27 + 1), meta(1, 2 ** 31 + 16), meta(1, 2 ** 27 + 1),
                              meta(1, 1, dtype=f32), meta(1024)),
        lambda: mx.mxfp4_expert_gemm(meta(BIG, 16), meta(BIG, 1), meta(1, 1, 16), meta(1, 1, 1), meta(2, dtype=torch.int32),
                                     meta(4, 1, dtype=f32), meta(1024)),
        lambda: mx.mxfp4_expert_gemm(meta(9, 16), meta(9, 1), meta(1, 1, 16), meta(1, 1, 1), meta(2, dtype=torch.int32),
                                     meta(BIG, 1, dtype=f32), meta(1024)),
        lambda: mx.mxfp4_expert_gemm(meta(9, 16), meta(9, 1), meta(BIG, 1, 16), meta(BIG, 1, 1),
                                     meta(BIG + 1, dtype=torch.int32), meta(4, 1, dtype=f32), meta(1024)),
        lambda: mx.mxfp4_expert_gemm(meta(9, 16), meta(9, 1), meta(1, 1, 16), meta(1, 1, 1), meta(2, dtype=torch.int32),
                                     meta(4, 1, dtype=f32), meta(1024), sorted_pair=meta(4, dtype=torch.int32), top_k=2 ** 32 + 1),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError) as e:
            call()
        assert NOT_ON_GPU not in str(e.value), i
    assert mx.mxfp4_gemm_workspace_bytes(BIG, 32, 32) == mx.mxfp4_gemm_workspace_bytes(32, BIG, 32) == 0
    for sizes in ((BIG, 32, 32, 32), (32, BIG, 32, 32), (32, 32, BIG, 32), (32, 32, 32, 2 ** 32 + 32)):
        assert mx.mxfp4_expert_gemm_workspace_bytes(*sizes) == 0
