"""The build's check of registers that an LDS read is still to fill: on assembly written for it, and on that of the
kernels with a wait made too weak."""
import os
import re

import pytest

from mxfp4_latent_moe_amd import build
from mxfp4_latent_moe_amd.asm_check import unsafe_reads

READS = """
kernel:                                 ; @kernel
; %bb.0:
	ds_read_b128 v[0:3], v20
	ds_read_b128 v[4:7], v21 offset:0x800
"""
END = "\ts_endpgm\n"


def lines(body):
    return [text for _, _, text in unsafe_reads(READS + body + END)]


@pytest.mark.parametrize("body", [
    "\ts_waitcnt lgkmcnt(1)\n\tv_add_f32_e32 v9, v2, v3\n",
    "\ts_waitcnt vmcnt(3) lgkmcnt(0)\n\tv_mfma_f32_16x16x32_bf16 v[8:11], v[0:3], v[4:7], 0\n",
    "\ts_waitcnt 0\n\tv_mov_b32_e32 v9, v7\n",
    "\tv_mov_b32_e32 v9, v8\n\tv_mov_b32_e32 a0, v30\n\ts_mov_b32 s0, s3\n",  # other registers, a0 is not v0
    "\tds_write_b32 v20, v9\n\ts_waitcnt lgkmcnt(2)\n\tv_mov_b32_e32 v9, v0\n",
    "\ts_waitcnt lgkmcnt(0)\n.LBB0_1:\n\tv_mov_b32_e32 v9, v0\n\ts_cbranch_scc1 .LBB0_1\n",
])
def test_sound(body):
    assert lines(body) == []


@pytest.mark.parametrize("body,at", [
    ("\tv_mov_b32_e32 v9, v0\n\ts_waitcnt lgkmcnt(0)\n", "v_mov_b32_e32 v9, v0"),  # a copy before the wait
    ("\ts_waitcnt lgkmcnt(1)\n\tv_mov_b32_e32 v9, v4\n", "v_mov_b32_e32 v9, v4"),  # the wait covers the first alone
    ("\tscratch_store_dwordx4 off, v[2:5], s0\n", "scratch_store_dwordx4 off, v[2:5], s0"),  # a spill
    ("\ts_waitcnt vmcnt(0)\n\tds_read_b64 v[6:7], v22\n", "ds_read_b64 v[6:7], v22"),  # filled twice
    ("\tds_read_b64 v[10:11], v1\n", "ds_read_b64 v[10:11], v1"),  # as an address
    ("\ts_cbranch_scc1 .LBB0_2\n\ts_waitcnt lgkmcnt(0)\n.LBB0_2:\n\tv_mov_b32_e32 v9, v0\n", "v_mov_b32_e32 v9, v0"),
    # round a loop: the read at its end, the use at its head
    ("\ts_waitcnt lgkmcnt(0)\n.LBB0_3:\n\tv_mov_b32_e32 v9, v12\n\tds_read_b32 v12, v22\n\ts_cbranch_scc0 .LBB0_3\n",
     "v_mov_b32_e32 v9, v12"),
])
def test_unsafe(body, at):
    assert at in lines(body)


def test_the_built_kernels():
    """Sound as built; with each wait in turn one too weak, most of them are not (a wait may be as strong as the one
    before the first use, and then one less changes nothing)."""
    path = os.path.join(build.BUILD, "fp8-hip-amdgcn-amd-amdhsa-gfx950.s")
    if not os.path.exists(path):
        pytest.skip("library not built here")
    with open(path) as f:
        asm = f.read()
    assert unsafe_reads(asm) == []
    text = asm.splitlines()
    # written by hand: a wait on a line of its own inside an inline block
    waits = [i for i, t in enumerate(text) if re.fullmatch(r"\s*s_waitcnt lgkmcnt\(\d+\)", t) and "ASMSTART" in text[i - 1]]
    assert len(waits) > 50
    caught, tried = 0, waits[::len(waits) // 25]
    for i in tried:
        weak = re.sub(r"\((\d+)\)", lambda m: "(%d)" % (int(m[1]) + 1), text[i])
        caught += bool(unsafe_reads("\n".join(text[:i] + [weak] + text[i + 1:])))
    assert caught > len(tried) // 2
