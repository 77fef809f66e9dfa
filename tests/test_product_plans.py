"""How 8-bit products and those of the gated feed-forward block are planned, from their sizes alone."""
import pytest
import torch

import post_weight_quantization_gq_amd as gq

F32 = torch.float32


@pytest.mark.parametrize("op", ["fp8_gemm", "fp8_ffn_gate", "fp8_ffn_gate_packed", "ffn_gate"])
def test_every_part_of_a_streamed_contraction_has_a_line(op):
    """A line is 128 bytes of a weight's row; the waves of all parts take equal runs of them, the last ones what is left."""
    split = set()
    for n in (1, 8, 16):
        for d_in in [*range(1100, 34000, 100), *range(2048, 33000, 128), 65536, 100000, 131072]:
            lines = -(-d_in // (64 if op == "ffn_gate" else 128))
            for d_out in (1, 130, 256, 512, 1000, 2048, 4100):
                for experts in (1, 4):
                    p = gq.product_plan(op, n, d_in, d_out, experts, dtype=gq.GQ_F32)
                    if p["streamed"]:
                        run = -(-lines // (p["waves"] * p["split"]))
                        assert (p["split"] - 1) * p["waves"] * run < lines, (n, d_in, d_out, experts)
                        split.add(p["split"])
    assert len(split) > 4 and max(split) <= 16


@pytest.mark.parametrize("op", ["gemm", "gemm_mx"])
def test_every_part_of_a_streamed_mxfp4_contraction_has_a_piece(op):
    """A piece is 512 values of a row, 256 where the activations are three planes."""
    split = set()
    for n in (1, 8, 16):
        for d_in in [*range(1100, 34000, 100), *range(2048, 33000, 128), 65536, 100000]:
            for d_out in (1, 130, 256, 512, 1000, 2048, 4100):
                for dtype in (gq.GQ_F32, gq.GQ_BF16):
                    p = gq.mxfp4_plan(op, n, d_in, d_out, dtype=dtype)
                    if p["streamed"]:
                        pieces = -(-d_in // (256 if p["planes"] == 3 else 512))
                        run = -(-pieces // (p["waves"] * p["split"]))
                        assert (p["split"] - 1) * p["waves"] * run < pieces or p["split"] == 1, (n, d_in, d_out, dtype)
                        split.add(p["split"])
    assert len(split) > 3
