"""Sizes that reach every kernel, tile and split that the 8-bit products and the gated feed-forward
block choose from: tests/test_fp8.py holds that they do, tests/test_gpu_product_kernels.py runs them."""
import torch

import post_weight_quantization_gq_amd as gq

U8, F32, BF = torch.uint8, torch.float32, torch.bfloat16

# of each product: rows, d_in, d_out (d_ff), experts (None: one weight)
CASES = {
    "fp8_gemm": [
        (1, 130, 130, None), (1, 2047, 130, None), (13, 8200, 130, None), (1, 130, 8200, None), (3, 8200, 8200, None),
        (56, 520, 1100, 8),                                                         # streamed weights
        (21, 130, 130, None), (21, 2047, 130, None), (21, 1001, 130, None),         # tiles of 32 rows
        (4099, 130, 130, None), (900, 2100, 130, None), (290, 1104, 333, 6),        # 64
        (4099, 130, 130, 130), (1500, 4200, 130, 6), (333, 130, 11008, None), (2050, 5000, 130, None),
        (2050, 130, 2047, 40), (4099, 8200, 130, 40), (1030, 2047, 4200, None)],    # 256
    "fp8_gemm_dx": [
        (1, 130, 130, None), (1, 130, 1104, None), (16, 1001, 2047, None), (56, 264, 520, 8), (4099, 264, 130, 130),
        (1500, 264, 2100, 6), (1500, 264, 1104, 40), (4099, 520, 130, 130), (2050, 33, 4200, 40),
        (1030, 4200, 2047, None)],
    "fp8_ffn_gate": [
        (1, 130, 130, None), (1, 4200, 130, None), (2, 8200, 2100, None), (9, 8200, 130, None), (56, 520, 264, 8),
        (21, 130, 130, None), (21, 2047, 130, None), (21, 1001, 130, None), (900, 130, 520, None),
        (290, 4200, 130, None), (1500, 130, 130, 130), (900, 8200, 130, None), (1500, 130, 333, 130),
        (520, 5000, 333, 6), (2050, 130, 1001, 40), (900, 11008, 520, None)],
    "fp8_ffn_gate_packed": [
        (1, 130, 130, None), (1, 4200, 130, None), (2, 8200, 2100, None), (9, 8200, 130, None), (56, 520, 264, 8),
        (21, 130, 130, None), (21, 520, 130, None), (900, 130, 520, None), (900, 1104, 130, None),
        (1500, 130, 130, 130), (2050, 1001, 264, 40), (333, 264, 4200, None)],
    "ffn_gate": [
        (1, 130, 130, None), (1, 2047, 130, None), (2, 4200, 2100, None), (9, 4200, 130, None), (56, 520, 264, 8),
        (21, 130, 130, None), (21, 1001, 130, None), (900, 130, 520, None), (333, 4200, 130, None),
        (900, 130, 1104, None), (333, 4200, 333, None), (2050, 130, 1001, 40), (1500, 8200, 130, None)],
    "ffn_gate_dx": [
        (1, 130, 130, None), (900, 520, 130, None), (1, 130, 520, None), (4099, 264, 130, 130), (45, 1001, 2047, None),
        (4099, 520, 130, 130), (4099, 264, 1001, None), (56, 264, 520, 8)],
    "ffn_gate_dw": [
        (1, 130, 130, None), (290, 130, 130, None), (1, 130, 8200, 2), (4099, 130, 8200, None), (333, 264, 520, 8)],
}


def types(op):
    """The (scales, output) types of a product."""
    if not op.startswith("fp8"):
        return [(None, BF), (None, F32)]
    return [(s, o) for s in (U8, F32) for o in ((F32,) if op.endswith("packed") else (BF, F32))]


def kernel(op, n, d_in, d_out, experts, scales, out):
    """What a call launches."""
    p = gq.product_plan(op, n, d_in, d_out, experts or 1, scales=scales or U8, dtype=gq.GQ_F32 if out == F32 else gq.GQ_BF16)
    return (op, scales, p["wide"], p["streamed"], p["rows"], p["cols"], p["waves"], p["split"] > 1)
