"""Sizes of the MXFP4 products that reach every kernel, tile and split the library chooses from:
tests/test_mxfp4_plans.py holds that they do, tests/test_gpu_mxfp4_kernels.py runs them."""
import post_weight_quantization_gq_amd as gq

# op, activations ("mx": packed too), rows, d_in, d_out, experts (None: one weight)
CASES = [
    # weights streamed by waves: 16 and 32 columns, 4 and 8 waves, the contraction whole and split
    ("gemm", "bf16", 1, 520, 48, None), ("gemm", "bf16", 16, 1104, 1001, None),
    ("gemm", "bf16", 16, 4200, 130, None), ("gemm", "bf16", 1, 4096, 4096, None),
    ("gemm", "bf16", 13, 8200, 130, None), ("gemm", "bf16", 3, 28672, 520, None),
    ("gemm", "bf16", 13, 1104, 8192, None), ("gemm", "bf16", 56, 520, 2100, 6),
    ("gemm", "bf16", 1, 4200, 14336, None), ("gemm", "bf16", 64, 4200, 130, 130),
    ("gemm", "f32", 1, 520, 264, None), ("gemm", "f32", 16, 520, 1001, None),
    ("gemm", "f32", 1, 2047, 48, None), ("gemm", "f32", 16, 2048, 1000, None),
    ("gemm", "f32", 8, 4096, 130, None), ("gemm", "f32", 1, 11008, 264, None),
    ("gemm", "f32", 1, 1024, 14336, None), ("gemm", "f32", 13, 640, 11008, None),
    ("gemm", "f32", 1, 2048, 14336, None), ("gemm", "f32", 56, 2047, 264, 40),
    ("gemm_mx", "mx", 8, 1100, 130, None), ("gemm_mx", "mx", 21, 2100, 264, 6),
    ("gemm_mx", "mx", 16, 4096, 1408, None), ("gemm_mx", "mx", 1, 4200, 264, None),
    ("gemm_mx", "mx", 13, 8200, 513, None), ("gemm_mx", "mx", 8, 28672, 48, 6),
    ("gemm_mx", "mx", 13, 1104, 8192, None), ("gemm_mx", "mx", 56, 520, 2100, 6),
    ("gemm_mx", "mx", 8, 28672, 8192, None), ("gemm_mx", "mx", 40, 4200, 264, 40),
    # tiles of 32 rows
    ("gemm", "bf16", 21, 640, 11008, None), ("gemm", "bf16", 290, 640, 1000, 130),
    ("gemm", "bf16", 24, 2100, 1408, None), ("gemm", "bf16", 100, 14336, 48, 6),
    ("gemm", "f32", 30, 520, 8192, None), ("gemm", "f32", 56, 4096, 513, 40),
    ("gemm", "f32", 16, 11008, 48, None), ("gemm", "f32", 128, 640, 513, 6),
    ("gemm_mx", "mx", 21, 640, 11008, None), ("gemm_mx", "mx", 256, 640, 1000, 130),
    ("gemm_mx", "mx", 21, 2100, 264, None), ("gemm_mx", "mx", 190, 2048, 264, 6),
    # 64 rows
    ("gemm", "bf16", 190, 520, 4096, None), ("gemm", "bf16", 290, 1104, 4603, 6),
    ("gemm", "bf16", 520, 2047, 264, None), ("gemm", "bf16", 256, 520, 513, 6),
    ("gemm", "f32", 700, 1104, 2100, None), ("gemm", "f32", 1500, 4200, 513, 6),
    ("gemm", "f32", 190, 2100, 130, None), ("gemm", "f32", 333, 4200, 130, 6),
    ("gemm_mx", "mx", 2050, 640, 1000, None), ("gemm_mx", "mx", 290, 1104, 4603, 6),
    ("gemm_mx", "mx", 520, 2047, 264, None), ("gemm_mx", "mx", 256, 520, 513, 6),
    ("gemm_dx", "bf16", 190, 4096, 640, None), ("gemm_dx", "bf16", 256, 4000, 1100, 6),
    ("gemm_dx", "bf16", 3, 2048, 2047, None), ("gemm_dx", "bf16", 8, 4000, 520, 6),
    ("gemm_dx", "f32", 290, 264, 1104, 130), ("gemm_dx", "f32", 4, 3712, 5120, None),
    ("gemm_dx", "f32", 90, 513, 4096, None), ("gemm_dx", "f32", 3, 1000, 2100, 6),
    # 128 rows
    ("gemm", "bf16", 2048, 4096, 4096, None), ("gemm", "bf16", 900, 2047, 4603, None),
    ("gemm", "bf16", 1500, 2100, 2100, 6), ("gemm", "f32", 700, 2047, 4000, None),
    ("gemm", "f32", 4000, 2047, 264, 40), ("gemm_mx", "mx", 900, 2100, 4603, None),
    ("gemm_mx", "mx", 2050, 2047, 2048, 6), ("gemm_dx", "bf16", 900, 2100, 520, None),
    ("gemm_dx", "bf16", 4000, 513, 1104, 40), ("gemm_dx", "bf16", 333, 4603, 2047, None),
    ("gemm_dx", "bf16", 700, 2100, 1100, 6), ("gemm_dx", "f32", 520, 4096, 1100, 6),
    ("gemm_dx", "f32", 2050, 1000, 640, None), ("gemm_dx", "f32", 4000, 130, 2047, 40),
    # 256 rows
    ("gemm", "bf16", 900, 1104, 14336, None), ("gemm", "bf16", 2050, 1100, 4000, 6),
    ("gemm", "f32", 2000, 2100, 4603, None), ("gemm", "f32", 900, 520, 4000, 6),
    ("gemm", "f32", 2048, 4096, 2048, None), ("gemm", "f32", 1030, 2047, 4000, None),
    ("gemm", "f32", 1500, 1104, 1408, 6), ("gemm_mx", "mx", 900, 1104, 14336, None),
    ("gemm_mx", "mx", 1030, 2100, 5000, 6), ("gemm_dx", "bf16", 1500, 4603, 1100, None),
    ("gemm_dx", "bf16", 900, 4000, 1104, 6), ("gemm_dx", "bf16", 520, 5000, 2100, None),
    ("gemm_dx", "bf16", 1030, 2048, 1100, 6), ("gemm_dx", "f32", 2050, 4603, 640, None),
    ("gemm_dx", "f32", 900, 4000, 520, 6), ("gemm_dx", "f32", 700, 4096, 1100, None),
    ("gemm_dx", "f32", 2050, 2048, 1100, 6),
    # two products: full rounds of large tiles, and the rows behind them
    ("gemm", "bf16", 3861, 520, 4200, None), ("gemm", "f32", 4200, 333, 4200, None),
    ("gemm_mx", "mx", 3856, 520, 4200, None), ("gemm_dx", "bf16", 4200, 4200, 333, None),
]


def kernels(op, dtype, n, d_in, d_out, experts):
    """What a call launches: for each of its one or two products (op, planes, streamed, rows and
    columns of a tile, waves, whether it is split)."""
    found = set()
    while n:
        p = gq.mxfp4_plan(op, n, d_in, d_out, experts, gq.GQ_F32 if dtype == "f32" else gq.GQ_BF16)
        found.add((op, p["planes"], p["streamed"], p["rows"], p["cols"], p["waves"], p["split"] > 1))
        n -= p["first_rows"]
    return found
