"""GPU tests of 8-bit products at the sizes where a launch's counts pass 32 bits."""
import pytest
import torch

import post_weight_quantization_gq_amd as gq
from _product_cases import F32, FP8, U8
from test_gpu_product_kernels import packed_rows, packed_weight

pytestmark = pytest.mark.gpu


def test_a_streamed_launch_of_more_than_2_to_32_lanes(device):
    """4096 experts by 4096 blocks of 256 lanes, of 64 GiB of codes: the first and the last expert's outputs."""
    E, m, k, n = 4096, 1 << 17, 128, 40
    p = gq.product_plan("fp8_gemm", n, k, m, E)
    assert p["streamed"] and p["cols"] == 32 and m // 32 * E * 64 * p["waves"] >= 1 << 32
    Q = torch.zeros(E, m, k, dtype=U8, device=device).view(FP8)
    S = torch.full((E, m // 128, 1), 127, dtype=U8, device=device)
    q, s, w = packed_weight(device, (), m, k, U8, 2, seed=2)
    for e in (0, E - 1):
        Q.view(U8)[e], S[e] = q.view(U8), s + (e > 0)
    XQ, XS, x = packed_rows(device, n, k, U8, seed=1)
    offsets = torch.tensor([0] + [n // 4] * (E // 2) + [n // 2] * (E // 2 - 1) + [n], device=device)
    y = gq.fp8_gemm(XQ, XS, Q, S, k, offsets=offsets, out_dtype=F32)
    want = x @ w.T
    want[n // 4:n // 2] = 0
    want[n // 2:] *= 2
    assert torch.equal(y.double(), want)
