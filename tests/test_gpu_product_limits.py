"""GPU tests of the 8-bit and gate products at sizes where counts pass 32 bits, or outputs what the caches hold."""
import pytest
import torch

import post_weight_quantization_gq_amd as gq
from _product_cases import BF, F32, FP8, U8
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


def integer_rows(device, n, k, seed):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randint(-2, 3, (n, k), generator=g, device=device).to(BF)


@pytest.mark.parametrize("n,d_in,d_ff", [(4099, 128, 8200), (8200, 40, 4099), (300, 128, 1000)])
def test_large_outputs_are_those_of_a_part_of_the_rows(device, n, d_in, d_ff):
    """h of more than 64 MB is stored by other instructions than a smaller one: the same bits, ends of rows included."""
    x, G, U = (integer_rows(device, r, d_in, s) for r, s in ((n, 1), (d_ff, 2), (d_ff, 3)))
    G, U = G * 2.0 ** -4, U * 2.0 ** -4
    h = gq.ffn_gate(x, G, U)
    assert (h.numel() * 2 >= 64 << 20) == (n > 4000)
    XQ, G8, U8_ = gq.fp8_quantize(x), gq.fp8_quantize_weight(G), gq.fp8_quantize_weight(U)
    h8 = gq.fp8_ffn_gate(*XQ, *G8, *U8_, d_in)
    for at in (0, n // 2, n - 290):
        some = slice(at, at + 290)
        assert torch.equal(h[some], gq.ffn_gate(x[some].clone(), G, U))
        assert torch.equal(h8[some], gq.fp8_ffn_gate(XQ[0][some], XQ[1][some], *G8, *U8_, d_in))


@pytest.mark.parametrize("n,d_in,d_ff", [(100, 4100, 8200), (100, 4099, 8190), (100, 333, 1000), (16384, 1024, 1024)])
def test_large_gradients_are_exact(device, n, d_in, d_ff):
    """Weights' gradients of more than 128 MB, smaller ones, and of a split contraction: sums that are exact."""
    x = integer_rows(device, n, d_in, 1)
    a, b = integer_rows(device, n, d_ff, 2), integer_rows(device, n, d_ff, 3)
    got = gq.ffn_gate_dw(a, b, x)
    assert (2 * 2 * d_in * d_ff >= 128 << 20) == (d_in > 4000)
    for d, z in zip(got, (a, b)):
        assert torch.equal(d, (z.float().T @ x.float()).to(BF))
