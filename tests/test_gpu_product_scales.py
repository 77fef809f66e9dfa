"""GPU tests of the scales of 8-bit products: exponents whose sum passes what float32 holds, NaN at streamed row
counts, any place in memory.

A scale byte s stands for 2^(s - 127), so a block's sum takes the exponent of both its bytes.  Sums here are of
few small integers, exact in float32, and so is their product with a power of two where the result is a number of the
normal range: results are compared for equality.
"""
import pytest
import torch

import post_weight_quantization_gq_amd as gq
from _product_cases import BF, F32, FP8, U8, counts
from _product_kernels import CASES

pytestmark = pytest.mark.gpu

ROWS = [(5, True), (300, False)]                           # streamed, by tiles
OPS = ["gemm", "dx", "gate", "packed"]


def integers(device, *shape, seed):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device=device)


def call(op, XQ, XS, Q, S, d_in, out):
    """The product, as values; the gate's with both weights the same."""
    if op == "gemm":
        return gq.fp8_gemm(XQ, XS, Q, S, d_in, out_dtype=out)
    if op == "dx":
        return gq.fp8_gemm_dx(XQ, XS, Q, S, d_in, out_dtype=out)
    if op == "gate":
        return gq.fp8_ffn_gate(XQ, XS, Q, S, Q, S, d_in, out_dtype=out)
    HQ, HS = gq.fp8_ffn_gate(XQ, XS, Q, S, Q, S, d_in, packed=True)
    return gq.fp8_dequantize(HQ, HS, Q.shape[0], dtype=F32)


def plan(op, n, d, out):
    name = dict(gemm="fp8_gemm", dx="fp8_gemm_dx", gate="fp8_ffn_gate", packed="fp8_ffn_gate_packed")[op]
    return gq.product_plan(name, n, d, d, dtype=gq.GQ_F32 if out == F32 else gq.GQ_BF16)


@pytest.mark.parametrize("op,out", [(op, out) for op in OPS for out in (BF, F32) if op != "packed" or out == F32])
@pytest.mark.parametrize("n,streamed", ROWS)
def test_zero_sums_under_the_largest_scales(device, n, streamed, op, out):
    """The first block of the contraction has scales of 2^100 on both sides and sums of zero, but for one output
    that is over the range: the others are the second block's."""
    d = 256
    assert plan(op, n, d, out)["streamed"] == (streamed and op != "dx")
    x, w = integers(device, n, d, seed=1), integers(device, d, d, seed=2)
    XS = torch.full((n, 4), 127, dtype=U8, device=device)
    S = torch.full((2, 2), 127 - 4, dtype=U8, device=device)
    XS[:, 0] = 227
    first = w if op != "dx" else w.T                       # [outputs][contraction]
    first[:, :128] = 0
    if op == "dx":
        S[0] = 227
    else:
        S[:, 0] = 227
    want = (x[:, 128:].double() @ first[:, 128:].double().T) * 2.0 ** -4
    first[7, 3], x[:, 3] = 1, 2                            # 2 by 1 by 2^200
    y = call(op, x.float().to(FP8), XS, w.float().to(FP8), S, d, out)
    keep = torch.ones(d, dtype=torch.bool, device=device)
    if op in ("gemm", "dx"):
        assert bool(torch.isinf(y[:, 7]).all())
        keep[7] = False
        assert torch.equal(y[:, keep].double(), want[:, keep].to(out).double())
        return
    # (packed, the output over the range takes its whole block along)
    keep[:128 if op == "packed" else 8] = False
    v = want * want * torch.sigmoid(want)
    limit = 2.0 ** -3 * v.abs() + 2.0 ** -9 * v.abs().amax(1, keepdim=True) if op == "packed" else 2.0 ** -7 * v.abs()
    assert bool(((y.double() - v).abs() <= limit + 1e-30)[:, keep].all())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("op", ["gemm", "dx"])
@pytest.mark.parametrize("n,streamed", ROWS)
@pytest.mark.parametrize("left,right", [(-75, -75), (-126, -24), (-24, -126), (100, 26), (127, -127), (-127, 127)])
def test_sums_within_the_range_under_scales_past_it(device, n, streamed, left, right, op, out):
    """Scales whose product is no float32 number, or at the end of the bytes' range, of sums whose
    product with them is one."""
    d = 128
    assert plan(op, n, d, out)["streamed"] == (streamed and op != "dx")
    # for small products of scales the largest codes, 128 448^2 2^-150 = 1.5 2^-126; for large ones one small code
    if left + right < -100:
        x, w = torch.full((n, d), 448.0, device=device), torch.full((d, d), 448.0, device=device)
    else:
        x, w = torch.zeros(n, d, device=device), torch.zeros(d, d, device=device)
        x[:, 0], w[0], w[:, 0] = 2.0 ** -6, 1.0, 1.0
    XS = torch.full((n, 4), 127 + left, dtype=U8, device=device)
    S = torch.full((1, 1), 127 + right, dtype=U8, device=device)
    y = call(op, x.to(FP8), XS, w.to(FP8), S, d, out)
    want = (x.double() @ (w.double() if op == "dx" else w.double().T)) * 2.0 ** (left + right)
    assert bool((want.abs() >= 2.0 ** -126)[want != 0].all()) and bool(torch.isfinite(want.float()).all())
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("op,out", [(op, out) for op in OPS for out in (BF, F32) if op != "packed" or out == F32])
@pytest.mark.parametrize("n,streamed", ROWS)
def test_a_scale_of_nan_makes_its_row_or_columns_nan(device, n, streamed, op, out, scales):
    """Also where all of the codes are zeros."""
    d = 256
    x, w = torch.zeros(n, d, device=device), integers(device, d, d, seed=2).float()
    x[1:] = integers(device, n - 1, d, seed=1).float()
    nan = 255 if scales == U8 else float("nan")
    XS = torch.full((n, 4), 127 if scales == U8 else 1.0, dtype=scales, device=device)
    S = torch.full((2, 2), 127 if scales == U8 else 1.0, dtype=scales, device=device)
    XS[0, 1] = nan
    bad = torch.isnan(call(op, x.to(FP8), XS, w.to(FP8), S, d, out))
    assert bool(bad[0].all()) and not bad[1:].any()
    XS[0, 1] = XS[0, 0]
    S[1, 0] = nan
    bad = torch.isnan(call(op, x.to(FP8), XS, w.to(FP8), S, d, out))
    cols = slice(0, 128) if op == "dx" else slice(128, 256)
    assert bool(bad[:, cols].all()) and int(bad.sum()) == n * 128


def place(t, at):
    """t's values, starting `at` elements past a 256-byte border."""
    some = torch.zeros(t.numel() + at, dtype=t.dtype, device=t.device)
    assert some.data_ptr() % 256 == 0
    some[at:] = t.flatten()
    return some[at:].view(t.shape)


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("op", [op for op in CASES if op.startswith("fp8")])
def test_scales_at_any_place_that_the_header_allows(device, op, scales):
    """Rows' scales off the 16-byte border that the tiles' copies of float32 ones would like, weights' off their own: the
    same bits, in every kernel."""
    name = op.replace("fp8_", "").replace("ffn_", "")
    for n, d_in, d_out, experts in CASES[op]:
        print(op, n, d_in, d_out, experts, flush=True)
        back = op == "fp8_gemm_dx"
        at = counts(n, experts, seed=n) if experts else None
        offsets = torch.tensor(at, device=device) if experts else None
        E = (experts,) if experts else ()
        XQ, XS = gq.fp8_quantize(torch.randn(n, d_out if back else d_in, device=device), scales=scales)
        Q, S = gq.fp8_quantize_weight(torch.randn(*E, d_out, d_in, device=device), scales=scales)
        for out in (BF, F32) if not name.endswith("packed") else (None,):
            def run(xs, s, u):
                k = dict(offsets=offsets)
                if back:
                    return gq.fp8_gemm_dx(XQ, xs, Q, s, d_in, out_dtype=out, **k)
                if name == "gemm":
                    return gq.fp8_gemm(XQ, xs, Q, s, d_in, out_dtype=out, **k)
                if out is not None:
                    return gq.fp8_ffn_gate(XQ, xs, Q, s, Q, u, d_in, out_dtype=out, **k)
                HS = place(torch.zeros(n, gq.fp8_row_scales(d_out), dtype=scales, device=device), 4 if scales == U8 else 3)
                HQ, HS = gq.fp8_ffn_gate(XQ, xs, Q, s, Q, u, d_in, packed=True, HS=HS, **k)
                return torch.cat([HQ.view(U8).flatten(), HS.contiguous().view(U8).flatten()])

            want = run(XS, S, S)
            for a, b in ((1, 1), (2, 3), (3, 2)):
                xs = place(XS, 4 * a if scales == U8 else a)
                assert xs.data_ptr() % 16 == 4 * a
                assert torch.equal(run(xs, place(S, b), place(S, a)), want), (n, d_in, d_out, experts, out, a, b)
