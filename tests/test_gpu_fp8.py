"""GPU tests of the 8-bit rows and products against float64 (bounds: _product_cases)."""
import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_gq_amd as gq
from _product_cases import (BF, F32, FP8, U8, act64, check, check_product, counts, f64, gate64, normal, of,
                            rows, spans, weight)

pytestmark = pytest.mark.gpu


def codes(t):
    return t.view(U8).cpu().numpy()


def as_scales(byte, scales):
    """Scale bytes as the type has them."""
    if scales == U8:
        return byte
    return np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127)).astype(np.float32)


def same(S, byte, scales):
    np.testing.assert_array_equal(S.cpu().numpy(), as_scales(byte, scales))


# ---- rows and weights -------------------------------------------------------------------

@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 127), (3, 128), (5, 129), (2, 7), (7, 512), (3, 520), (9, 1032),
                                 (1, 4096), (33, 1001), (257, 640)])
def test_quantize_rows(device, n, d, dtype, scales):
    rng = np.random.default_rng(n * 1000 + d)
    x = rng.standard_normal((n, d)) * np.exp2(rng.integers(-30, 30, (n, 1)))
    x[rng.random((n, d)) < 0.1] = 0.0
    x[rng.random((n, d)) < 0.1] *= 300.0
    t = torch.from_numpy(x).to(dtype)
    Q, S = gq.fp8_quantize(t.to(device), scales=scales)
    Qr, Sr = O.fp8_quantize(f64(t))
    same(S, Sr, scales)
    np.testing.assert_array_equal(codes(Q), Qr)
    for out in (BF, F32):
        np.testing.assert_array_equal(f64(gq.fp8_dequantize(Q, S, d, dtype=out)), O.fp8_values(Qr, Sr, d))


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("experts,d_out,d_in", [(None, 1, 1), (None, 128, 128), (None, 129, 127), (None, 300, 520),
                                                (3, 130, 1001), (2, 64, 256), (5, 1, 129)])
def test_quantize_weights(device, experts, d_out, d_in, dtype, scales):
    rng = np.random.default_rng(d_out * 1000 + d_in)
    w = rng.standard_normal((experts or 1, d_out, d_in)) * np.exp2(rng.integers(-20, 20, (experts or 1, d_out, 1)))
    t = torch.from_numpy(w).to(dtype)
    given = t.to(device) if experts else t[0].to(device)
    Q, S = gq.fp8_quantize_weight(given, scales=scales)
    back = gq.fp8_dequantize_weight(Q, S, d_in, dtype=F32)
    assert back.shape == given.shape
    for e in range(experts or 1):
        Qr, Sr = O.fp8_quantize_weight(f64(t[e]))
        q, s, b = (Q[e], S[e], back[e]) if experts else (Q, S, back)
        same(s, Sr, scales)
        np.testing.assert_array_equal(codes(q), Qr)
        np.testing.assert_array_equal(f64(b), O.fp8_weight_values(Qr, Sr, d_in))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_every_border_and_scale(device, dtype):
    """Each border between two codes, its neighbours in the type and both signs, under each scale from
    the subnormal range to the type's largest."""
    eps = 2.0 ** -8 if dtype == BF else 2.0 ** -23
    mid = (O.FP8_GRID[1:] + O.FP8_GRID[:-1]) / 2
    u = np.concatenate([mid, mid * (1 + eps), mid * (1 - eps)])[:378]
    u = np.concatenate([u, -u, O.FP8_GRID, -O.FP8_GRID])
    u = np.concatenate([u, np.zeros(-len(u) % 127)]).reshape(-1, 127)
    u = np.concatenate([np.full((len(u), 1), 448.0), u], axis=1).reshape(-1)          # the block's scale is the unit
    lo = -126 if dtype == F32 else -126
    x = np.stack([u * 2.0 ** e for e in range(lo, 120)])
    t = torch.from_numpy(x).to(dtype)
    for scales in (U8, F32):
        Q, S = gq.fp8_quantize(t.to(device), scales=scales)
        Qr, Sr = O.fp8_quantize(f64(t))
        same(S, Sr, scales)
        np.testing.assert_array_equal(codes(Q), Qr)


@pytest.mark.parametrize("scales", [U8, F32])
def test_quantize_borders_between_scales_and_tiny_blocks(device, scales):
    top = np.concatenate([[448 * 2.0 ** e for e in range(-137, 119)], [0.0, 2.0 ** -149]]).astype(np.float32)
    top = np.concatenate([top, np.nextafter(top, np.float32(np.inf)), np.nextafter(top, np.float32(-np.inf))])
    x = np.zeros((len(top), 128), np.float32)
    x[:, 77] = top
    x[:, 3] = -top / 3
    t = torch.from_numpy(x)
    Q, S = gq.fp8_quantize(t.to(device), scales=scales)
    Qr, Sr = O.fp8_quantize(f64(t))
    same(S, Sr, scales)
    np.testing.assert_array_equal(codes(Q), Qr)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dequantize_every_code_and_scale(device, dtype):
    """All 256 codes under all 256 scale bytes, and under float32 scales that are no powers of two."""
    Q = np.tile(np.arange(256, dtype=np.uint8), (256, 2))
    S = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    t = torch.from_numpy(Q).to(device).view(FP8)
    with np.errstate(over="ignore", invalid="ignore"):
        ref = torch.from_numpy(O.fp8_values(Q, S, 512)).to(F32).to(dtype)
        np.testing.assert_array_equal(f64(gq.fp8_dequantize(t, torch.from_numpy(S).to(device), 512, dtype=dtype)), f64(ref))
        any32 = np.random.default_rng(0).standard_normal((256, 4)).astype(np.float32)
        ref = torch.from_numpy(O.code_values(Q).astype(np.float32) * np.repeat(any32, 128, axis=1)).to(dtype)
        np.testing.assert_array_equal(f64(gq.fp8_dequantize(t, torch.from_numpy(any32).to(device), 512, dtype=dtype)), f64(ref))


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_nonfinite(device, dtype, scales):
    """A NaN or an infinity makes its own block NaN and no other; the type's largest value does not."""
    x = torch.ones(6, 300, dtype=dtype)
    x[0, 130], x[1, 299], x[2, 0], x[3, 64] = float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max
    x[4] = 0
    Q, S = gq.fp8_quantize(x.to(device), scales=scales)
    Qr, Sr = O.fp8_quantize(f64(x))
    same(S, Sr, scales)
    np.testing.assert_array_equal(codes(Q), Qr)
    assert np.isnan(f64(gq.fp8_dequantize(Q, S, 300))).sum() == 128 + 44 + 128
    Q, S = gq.fp8_quantize_weight(x.to(device), scales=scales)
    v = f64(gq.fp8_dequantize_weight(Q, S, 300))
    assert np.isnan(v).all()          # (each of its three blocks has one)


def test_quantize_offset_views_and_given_outputs(device):
    """Values that start off a 16-byte border; outputs of the caller's."""
    flat = normal(device, 5 * 333 + 8, seed=3, dtype=BF)
    for at in (1, 3, 8):
        x = flat[at:at + 5 * 333].view(5, 333)
        Q = torch.empty(5, 384, dtype=U8, device=device).view(FP8)
        S = torch.empty(5, 4, dtype=F32, device=device)
        q, s = gq.fp8_quantize(x, Q=Q, S=S)
        assert q is Q and s is S
        Qr, Sr = O.fp8_quantize(f64(x))
        np.testing.assert_array_equal(codes(Q), Qr)
        same(S, Sr, F32)
        y = torch.empty(5 * 333 + 1, dtype=F32, device=device)[1:].view(5, 333)
        np.testing.assert_array_equal(f64(gq.fp8_dequantize(Q, S, 333, dtype=F32, y=y)), O.fp8_values(Qr, Sr, 333))
    x = normal(device, 2, 3, 200, seed=4)                       # more dimensions
    Q, S = gq.fp8_quantize(x)
    assert Q.shape == (2, 3, 256) and S.shape == (2, 3, 4)
    np.testing.assert_array_equal(codes(Q).reshape(6, 256), O.fp8_quantize(f64(x).reshape(6, 200))[0])
    assert gq.fp8_dequantize(Q, S, 200).shape == (2, 3, 200)
    none = gq.fp8_quantize(x[:0].reshape(0, 200))
    assert none[0].shape == (0, 256) and gq.fp8_dequantize(*none, 200).shape == (0, 200)


# ---- products ---------------------------------------------------------------------------

SIZES = [(1, 128, 128), (1, 1, 1), (1, 4096, 4096), (3, 130, 200), (16, 1000, 333), (17, 257, 129), (24, 2048, 512),
         (40, 640, 1000), (64, 1408, 264), (65, 384, 300), (128, 512, 520), (129, 1024, 257), (200, 2047, 1001),
         (256, 256, 256), (300, 4096, 640), (513, 520, 384), (1000, 300, 2100)]


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n,d_in,d_out", SIZES)
def test_gemm(device, n, d_in, d_out, out, scales):
    XQ, XS, x = rows(device, n, d_in, scales, seed=1)
    Q, S, W = weight(device, d_out, d_in, scales, seed=2)
    y = gq.fp8_gemm(XQ, XS, Q, S, d_in, out_dtype=out)
    assert y.shape == (n, d_out) and y.dtype == out
    check_product(y, x, W, None, d_in, out, "gemm", eight=out == BF)
    assert torch.equal(y, gq.fp8_gemm(XQ, XS, Q, S, d_in, out_dtype=out))


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n,d_in,d_out", SIZES)
def test_gemm_dx(device, n, d_in, d_out, out, scales):
    GQ, GS, g = rows(device, n, d_out, scales, seed=3)
    Q, S, W = weight(device, d_out, d_in, scales, seed=4)
    y = gq.fp8_gemm_dx(GQ, GS, Q, S, d_in, out_dtype=out)
    assert y.shape == (n, d_in) and y.dtype == out
    check_product(y, g, W.T, None, d_out, out, "dx", eight=out == BF)
    assert torch.equal(y, gq.fp8_gemm_dx(GQ, GS, Q, S, d_in, out_dtype=out))


GROUPED = [(5, 200, 130, 3), (33, 256, 384, 4), (96, 512, 256, 40), (300, 640, 264, 6), (700, 257, 520, 9),
           (1500, 1024, 384, 3), (64, 300, 200, 130)]


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("n,d_in,d_out,experts", GROUPED)
def test_experts(device, n, d_in, d_out, experts, back, scales):
    at = counts(n, experts, seed=n)
    offsets = torch.tensor(at, device=device)
    Q, S, W = weight(device, d_out, d_in, scales, seed=5, experts=experts)
    AQ, AS, a = rows(device, n, d_out if back else d_in, scales, seed=6)
    fn = gq.fp8_gemm_dx if back else gq.fp8_gemm
    y = fn(AQ, AS, Q, S, d_in, offsets=offsets, out_dtype=F32)
    check_product(y, a, W.transpose(1, 2) if back else W, at, d_out if back else d_in, F32, "experts")
    given = torch.full_like(y, 7.0)
    assert fn(AQ, AS, Q, S, d_in, offsets=offsets, y=given) is given
    assert bool((given[:at[0]] == 7).all()) and bool((given[at[-1]:] == 7).all())
    assert torch.equal(given[at[0]:at[-1]], y[at[0]:at[-1]])


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("back", [False, True])
def test_nonfinite_stays_in_its_row_or_columns(device, back, scales):
    """A NaN block of x makes its row NaN; one of a weight the 128 columns (or rows) that it reaches."""
    n, d_in, d_out = 70, 384, 300
    x = normal(device, n, d_out if back else d_in, seed=1)
    x[13, 5] = float("inf")
    w = normal(device, d_out, d_in, seed=2)
    A, Wp = gq.fp8_quantize(x, scales=scales), gq.fp8_quantize_weight(w, scales=scales)
    fn = gq.fp8_gemm_dx if back else gq.fp8_gemm
    bad = torch.isnan(fn(*A, *Wp, d_in, out_dtype=F32))
    assert bool(bad[13].all()) and int(bad.sum()) == bad.shape[1]
    w[130, 257] = float("nan")
    Wp = gq.fp8_quantize_weight(w, scales=scales)
    bad = torch.isnan(fn(*A, *Wp, d_in, out_dtype=F32))
    want = torch.zeros_like(bad)
    want[13] = True
    want[:, 256:384] = True if back else want[:, 256:384]
    if not back:
        want[:, 128:256] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("back", [False, True])
def test_largest_and_smallest_scales(device, back, scales):
    """Operands near the ends of the scales' range whose product is ordinary; each one-term output exact."""
    n, d = 20, 256
    x = torch.zeros(n, d, device=device)
    w = torch.zeros(d, d, device=device)
    k = torch.arange(n, device=device)
    x[k, k * 12 % d] = 2.0 ** 100 * (1 + k / 8)
    w.fill_diagonal_(2.0 ** -110)
    y = (gq.fp8_gemm_dx if back else gq.fp8_gemm)(*gq.fp8_quantize(x, scales=scales), *gq.fp8_quantize_weight(w, scales=scales), d, out_dtype=F32)
    want = torch.zeros_like(y)
    want[k, k * 12 % d] = 2.0 ** -10 * gq.fp8_dequantize(*gq.fp8_quantize(1 + k[:, None] / 8), 1, dtype=F32)[:, 0]
    assert torch.equal(y, want)


@pytest.mark.parametrize("scales", [U8, F32])
def test_empty_calls_and_bad_offsets(device, scales):
    Q, S, W = weight(device, 200, 300, scales, seed=1, experts=3)
    XQ, XS, x = rows(device, 50, 300, scales, seed=2)
    for at in ([0, 0, 0, 0], [50, 50, 50, 50], [-5, 10, 400, 1000], [30, 10, 5, 50], [1 << 62, 0, -(1 << 62), 7]):
        offsets = torch.tensor(at, device=device)
        y = gq.fp8_gemm(XQ, XS, Q, S, 300, offsets=offsets)
        g = gq.fp8_gemm_dx(*gq.fp8_quantize(y, scales=scales), Q, S, 300, offsets=offsets)
        assert y.shape == (50, 200) and g.shape == (50, 300)
    y = gq.fp8_gemm(XQ[:0], XS[:0], Q[0], S[0], 300)
    assert y.shape == (0, 200)
    at = torch.tensor([0, 20, 20, 50], device=device)             # one expert of three without rows
    check_product(gq.fp8_gemm(XQ, XS, Q, S, 300, offsets=at, out_dtype=F32), x, W, at.tolist(), 300, F32, "empty expert")


# ---- the gate with packed weights ---------------------------------------------------------

@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("act,out", [("silu", BF), ("gelu", F32), ("gelu_tanh", BF), ("silu", F32)])
@pytest.mark.parametrize("n,d_in,d_ff", [(1, 128, 128), (1, 4096, 1408), (5, 130, 200), (16, 1000, 333), (40, 640, 300),
                                         (65, 384, 520), (130, 2048, 257), (300, 512, 1000)])
def test_gate(device, n, d_in, d_ff, act, out, scales):
    XQ, XS, x = rows(device, n, d_in, scales, seed=1)
    G, GS, g = weight(device, d_ff, d_in, scales, seed=2)
    U, US, u = weight(device, d_ff, d_in, scales, seed=3)
    h = gq.fp8_ffn_gate(XQ, XS, G, GS, U, US, d_in, act=act, out_dtype=out)
    ref, limit = gate64(x, g, u, act, d_in, eight=out == BF)[:2]
    check(h, ref, limit, out, "gate")
    assert torch.equal(h, gq.fp8_ffn_gate(XQ, XS, G, GS, U, US, d_in, act=act, out_dtype=out))


@pytest.mark.parametrize("scales", [U8, F32])
@pytest.mark.parametrize("n,d_in,d_ff,experts", [(1, 256, 128, None), (7, 300, 130, None), (16, 1024, 1408, None), (50, 384, 520, None),
                                                 (200, 512, 1000, None), (600, 256, 2049, None), (90, 300, 200, 5), (700, 384, 640, 4)])
def test_gate_packed(device, n, d_in, d_ff, experts, scales):
    """The packed h is what packing the float32 h gives (the same sums, rounded later)."""
    at = counts(n, experts, seed=1) if experts else None
    offsets = torch.tensor(at, device=device) if experts else None
    XQ, XS, x = rows(device, n, d_in, scales, seed=1)
    G, GS, g = weight(device, d_ff, d_in, scales, seed=2, experts=experts)
    U, US, u = weight(device, d_ff, d_in, scales, seed=3, experts=experts)
    h = gq.fp8_ffn_gate(XQ, XS, G, GS, U, US, d_in, offsets=offsets, out_dtype=F32)
    HQ, HS = gq.fp8_ffn_gate(XQ, XS, G, GS, U, US, d_in, offsets=offsets, packed=True)
    assert HS.dtype == scales
    r = slice(at[0], at[-1]) if experts else slice(0, n)
    got, want = gq.fp8_dequantize(HQ, HS, d_ff, dtype=F32).double(), h.double()
    unit = HS.double() if scales == F32 else torch.exp2(HS.double() - 127)
    unit = unit.repeat_interleave(128, 1)[:, :d_ff]
    # half a step of the code (its place on the other side of a border apart), and as far as h is off itself
    slack = torch.zeros_like(want)
    for e, part in spans(n, at):
        slack[part] = gate64(x[part], of(g, e), of(u, e), "silu", d_in)[1] * 2.07
    limit = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * unit) + slack
    assert bool(((got - want).abs() <= limit)[r].all())
    assert not got[:r.start].abs().sum() and not got[r.stop:].abs().sum()
    top = torch.zeros(n, HQ.shape[1], dtype=torch.float64, device=device)
    top[:, :d_ff] = want.abs()
    top = top.view(n, -1, 128).amax(2)[r]
    s = (HS.double() if scales == F32 else torch.exp2(HS.double() - 127))[r, :top.shape[1]]
    edge = torch.nn.functional.pad(slack, (0, HQ.shape[1] - d_ff)).view(n, -1, 128).amax(2)[r]
    assert bool((top <= 448 * s + edge).all()) and bool(((top > 224 * s - edge) | (top == 0)).all())
    assert not HQ.view(U8)[r, d_ff:].any()
    tail = HS[r, -(-d_ff // 128):]
    assert bool((tail == (127 if scales == U8 else 1)).all())


def test_gate_packed_keeps_given_rows_of_no_expert(device):
    n, d_in, d_ff, E = 60, 200, 300, 3
    at = [10, 20, 20, 50]
    XQ, XS, _ = rows(device, n, d_in, U8, seed=1)
    G, GS, _ = weight(device, d_ff, d_in, U8, seed=2, experts=E)
    HQ = torch.full((n, 384), 9, dtype=U8, device=device).view(FP8)
    HS = torch.full((n, 4), 9, dtype=U8, device=device)
    q, s = gq.fp8_ffn_gate(XQ, XS, G, GS, G, GS, d_in, offsets=torch.tensor(at, device=device), packed=True, HQ=HQ, HS=HS)
    assert q is HQ and s is HS
    keep = torch.ones(n, dtype=torch.bool)
    keep[10:50] = False
    assert bool((HQ.view(U8)[keep] == 9).all()) and bool((HS[keep] == 9).all()) and not bool((HS[~keep] == 9).any())


@pytest.mark.parametrize("scales", [U8, F32])
def test_feed_forward_block(device, scales):
    """Pack, gate, down projection and the gradients back to the Fisher, as they are used together."""
    n, d, f = 150, 512, 640
    x = normal(device, n, d, seed=1, dtype=BF)
    XQ, XS = gq.fp8_quantize(x, scales=scales)
    G, GS, g = weight(device, f, d, scales, seed=2)
    U, US, u = weight(device, f, d, scales, seed=3)
    D, DS, w = weight(device, d, f, scales, seed=4)
    HQ, HS = gq.fp8_ffn_gate(XQ, XS, G, GS, U, US, d, packed=True)
    y = gq.fp8_gemm(HQ, HS, D, DS, f, out_dtype=F32)
    check_product(y, gq.fp8_dequantize(HQ, HS, f, dtype=F32).double(), w, None, f, F32, "down")
    a = gq.fp8_dequantize(XQ, XS, d, dtype=F32).double()
    h = act64(a @ g.T, "silu")[0] * (a @ u.T)
    # h packed is off by half a step, 2^-4 of each value or 2^-10 of a unit that is at most its row's
    # largest over 224 (a row's sums apart): carried through |w|
    half = torch.maximum(2.0 ** -4 * h.abs(), 2.0 ** -10 / 200 * h.abs().amax(1, keepdim=True)) * 1.01
    assert bool(((y.double() - h @ w.T).abs() <= half @ w.T.abs() + 1e-4 * (h.abs() @ w.T.abs())).all())
    # the gradient of h, for the layers before
    dy = normal(device, n, d, seed=5, scale=1e-3)
    dh = gq.fp8_gemm_dx(*gq.fp8_quantize(dy, scales=scales), D, DS, f)
    F = gq.gq_fisher_accumulate(gq.fp8_dequantize(HQ, HS, f), dy.to(BF), 2)
    assert dh.shape == (n, f) and F.shape == (2, f, f) and bool(torch.isfinite(F).all())


def test_product_refusals_on_the_gpu(device):
    XQ, XS, _ = rows(device, 4, 200, U8, seed=1)
    Q, S, _ = weight(device, 64, 200, F32, seed=2)
    with pytest.raises(gq.GQError) as e:
        gq.fp8_gemm(XQ, XS, Q, S, 200)
    assert "scales" in e.value.message                              # of different types
    Q, S, _ = weight(device, 64, 200, U8, seed=2)
    with pytest.raises(gq.GQError) as e:
        gq.fp8_gemm(XQ.view(U8), XS, Q, S, 200)
    assert e.value.status == 3                                      # bytes of no format
    with pytest.raises(gq.GQError) as e:
        gq.fp8_gemm(XQ, XS, Q[:, ::2], S, 200)
    with pytest.raises(gq.GQError) as e:
        gq.fp8_gemm(XQ, XS, Q, S, 200, y=torch.empty(4, 64, device=device), out_dtype=BF)
    wide = torch.zeros(4, 512, dtype=U8, device=device).view(FP8)[:, :256]
    with pytest.raises(gq.GQError) as e:
        gq.fp8_gemm(wide, XS, Q, S, 200)
    assert "contiguous" in e.value.message


