"""GPU tests of the MXFP4 rows and products against the float64 oracle.

Bars:
  * codes, scales and read-back values: equal (a rounding to a grid, exact products of powers
    of two);
  * products: every term a w is exact in float32 (bfloat16 by two significant bits, planes of a
    float32 likewise), so only the K sums round.  A float32 addition is off by at most 2^-24 of
    its result where it rounds to nearest and 2^-23 where it truncates, and every partial sum is
    at most A = sum |a w|, so |y - y64| <= (T + 8) 2^-23 A, T the number of terms (three planes
    of float32 a: 3 K, of total size at most (1 + 2^-7) A, within the 8 and the slack of
    truncation), plus a bfloat16 output's half step 2^-8 |y| (and 2^-134 below the normal range).
"""
import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_gq_amd as gq

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def u8(a, device):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def random_weight(rng, experts, d_out, d_in):
    """Packed Gaussian weights whose blocks' scales vary, and their values."""
    w = rng.standard_normal((experts * d_out, d_in)) * np.exp(rng.standard_normal((experts * d_out, 1)))
    Q, S = O.mx_quantize(w)
    v = O.mx_values(Q, S, d_in).reshape(experts, d_out, d_in)
    return Q.reshape(experts, d_out, -1), S.reshape(experts, d_out, -1), v


def bound(a, W, y_ref, terms, out):
    b = (terms + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(W).T)
    return b + (2.0 ** -8 * np.abs(y_ref) + 2.0 ** -134 if out == BF else 0.0)


def check(y, a, W, terms, out, what="", lost=0.0):
    """lost: how far the path holds each value of a (absolutely), which adds lost sum |w|."""
    ref = a @ W.T
    err, b = np.abs(f64(y) - ref), bound(a, W, ref, terms, out) + lost * np.abs(W).sum(axis=1)
    print(what, "worst error / bound", float(np.max(err / np.maximum(b, 1e-300))) if err.size else 0.0)
    assert np.all(err <= b)


# ---- rows -------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 31), (3, 32), (5, 33), (2, 127), (7, 128), (3, 130),
                                    (9, 136), (1, 4096), (33, 1001), (257, 520)])
def test_quantize_rows(device, rows, d, dtype):
    rng = np.random.default_rng(rows * 1000 + d)
    x = rng.standard_normal((rows, d)) * np.exp2(rng.integers(-30, 30, (rows, 1)))
    x[rng.random((rows, d)) < 0.1] = 0.0
    x[rng.random((rows, d)) < 0.1] *= 30.0
    t = torch.from_numpy(x).to(dtype)
    Q, S = gq.mxfp4_quantize(t.to(device))
    Qr, Sr = O.mx_quantize(f64(t))
    np.testing.assert_array_equal(S.cpu().numpy(), Sr)
    np.testing.assert_array_equal(Q.cpu().numpy(), Qr)
    for out in (BF, F32):
        np.testing.assert_array_equal(f64(gq.mxfp4_dequantize(Q, S, d, dtype=out)), O.mx_values(Qr, Sr, d))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_every_tie_and_scale(device, dtype):
    """Each boundary between two codes, its neighbours in the type and both signs, under each
    scale from the subnormal range to the type's largest."""
    half = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    eps = 2.0 ** -8 if dtype == BF else 2.0 ** -23
    u = np.concatenate([half, half * (1 + eps), half * (1 - eps), [0.0, 6.0, 7.9375, 4.0]])
    rows = []
    for e in range(-149 if dtype == F32 else -133, 126):
        r = np.zeros(64)
        r[:len(u)] = u * 2.0 ** e
        r[32:32 + 25] = -r[:25]
        rows.append(r)
    t = torch.from_numpy(np.stack(rows)).to(dtype)
    Q, S = gq.mxfp4_quantize(t.to(device))
    Qr, Sr = O.mx_quantize(f64(t))
    np.testing.assert_array_equal(S.cpu().numpy(), Sr)
    np.testing.assert_array_equal(Q.cpu().numpy(), Qr)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dequantize_every_code_and_scale(device, dtype):
    """All 16 codes under all 256 scale bytes."""
    Q = np.tile(np.arange(0, 256, 1, dtype=np.uint8).reshape(1, 256)[:, :64], (64, 1))
    Q[:, :16] = np.arange(16) | (np.arange(16)[::-1] << 4)
    S = np.arange(256, dtype=np.uint8).reshape(64, 4)
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(O.mx_values(Q, S, 128)).to(dtype).to(torch.float64).numpy()
    got = f64(gq.mxfp4_dequantize(u8(Q, device), u8(S, device), 128, dtype=dtype))
    np.testing.assert_array_equal(got, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_nonfinite(device, dtype):
    """A NaN or an infinity makes its own block NaN and no other."""
    x = torch.ones(6, 160, dtype=dtype)
    x[0, 40], x[1, 159], x[2, 0], x[3, 64] = float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max
    x[4] = 0
    Q, S = gq.mxfp4_quantize(x.to(device))
    Qr, Sr = O.mx_quantize(f64(x))
    np.testing.assert_array_equal(S.cpu().numpy(), Sr)
    np.testing.assert_array_equal(Q.cpu().numpy(), Qr)
    v = f64(gq.mxfp4_dequantize(Q, S, 160))
    assert np.isnan(v[0, 32:64]).all() and np.isnan(v).sum() == 96


def test_quantize_offset_views(device):
    """Rows that start off a 16-byte border (element-aligned) take the scalar loads."""
    base = torch.randn(1 + 4 * 256, device=device)
    for dtype in (BF, F32):
        x = base.to(dtype)[1:].view(4, 256)
        Q, S = gq.mxfp4_quantize(x)
        Qr, Sr = O.mx_quantize(f64(x))
        np.testing.assert_array_equal(Q.cpu().numpy(), Qr)
        y = torch.full((1 + 4 * 256,), 7.0, dtype=dtype, device=device)
        gq.mxfp4_dequantize(Q, S, 256, dtype=dtype, y=y[1:].view(4, 256))
        assert float(y[0]) == 7.0
        np.testing.assert_array_equal(f64(y[1:]).reshape(4, 256), O.mx_values(Qr, Sr, 256))


# ---- products ---------------------------------------------------------------------------

# rows from one to past the widest tile, widths of less than a block to several tiles, whole
# and ragged
SIZES = [(1, 1, 1), (1, 4096, 64), (2, 33, 17), (3, 128, 16), (8, 1000, 200), (16, 512, 48),
         (17, 640, 130), (24, 2048, 256), (33, 96, 300), (64, 1024, 128), (65, 4096, 96), (100, 257, 513),
         (129, 384, 1024), (256, 256, 256), (257, 520, 264), (600, 129, 520), (1024, 1024, 512)]


@pytest.mark.parametrize("n,d_in,d_out", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_gemm(device, n, d_in, d_out, dtype, out):
    rng = np.random.default_rng(n * 7 + d_in + d_out)
    Q, S, W = random_weight(rng, 1, d_out, d_in)
    x = torch.from_numpy(rng.standard_normal((n, d_in))).to(dtype)
    y = gq.mxfp4_gemm(x.to(device), u8(Q[0], device), u8(S[0], device), out_dtype=out)
    assert y.dtype == out and tuple(y.shape) == (n, d_out)
    check(y, f64(x), W[0], d_in * (1 if dtype == BF else 3), out)


@pytest.mark.parametrize("n,d_in,d_out", SIZES)
@pytest.mark.parametrize("out", [BF, F32])
def test_gemm_mx(device, n, d_in, d_out, out):
    rng = np.random.default_rng(n * 7 + d_in + d_out + 1)
    Q, S, W = random_weight(rng, 1, d_out, d_in)
    XQ, XS, X = random_weight(rng, 1, n, d_in)
    y = gq.mxfp4_gemm_mx(u8(XQ[0], device), u8(XS[0], device), u8(Q[0], device), u8(S[0], device),
                         d_in, out_dtype=out)
    check(y, X[0], W[0], d_in, out)


@pytest.mark.parametrize("n,d_in,d_out", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_gemm_dx(device, n, d_in, d_out, dtype, out):
    rng = np.random.default_rng(n * 7 + d_in + d_out + 2)
    Q, S, W = random_weight(rng, 1, d_out, d_in)
    g = torch.from_numpy(rng.standard_normal((n, d_out))).to(dtype)
    dx = gq.mxfp4_gemm_dx(g.to(device), u8(Q[0], device), u8(S[0], device), d_in, out_dtype=out)
    assert tuple(dx.shape) == (n, d_in)
    check(dx, f64(g), np.ascontiguousarray(W[0].T), d_out * (1 if dtype == BF else 3), out)


GROUPS = [([0, 0, 5, 5, 12], 12, 160, 72), ([0, 1], 1, 64, 16), ([3, 10, 10, 40], 47, 300, 130),
          ([0, 17, 18, 82, 82, 339, 340], 352, 256, 144), ([0, 0, 0], 6, 128, 64),
          ([0, 300, 301, 640], 640, 512, 272)]


@pytest.mark.parametrize("op", ["gemm", "gemm_mx", "gemm_dx"])
@pytest.mark.parametrize("offsets,n,d_in,d_out", GROUPS)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32)])
def test_experts(device, op, offsets, n, d_in, d_out, dtype, out):
    """Empty experts, one row, ragged tiles, rows before the first and behind the last, which
    keep their values; NaN in those rows of the input reaches nothing."""
    E = len(offsets) - 1
    rng = np.random.default_rng(n + E)
    Q, S, W = random_weight(rng, E, d_out, d_in)
    width, k = (d_in, d_out) if op == "gemm_dx" else (d_out, d_in)
    y = torch.full((n, width), -77.0, dtype=out, device=device)
    off = torch.tensor(offsets, dtype=torch.int64, device=device)
    Qd, Sd = u8(Q, device), u8(S, device)
    lo, hi = offsets[0], offsets[-1]
    if op == "gemm_mx":
        XQ, XS, X = random_weight(rng, 1, n, d_in)
        a, XS = X[0], XS[0]
        XS[:lo], XS[hi:] = 255, 255
        got = gq.mxfp4_gemm_mx(u8(XQ[0], device), u8(XS, device), Qd, Sd, d_in, offsets=off, y=y)
        terms = k
    else:
        x = torch.from_numpy(rng.standard_normal((n, k))).to(dtype)
        a = f64(x)
        x[:lo], x[hi:] = float("nan"), float("nan")
        if op == "gemm":
            got = gq.mxfp4_gemm(x.to(device), Qd, Sd, offsets=off, y=y)
        else:
            got = gq.mxfp4_gemm_dx(x.to(device), Qd, Sd, d_in, offsets=off, y=y)
        terms = k * (1 if dtype == BF else 3)
    assert got is y
    v = f64(y)
    assert (v[:lo] == -77.0).all() and (v[hi:] == -77.0).all()
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        check(y[r], a[r], np.ascontiguousarray(W[e].T) if op == "gemm_dx" else W[e], terms, out, f"expert {e}")


@pytest.mark.parametrize("op", ["gemm", "gemm_mx", "gemm_dx"])
@pytest.mark.parametrize("n", [3, 40, 300])
def test_nan_and_infinity_stay_in_their_row(device, op, n):
    d_in, d_out = 320, 192
    rng = np.random.default_rng(n)
    Q, S, W = random_weight(rng, 1, d_out, d_in)
    S = S[0].copy()
    S[5, 1] = 255                                     # W[5, 32:64] is NaN
    k = d_out if op == "gemm_dx" else d_in
    x = torch.from_numpy(rng.standard_normal((n, k))).to(BF)
    Qd, Sd = u8(Q[0], device), u8(S, device)
    if op == "gemm_mx":
        x[1, 7] = float("nan")
        y = f64(gq.mxfp4_gemm_mx(*gq.mxfp4_quantize(x.to(device)), Qd, Sd, d_in))
    elif op == "gemm":
        x[1, 7], x[2, 200] = float("nan"), float("inf")
        y = f64(gq.mxfp4_gemm(x.to(device), Qd, Sd))
        assert not np.isfinite(y[2]).any()            # infinity times every weight (0 gives NaN)
    else:
        x[1, 7] = float("nan")
        y = f64(gq.mxfp4_gemm_dx(x.to(device), Qd, Sd, d_in))
    assert np.isnan(y[1]).all()
    col = slice(32, 64) if op == "gemm_dx" else slice(5, 6)
    assert np.isnan(y[:, col]).all()
    ok = np.ones(y.shape, bool)
    ok[1], ok[:, col] = False, False
    if op == "gemm":
        ok[2] = False
    assert np.isfinite(y[ok]).all()


@pytest.mark.parametrize("n", [2, 200])
def test_gemm_extreme_scales(device, n):
    """Weights at the ends of the scale range: 2^-127 (subnormal values in bfloat16) and 2^125,
    against activations that bring the products back into range."""
    d = 256
    rng = np.random.default_rng(4)
    Q, S, _ = random_weight(rng, 1, 64, d)
    for s, a in ((0, 2.0 ** 120), (1, 2.0 ** 120), (252, 2.0 ** -126), (252, 2.0 ** -120)):
        S1 = np.full_like(S[0], s)
        W = O.mx_values(Q[0], S1, d)
        for dtype in (BF, F32):
            x = torch.from_numpy(rng.standard_normal((n, d)) * a).to(dtype)
            y = gq.mxfp4_gemm(x.to(device), u8(Q[0], device), u8(S1, device), out_dtype=F32)
            # the third plane of a float32 ends at the smallest bfloat16, 2^-133: x 2^-149-grid
            # bits below it are cut, so a value is held to within 2^-133 (nothing is cut, and
            # the term is far below the bound, where |x| >= 2^-110)
            check(y, f64(x), W, d * 3, F32, f"s={s} {dtype}", lost=2.0 ** -133 if dtype == F32 else 0.0)


def test_float32_planes_are_exact(device):
    """One term a product: y = x w with w = +-1 returns float32 x to the bit, whatever its
    bits (three bfloat16 planes hold 24), and infinities and NaN as they are."""
    n, d = 40, 128
    W = np.eye(d)
    Q, S = O.mx_quantize(W)
    S[S == 0] = 127
    S[np.arange(d), np.arange(d) // 32] = 125          # the block with the 1 (4 units of 2^-2)
    rng = np.random.default_rng(0)
    x = (rng.integers(1 << 23, 1 << 24, (n, d)) * np.exp2(rng.integers(-100, 60, (n, d)))).astype(np.float32)
    x *= rng.choice([-1, 1], (n, d)).astype(np.float32)
    y = gq.mxfp4_gemm(torch.from_numpy(x).to(device), u8(Q, device), u8(S, device))
    np.testing.assert_array_equal(y.cpu().numpy(), x)


def test_bad_offsets_stay_in_range(device):
    """Offsets out of [0, n] or out of order: nothing outside y is touched and well-formed
    experts are right."""
    n, d, m, E = 50, 128, 64, 4
    rng = np.random.default_rng(1)
    Q, S, W = random_weight(rng, E, m, d)
    x = torch.from_numpy(rng.standard_normal((n, d))).to(BF)
    for op in ("gemm", "gemm_mx", "gemm_dx"):
        for off in ([-5, 10, 20, 1 << 40, 1 << 40], [0, 30, 10, 10, 50], [60, 70, 80, 90, 100]):
            width = d if op == "gemm_dx" else m
            buf = torch.full((n + 2, width), 3.0, device=device)
            o = torch.tensor(off, dtype=torch.int64, device=device)
            a, y = x, buf[1:n + 1]
            if op == "gemm_mx":
                gq.mxfp4_gemm_mx(*gq.mxfp4_quantize(a.to(device)), u8(Q, device), u8(S, device), d, offsets=o, y=y)
            elif op == "gemm":
                gq.mxfp4_gemm(a.to(device), u8(Q, device), u8(S, device), offsets=o, y=y)
            else:
                a = x[:, :m].contiguous()
                gq.mxfp4_gemm_dx(a.to(device), u8(Q, device), u8(S, device), d, offsets=o, y=y)
            assert (buf[0] == 3.0).all() and (buf[-1] == 3.0).all()
            if off[0] == -5 and op == "gemm":
                check(y[:10], f64(a)[:10], W[0], d, F32)
                check(y[20:50], f64(a)[20:50], W[2], d, F32)
            if off[0] == 60:
                assert (buf == 3.0).all()


def test_gradient_against_differences(device):
    """d(sum y g) / dx by the product itself: y is linear in x, so a difference over a step is
    the gradient's product with it."""
    n, d_in, d_out = 20, 256, 96
    rng = np.random.default_rng(9)
    Q, S, W = random_weight(rng, 1, d_out, d_in)
    Qd, Sd = u8(Q[0], device), u8(S[0], device)
    x = torch.from_numpy(rng.standard_normal((n, d_in))).to(F32).to(device)
    g = torch.from_numpy(rng.standard_normal((n, d_out))).to(F32).to(device)
    step = torch.from_numpy(rng.standard_normal((n, d_in))).to(F32).to(device)
    dx = gq.mxfp4_gemm_dx(g, Qd, Sd, d_in)
    y0, y1 = gq.mxfp4_gemm(x, Qd, Sd), gq.mxfp4_gemm(x + step, Qd, Sd)
    taken = f64(x + step) - f64(x)                    # the step as float32 holds it
    left = (f64(y1) - f64(y0)) * f64(g)
    right = f64(dx) * taken
    size = (np.abs(f64(x)) + np.abs(f64(x + step))) @ np.abs(W[0]).T
    slack = (3 * d_in + 8) * 2.0 ** -23 * (size * np.abs(f64(g))).sum()
    slack += (3 * d_out + 8) * 2.0 ** -23 * ((np.abs(f64(g)) @ np.abs(W[0])) * np.abs(taken)).sum()
    assert abs(left.sum() - right.sum()) <= slack
    assert slack < 0.05 * np.abs(right).sum()


def test_chain_of_a_quantised_expert_layer(device):
    """The operators as one runs them: pack the experts' weights and the routed activations,
    both products, and the gradient of the input, each against the oracle on its own inputs;
    twice, with equal bits."""
    E, n, d, h = 4, 150, 384, 288
    rng = np.random.default_rng(12)
    off_h = [0, 40, 40, 139, 146]
    off = torch.tensor(off_h, device=device)
    W1 = torch.from_numpy(rng.standard_normal((E, h, d)) * 0.05).to(BF).to(device)
    W2 = torch.from_numpy(rng.standard_normal((E, d, h)) * 0.05).to(BF).to(device)
    x = torch.from_numpy(rng.standard_normal((n, d))).to(BF).to(device)
    first = None
    for _ in range(2):
        Q1, S1 = gq.mxfp4_quantize(W1)
        Q2, S2 = gq.mxfp4_quantize(W2)
        XQ, XS = gq.mxfp4_quantize(x)
        u = gq.mxfp4_gemm_mx(XQ, XS, Q1, S1, d, offsets=off)
        v = gq.mxfp4_gemm(u, Q2, S2, offsets=off, out_dtype=F32)
        gu = gq.mxfp4_gemm_dx(v, Q2, S2, h, offsets=off)
        got = [t.clone() for t in (Q1, S1, XQ, u, v, gu)]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    w1 = O.mx_values(*O.mx_quantize(f64(W1).reshape(-1, d)), d).reshape(E, h, d)
    w2 = O.mx_values(*O.mx_quantize(f64(W2).reshape(-1, h)), h).reshape(E, d, h)
    a = O.mx_values(*O.mx_quantize(f64(x)), d)
    for e in range(E):
        r = slice(off_h[e], off_h[e + 1])
        check(u[r], a[r], w1[e], d, BF)
        check(v[r], f64(u)[r], w2[e], h, F32)
        check(gu[r], f64(v)[r], np.ascontiguousarray(w2[e].T), 3 * d, F32)
    assert (u[146:] == 0).all() and (v[146:] == 0).all() and (gu[146:] == 0).all()


@pytest.mark.parametrize("op", ["gemm", "gemm_mx", "gemm_dx"])
@pytest.mark.parametrize("n", [4, 40, 300])
def test_graph_replays_and_side_streams(device, op, n):
    """A captured call, replayed with new inputs in place between eager calls, and a call on
    another stream, give the eager results' bits; two graphs share a workspace."""
    d_in, d_out = 1024, 512
    rng = np.random.default_rng(n)
    Q, S, _ = random_weight(rng, 1, d_out, d_in)
    Qd, Sd = u8(Q[0], device), u8(S[0], device)
    k, width = (d_out, d_in) if op == "gemm_dx" else (d_in, d_out)
    xs = [torch.randn(n, k, device=device) for _ in range(4)]

    def call(x, y=None, ws=None, stream=None):
        if op == "gemm_mx":
            XQ, XS = gq.mxfp4_quantize(x, stream=stream)
            return gq.mxfp4_gemm_mx(XQ, XS, Qd, Sd, d_in, y=y, ws=ws, out_dtype=F32, stream=stream)
        if op == "gemm":
            return gq.mxfp4_gemm(x, Qd, Sd, y=y, ws=ws, stream=stream)
        return gq.mxfp4_gemm_dx(x, Qd, Sd, d_in, y=y, ws=ws, stream=stream)

    want = [call(x).clone() for x in xs]
    size = {"gemm": gq.mxfp4_gemm_workspace_size, "gemm_mx": lambda *a: gq.mxfp4_gemm_mx_workspace_size(*a[:4]),
            "gemm_dx": gq.mxfp4_gemm_dx_workspace_size}[op](n, d_in, d_out, 1, gq.GQ_F32)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=device)
    x1, x2 = xs[0].clone(), xs[1].clone()
    y1, y2 = torch.empty(n, width, device=device), torch.empty(n, width, device=device)
    torch.cuda.synchronize()
    graphs = []
    for x, y in ((x1, y1), (x2, y2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x, y=y, ws=ws)
        graphs.append(g)
    for rep in range(3):
        x1.copy_(xs[rep]), x2.copy_(xs[rep + 1])
        y1.fill_(-1.0), y2.fill_(-1.0)
        graphs[0].replay(), graphs[1].replay()
        eager = call(xs[rep])
        torch.cuda.synchronize()
        assert torch.equal(y1, want[rep]) and torch.equal(y2, want[rep + 1]) and torch.equal(eager, want[rep])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ys = [call(x, stream=side) for x in xs]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))


def test_no_rows(device):
    Q, S = gq.mxfp4_quantize(torch.randn(32, 64, device=device))
    assert gq.mxfp4_quantize(torch.empty(0, 64, device=device))[0].shape == (0, 64)
    assert gq.mxfp4_gemm(torch.empty(0, 64, device=device), Q, S).shape == (0, 32)
    assert gq.mxfp4_gemm_dx(torch.empty(0, 32, device=device), Q, S, 64).shape == (0, 64)
    assert gq.mxfp4_dequantize(Q[:0], S[:0], 64).shape == (0, 64)


def test_library_allocated_workspace(device):
    x = torch.randn(40, 200, device=device)
    Q, S = gq.mxfp4_quantize(torch.randn(96, 200, device=device))
    assert torch.equal(gq.mxfp4_gemm(x, Q, S, ws=False), gq.mxfp4_gemm(x, Q, S))


def test_refusals_on_the_device(device):
    x = torch.randn(8, 256, device=device, dtype=BF)
    Q, S = gq.mxfp4_quantize(torch.randn(64, 256, device=device))

    def status(fn, *a, **k):
        with pytest.raises(gq.GQError) as ei:
            fn(*a, **k)
        return ei.value.status

    assert status(gq.mxfp4_gemm, x.to(torch.float16), Q, S) == 3
    assert status(gq.mxfp4_gemm, x, Q, S, y=torch.empty(8, 64, device=device), out_dtype=BF) == 3
    assert status(gq.mxfp4_gemm, x, Q, S, y=torch.empty(8, 65, device=device)) == 2
    assert status(gq.mxfp4_gemm, x.t().contiguous().t(), Q, S) == 1              # strided
    assert status(gq.mxfp4_gemm, x, Q.to(torch.int8), S) == 3
    assert status(gq.mxfp4_gemm, x, Q[None], S[None], offsets=torch.zeros(2, dtype=torch.int32, device=device)) == 3
    assert status(gq.mxfp4_gemm, x, Q[None], S[None], offsets=torch.zeros(2, dtype=torch.int64)) == 1   # host
    flat = torch.zeros(8 * 256 + 1, device=device, dtype=BF)
    assert status(gq.mxfp4_gemm, flat[1:].view(8, 256), Q, S) == 1               # not 16-byte aligned
    need = gq.mxfp4_gemm_workspace_size(8, 256, 64, 1, gq.GQ_F32)
    if need:
        assert status(gq.mxfp4_gemm, x.float(), Q, S, ws=torch.empty(need - 1, dtype=torch.uint8, device=device)) == 1


def test_output_on_the_input_is_refused(device):
    x = torch.randn(40, 128, device=device)
    Q, S = gq.mxfp4_quantize(torch.randn(128, 128, device=device))
    for fn in (lambda: gq.mxfp4_gemm(x, Q, S, y=x), lambda: gq.mxfp4_gemm_dx(x, Q, S, 128, y=x)):
        with pytest.raises(gq.GQError) as e:
            fn()
        assert e.value.status == 1 and "overlap" in e.value.message


@pytest.mark.parametrize("n", [3, 40, 200])
def test_views_off_the_vector_borders(device, n):
    """Outputs, and float32 inputs, that start one element off a 16-byte border."""
    d, m = 256, 64
    rng = np.random.default_rng(n)
    Q, S, W = random_weight(rng, 1, m, d)
    Qd, Sd = u8(Q[0], device), u8(S[0], device)
    flat = torch.randn(1 + n * d, device=device)
    x = flat[1:].view(n, d)
    for out in (BF, F32):
        buf = torch.full((2 + n * m,), 5.0, dtype=out, device=device)
        gq.mxfp4_gemm(x, Qd, Sd, y=buf[1:1 + n * m].view(n, m))
        assert float(buf[0]) == 5.0 and float(buf[-1]) == 5.0
        check(buf[1:1 + n * m].view(n, m), f64(x), W[0], 3 * d, out)
        buf = torch.full((2 + n * d,), 5.0, dtype=out, device=device)
        g = torch.randn(1 + n * m, device=device)[1:].view(n, m)
        gq.mxfp4_gemm_dx(g, Qd, Sd, d, y=buf[1:1 + n * d].view(n, d))
        assert float(buf[0]) == 5.0 and float(buf[-1]) == 5.0
        check(buf[1:1 + n * d].view(n, d), f64(g), np.ascontiguousarray(W[0].T), 3 * m, out)


@pytest.mark.parametrize("op", ["gemm", "gemm_mx", "gemm_dx"])
@pytest.mark.parametrize("E,n", [(130, 600), (130, 4500), (64, 640)])
def test_many_and_skewed_experts(device, op, E, n):
    """More experts than a wave counts at once, most of them empty, one with most of the rows."""
    d, m = 160, 96
    rng = np.random.default_rng(E + n)
    counts = np.zeros(E, np.int64)
    counts[rng.choice(E, 9, replace=False)] = rng.integers(1, n // 20, 9)
    counts[E // 2] += n - counts.sum() - 5
    offsets = np.concatenate([[0], np.cumsum(counts)])
    Q, S, W = random_weight(rng, E, m, d)
    off = torch.from_numpy(offsets).to(device)
    k, width = (m, d) if op == "gemm_dx" else (d, m)
    y = torch.full((n, width), -1.0, device=device)
    if op == "gemm_mx":
        XQ, XS, X = random_weight(rng, 1, n, d)
        a = X[0]
        gq.mxfp4_gemm_mx(u8(XQ[0], device), u8(XS[0], device), u8(Q, device), u8(S, device), d, offsets=off, y=y)
    else:
        x = torch.from_numpy(rng.standard_normal((n, k))).to(BF)
        a = f64(x)
        if op == "gemm":
            gq.mxfp4_gemm(x.to(device), u8(Q, device), u8(S, device), offsets=off, y=y)
        else:
            gq.mxfp4_gemm_dx(x.to(device), u8(Q, device), u8(S, device), d, offsets=off, y=y)
    assert (y[offsets[-1]:] == -1.0).all()
    for e in np.nonzero(counts)[0]:
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        check(y[r], a[r], np.ascontiguousarray(W[e].T) if op == "gemm_dx" else W[e], k, F32, f"expert {e}")


@pytest.mark.parametrize("op", ["gemm", "gemm_mx", "gemm_dx"])
@pytest.mark.parametrize("d_in", [2100, 1200])
def test_experts_of_large_tiles(device, op, d_in):
    """Ragged experts with enough rows and columns for the largest tiles, and (fp4, up to 2048
    values) for the smaller ones that short contractions take; a contraction of an odd number of
    128s; an output width that is no multiple of 8."""
    offsets, d_out = [5, 900, 901, 2090], 4603
    n, E = 2100, 3
    rng = np.random.default_rng(d_in)
    Q, S, W = random_weight(rng, E, d_out, d_in)
    off = torch.tensor(offsets, dtype=torch.int64, device=device)
    Qd, Sd = u8(Q, device), u8(S, device)
    k, m = (d_out, d_in) if op == "gemm_dx" else (d_in, d_out)
    y = torch.full((n, m), -77.0, dtype=BF, device=device)
    if op == "gemm_mx":
        XQ, XS, X = random_weight(rng, 1, n, d_in)
        a = X[0]
        gq.mxfp4_gemm_mx(u8(XQ[0], device), u8(XS[0], device), Qd, Sd, d_in, offsets=off, y=y)
    else:
        x = torch.from_numpy(rng.standard_normal((n, k))).to(BF)
        a = f64(x)
        if op == "gemm":
            gq.mxfp4_gemm(x.to(device), Qd, Sd, offsets=off, y=y)
        else:
            gq.mxfp4_gemm_dx(x.to(device), Qd, Sd, d_in, offsets=off, y=y)
    v = f64(y)
    assert (v[:5] == -77.0).all() and (v[2090:] == -77.0).all()
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        check(y[r], a[r], np.ascontiguousarray(W[e].T) if op == "gemm_dx" else W[e], k, BF, f"expert {e}")


@pytest.mark.parametrize("op", ["gemm", "gemm_mx", "gemm_dx"])
@pytest.mark.parametrize("n,k", [(4200, 333), (3856, 1100), (3861, 1104)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_behind_full_rounds_of_tiles(device, op, n, k, dtype):
    """17 columns of large tiles: 3840 rows fill a round of them, the others are a product of
    their own (360 rows by tiles, 16 streamed or split, 21 split).  The same from a captured
    graph, and as one expert that leaves rows at both ends alone, which is not divided."""
    m = 4200
    rng = np.random.default_rng(n + k)
    d_in, d_out = (m, k) if op == "gemm_dx" else (k, m)
    Q, S, W = random_weight(rng, 1, d_out, d_in)
    Qd, Sd = u8(Q[0], device), u8(S[0], device)
    V = np.ascontiguousarray(W[0].T) if op == "gemm_dx" else W[0]
    if op == "gemm_mx":
        XQ, XS, X = random_weight(rng, 1, n, k)
        a, xq, xs, terms = X[0], u8(XQ[0], device), u8(XS[0], device), k
        call = lambda Q, S, **o: gq.mxfp4_gemm_mx(xq, xs, Q, S, d_in, **o)
    else:
        x = torch.from_numpy(rng.standard_normal((n, k))).to(dtype)
        a, x, terms = f64(x), x.to(device), k * (1 if dtype == BF else 3)
        if op == "gemm":
            call = lambda Q, S, **o: gq.mxfp4_gemm(x, Q, S, **o)
        else:
            call = lambda Q, S, **o: gq.mxfp4_gemm_dx(x, Q, S, d_in, **o)
    y = torch.full((n, m), -77.0, dtype=dtype, device=device)
    call(Qd, Sd, y=y)
    check(y, a, V, terms, dtype, "all rows")
    z = torch.zeros_like(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(Qd, Sd, y=z)
    for _ in range(3):
        z.zero_()
        g.replay()
        assert torch.equal(y, z)
    off = torch.tensor([7, n - 9], dtype=torch.int64, device=device)
    z.fill_(-77.0)
    call(Qd[None], Sd[None], y=z, offsets=off)
    assert (z[:7] == -77.0).all() and (z[n - 9:] == -77.0).all()
    check(z[7:n - 9], a[7:n - 9], V, terms, dtype, "one expert")


@pytest.mark.parametrize("dtype,d_out", [(BF, 6200), (F32, 2060), (BF, 2060)])
def test_gradient_of_a_weight_in_thirds(device, dtype, d_out):
    """144 large tiles: long contractions are split in three, the last of 2060 values is not."""
    n, d_in = 2244, 4096
    rng = np.random.default_rng(d_out)
    Q, S, W = random_weight(rng, 1, d_out, d_in)
    g = torch.from_numpy(rng.standard_normal((n, d_out))).to(dtype)
    dx = gq.mxfp4_gemm_dx(g.to(device), u8(Q[0], device), u8(S[0], device), d_in)
    check(dx, f64(g), np.ascontiguousarray(W[0].T), d_out * (1 if dtype == BF else 3), dtype)


def test_rows_past_32_bits(device):
    """Activations of more than 2^31 elements and 4 GiB: the last rows are those of a call on them
    alone (to the sums' rounding), and packing them equals packing the last rows alone."""
    n, d, m, t = 140000, 16384, 48, 40
    gen = torch.Generator(device=device)
    gen.manual_seed(1)
    x = torch.randn((n, d), generator=gen, device=device, dtype=BF)
    W = torch.randn((m, d), generator=gen, device=device)
    Q, S = gq.mxfp4_quantize(W)
    w = O.mx_values(Q.cpu().numpy(), S.cpu().numpy(), d)
    y = gq.mxfp4_gemm(x, Q, S, out_dtype=F32)
    check(y[-t:], f64(x[-t:]), w, d, F32, "gemm")
    XQ, XS = gq.mxfp4_quantize(x)
    TQ, TS = gq.mxfp4_quantize(x[-t:].contiguous())
    assert torch.equal(XQ[-t:], TQ) and torch.equal(XS[-t:], TS)
    z = gq.mxfp4_gemm_mx(XQ, XS, Q, S, d, out_dtype=F32)
    check(z[-t:], O.mx_values(TQ.cpu().numpy(), TS.cpu().numpy(), d), w, d, F32, "gemm_mx")
    del XQ, XS, x
    g = torch.randn((n, m), generator=gen, device=device, dtype=BF)
    dx = gq.mxfp4_gemm_dx(g, Q, S, d)                  # 2.3e9 outputs
    check(dx[-t:], f64(g[-t:]), np.ascontiguousarray(w.T), m, BF, "gemm_dx")
    del dx


def test_weights_past_32_bits(device):
    """Codes of more than 4 GiB: the last expert's product."""
    E, m, d, n = 36, 16384, 16384, 24
    Q = torch.randint(0, 256, (E, m, d // 2), dtype=torch.uint8, device=device)
    S = torch.randint(110, 125, (E, m, d // 32), dtype=torch.uint8, device=device)
    off = torch.tensor([0] * E + [n], device=device)
    x = torch.randn(n, d, device=device, dtype=BF)
    y = gq.mxfp4_gemm(x, Q, S, offsets=off, out_dtype=F32)
    rows = torch.arange(0, m, 1031)
    w = O.mx_values(Q[-1, rows].cpu().numpy(), S[-1, rows].cpu().numpy(), d)
    check(y[:, rows], f64(x), w, d, F32)
    dx = gq.mxfp4_gemm_dx(y.to(BF), Q, S, d, offsets=off, out_dtype=F32)
    cols = slice(d - 64, d)
    wc = gq.mxfp4_dequantize(Q[-1].contiguous(), S[-1].contiguous(), d, dtype=F32)[:, cols]
    check(dx[:, cols], f64(y.to(BF)), np.ascontiguousarray(f64(wc).T), m, F32)
