"""GPU tests of the gated feed-forward block with bfloat16 weights, forward and back, against float64
(bounds: _product_cases)."""
import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_gq_amd as gq
from _product_cases import BF, EPS, F32, act64, check, check_product, counts, f64, gate64, normal, of, spans

pytestmark = pytest.mark.gpu

SIZES = [(1, 64, 64), (1, 1, 1), (1, 4096, 1408), (3, 130, 200), (16, 1000, 333), (17, 257, 129), (40, 640, 1000),
         (64, 1408, 264), (65, 384, 300), (129, 1024, 257), (200, 2047, 1001), (256, 256, 256), (513, 520, 384),
         (1000, 300, 2100)]
GROUPED = [(5, 200, 130, 3), (33, 256, 384, 4), (96, 512, 256, 40), (300, 640, 264, 6), (700, 257, 520, 9), (1500, 1000, 384, 3),
           (64, 300, 200, 130)]


def operands(device, n, d_in, d_ff, experts=None, seed=0):
    shape = (d_ff, d_in) if experts is None else (experts, d_ff, d_in)
    x = normal(device, n, d_in, seed=seed, dtype=BF, spread=0.5)
    G, U = (normal(device, *shape, seed=seed + k, dtype=BF, scale=d_in ** -0.5, spread=0.3) for k in (1, 2))
    return x, G, U


def check_gate(h, x, G, U, act, at, out, saved=None):
    done = torch.zeros(x.shape[0], dtype=torch.bool)
    for e, r in spans(x.shape[0], at):
        ref, limit, zg, zu, bg, bu = gate64(x[r].double(), of(G, e).double(), of(U, e).double(), act, x.shape[1])
        check(h[r], ref, limit, out, "h")
        if saved:
            check(saved[0][r], zg, bg, F32, "zg")
            check(saved[1][r], zu, bu, F32, "zu")
        done[r] = True
    assert not h[~done].double().abs().sum().item()


@pytest.mark.parametrize("act,out", [("silu", BF), ("gelu", F32), ("gelu_tanh", BF)])
@pytest.mark.parametrize("n,d_in,d_ff", SIZES)
def test_gate(device, n, d_in, d_ff, act, out):
    x, G, U = operands(device, n, d_in, d_ff)
    h, zg, zu = gq.ffn_gate(x, G, U, act=act, out_dtype=out, save=True)
    assert h.dtype == out and zg.dtype == zu.dtype == F32 and h.shape == (n, d_ff)
    check_gate(h, x, G, U, act, None, out, (zg, zu))
    assert torch.equal(h, gq.ffn_gate(x, G, U, act=act, out_dtype=out))


@pytest.mark.parametrize("n,d_in,d_ff,experts", GROUPED)
def test_gate_of_experts(device, n, d_in, d_ff, experts):
    x, G, U = operands(device, n, d_in, d_ff, experts)
    at = counts(n, experts, seed=n)
    offsets = torch.tensor(at, device=device)
    h, zg, zu = gq.ffn_gate(x, G, U, offsets=offsets, save=True)
    check_gate(h, x, G, U, "silu", at, BF, (zg, zu))
    given = torch.full_like(h, 7.0)
    assert gq.ffn_gate(x, G, U, offsets=offsets, y=given) is given
    assert bool((given[:at[0]] == 7).all()) and bool((given[at[-1]:] == 7).all())
    assert torch.equal(given[at[0]:at[-1]], h[at[0]:at[-1]])


# ---- the backward pass ------------------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("count,at", [(1, 0), (7, 0), (8, 0), (1001, 0), (4096, 0), (65537, 1)])
def test_dz(device, count, at, dtype, act):
    """Element by element, with views off the 16-byte borders."""
    dh = normal(device, count + at, seed=1, dtype=dtype)[at:]
    zg = (4 * normal(device, count + at, seed=2))[at:]
    zu = normal(device, count + at, seed=3)[at:]
    if count > 100:
        zg[:20] = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 100, -100, 1e20, -1e20] * 2, device=device)
    a, b = gq.ffn_gate_dz(dh, zg, zu, act=act)
    v, slope = (torch.from_numpy(t).to(device) for t in O.ffn_act(f64(zg), act))
    d, u = dh.double(), zu.double()
    loose = 36 * EPS * (1 + zg.double() ** 2)
    # the slope's terms cancel near its zero only, which lies within |z| < 8
    size = torch.where(zg.abs() < 8, slope.abs().clamp_min(1.0), slope.abs())
    check(a, d * u * slope, loose * (d * u).abs() * size + 1e-30, BF, "dzg")
    check(b, d * v, loose * (d * v).abs() + 1e-30, BF, "dzu")


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n,d_in,d_ff", SIZES)
def test_dx(device, n, d_in, d_ff, out):
    _, G, U = operands(device, n, d_in, d_ff)
    a, b = normal(device, n, d_ff, seed=5, dtype=BF), normal(device, n, d_ff, seed=6, dtype=BF)
    dx = gq.ffn_gate_dx(a, b, G, U, out_dtype=out)
    both, W = torch.cat([a, b], 1).double(), torch.cat([G, U]).double()
    check_product(dx, both, W.T, None, 2 * d_ff, out, "dx")
    assert torch.equal(dx, gq.ffn_gate_dx(a, b, G, U, out_dtype=out))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n,d_in,d_ff", SIZES)
def test_dw(device, n, d_in, d_ff, out):
    x = normal(device, n, d_in, seed=1, dtype=BF)
    a, b = normal(device, n, d_ff, seed=5, dtype=BF), normal(device, n, d_ff, seed=6, dtype=BF)
    got = gq.ffn_gate_dw(a, b, x, out_dtype=out)
    for d, g in zip(got, (a, b)):
        assert d.shape == (d_ff, d_in) and d.dtype == out
        check_product(d, g.double().T, x.double().T, None, n, out, "dw")
    one = gq.ffn_gate_dw(a, b, x, out_dtype=out, which=(False, True))
    assert one[0] is None and torch.equal(one[1], got[1])
    one = gq.ffn_gate_dw(a, b, x, out_dtype=out, which=(True, False))
    assert one[1] is None and torch.equal(one[0], got[0])


@pytest.mark.parametrize("n,d_in,d_ff,experts", GROUPED)
def test_gradients_of_experts(device, n, d_in, d_ff, experts):
    x, G, U = operands(device, n, d_in, d_ff, experts)
    at = counts(n, experts, seed=n)
    offsets = torch.tensor(at, device=device)
    a, b = normal(device, n, d_ff, seed=5, dtype=BF), normal(device, n, d_ff, seed=6, dtype=BF)
    dx = gq.ffn_gate_dx(a, b, G, U, offsets=offsets, out_dtype=F32)
    dG, dU = gq.ffn_gate_dw(a, b, x, experts=experts, offsets=offsets, out_dtype=F32)
    both, W = torch.cat([a, b], 1).double(), torch.cat([G, U], 1).double()
    check_product(dx, both, W.transpose(1, 2), at, 2 * d_ff, F32, "dx")
    for e, r in spans(n, at):
        for d, g in ((dG, a), (dU, b)):
            check_product(d[e], g[r].double().T, x[r].double().T, None, r.stop - r.start, F32, "dw")
    given = torch.full_like(dx, 7.0)
    gq.ffn_gate_dx(a, b, G, U, offsets=offsets, y=given)
    assert bool((given[:at[0]] == 7).all()) and bool((given[at[-1]:] == 7).all())


def test_no_rows(device):
    """Outputs of no rows; weights' gradients of zero, over whatever was there."""
    x, G, U = operands(device, 8, 200, 130)
    z = torch.empty(0, 130, dtype=BF, device=device)
    assert gq.ffn_gate(x[:0], G, U).shape == (0, 130)
    assert gq.ffn_gate_dx(z, z, G, U).shape == (0, 200)
    dG = torch.full((130, 200), 7.0, dtype=BF, device=device)
    got = gq.ffn_gate_dw(z, z, x[:0], dG=dG)
    assert got[0] is dG and not dG.any() and not got[1].any()
    leaves = [t.clone().requires_grad_() for t in (x[:0], G, U)]
    gq.ffn_gate(*leaves).sum().backward()
    assert leaves[0].grad.shape == (0, 200) and not leaves[1].grad.any() and not leaves[2].grad.any()


def test_nonfinite_stays_in_its_row(device):
    x, G, U = operands(device, 70, 300, 200)
    x[13, 5], x[20, 299] = float("inf"), float("nan")
    bad = torch.isfinite(gq.ffn_gate(x, G, U, out_dtype=F32)).logical_not()
    assert bool(bad[13].any()) and bool(bad[20].all())
    bad[13], bad[20] = False, False
    assert not bad.any()
    a, b = normal(device, 70, 200, seed=1, dtype=BF), normal(device, 70, 200, seed=2, dtype=BF)
    a[7, 199] = float("nan")
    bad = torch.isnan(gq.ffn_gate_dx(a, b, G, U))
    assert bool(bad[7].all()) and int(bad.sum()) == 300
    bad = torch.isnan(gq.ffn_gate_dw(a, b, normal(device, 70, 300, seed=3, dtype=BF))[0])
    assert bool(bad[199].all()) and int(bad.sum()) == 300


# ---- through autograd -------------------------------------------------------------------

@pytest.mark.parametrize("experts", [None, 3])
@pytest.mark.parametrize("out", [None, F32])
def test_gradients_through_autograd(device, experts, out):
    """Each leaf's gradient is the entry points'; leaves that need none get none."""
    n, d_in, d_ff = 90, 264, 130
    x, G, U = operands(device, n, d_in, d_ff, experts)
    at = [4, 30, 30, 80]
    offsets = torch.tensor(at, device=device) if experts else None
    dh = normal(device, n, d_ff, seed=9, dtype=out or BF)
    h, zg, zu = gq.ffn_gate(x, G, U, act="gelu", offsets=offsets, out_dtype=out, save=True)
    dzg, dzu = gq.ffn_gate_dz(dh, zg, zu, act="gelu")
    want = [gq.ffn_gate_dx(dzg, dzu, G, U, offsets=offsets), *gq.ffn_gate_dw(dzg, dzu, x, experts=experts, offsets=offsets)]
    for mask in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1)):
        leaves = [t.clone().requires_grad_(bool(m)) for t, m in zip((x, G, U), mask)]
        y = gq.ffn_gate(*leaves, act="gelu", offsets=offsets, out_dtype=out)
        assert y.requires_grad and torch.equal(y.detach(), h)
        y.backward(dh)
        for leaf, m, w in zip(leaves, mask, want):
            assert (leaf.grad is None) if not m else torch.equal(leaf.grad, w)
    if experts:
        assert not want[0][:4].any() and not want[0][80:].any() and not want[1][1].any()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_the_formula(device, act):
    """End to end: the errors of h's products, of dz's rounding (2^-8) and of the sums after it."""
    n, d_in, d_ff = 100, 200, 160
    x, G, U = operands(device, n, d_in, d_ff)
    dh = normal(device, n, d_ff, seed=9, dtype=BF)
    leaves = [t.clone().requires_grad_() for t in (x, G, U)]
    gq.ffn_gate(*leaves, act=act).backward(dh)
    X, g, u, d = (t.double() for t in (x, G, U, dh))
    zg, zu = X @ g.T, X @ u.T
    v, s = act64(zg, act)
    dzg, dzu = d * zu * s, d * v
    # |act''| <= 1.3 for all three; products off by at most (d_in + 8) 2^-23 sum |x w|
    bg, bu = ((d_in + 8) * EPS * (X.abs() @ w.T.abs()) for w in (g, u))
    eg = 2.0 ** -8 * dzg.abs() + d.abs() * (1.2 * bu + 1.3 * bg * zu.abs() + 40 * EPS * (1 + zg * zg) * zu.abs()) * 1.01
    eu = 2.0 ** -8 * dzu.abs() + d.abs() * (1.2 * bg + 40 * EPS * (1 + zg * zg) * v.abs()) * 1.01
    sums = 400 * EPS
    check(leaves[0].grad, dzg @ g + dzu @ u, eg @ g.abs() + eu @ u.abs() + sums * (dzg.abs() @ g.abs() + dzu.abs() @ u.abs()), BF, "dx")
    check(leaves[1].grad, dzg.T @ X, eg.T @ X.abs() + sums * (dzg.T.abs() @ X.abs()), BF, "dG")
    check(leaves[2].grad, dzu.T @ X, eu.T @ X.abs() + sums * (dzu.T.abs() @ X.abs()), BF, "dU")


def test_gradient_against_differences(device):
    """The slope of h . dh along a direction of each leaf, by central differences of the forward
    pass in float32 outputs."""
    n, d_in, d_ff = 32, 128, 64
    x, G, U = operands(device, n, d_in, d_ff)
    dh = normal(device, n, d_ff, seed=9, dtype=F32)
    leaves = [t.clone().requires_grad_() for t in (x, G, U)]
    gq.ffn_gate(*leaves, out_dtype=F32).backward(dh)

    def value(ts):
        X, g, u = (t.double() for t in ts)
        return (act64(X @ g.T, "silu")[0] * (X @ u.T) * dh.double()).sum()

    for k in range(3):
        step = normal(device, *leaves[k].shape, seed=20 + k).double()
        e = 1e-5
        hi = [t.detach().double() + (e * step if i == k else 0) for i, t in enumerate(leaves)]
        lo = [t.detach().double() - (e * step if i == k else 0) for i, t in enumerate(leaves)]
        slope = (value(hi) - value(lo)) / (2 * e)
        got = (leaves[k].grad.double() * step).sum()
        # every entry of the gradient is off by at most 2^-7 of its terms' sizes (two bfloat16 roundings):
        # that many independent roundings of random sign stay below 8 standard deviations
        size = (leaves[k].grad.double() * step).norm()
        assert abs(got - slope) <= 8 * 2.0 ** -7 * size, k


def test_a_second_gradient_is_refused(device):
    x, G, U = operands(device, 8, 64, 64)
    x.requires_grad_()
    g, = torch.autograd.grad(gq.ffn_gate(x, G, U).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_saved_products_feed_the_fisher(device):
    """A calibration step: X and dl/dZ of both projections into their Fishers."""
    n, d_in, d_ff, groups = 256, 128, 256, 2
    x, G, U = operands(device, n, d_in, d_ff)
    h, zg, zu = gq.ffn_gate(x, G, U, save=True)
    dzg, dzu = gq.ffn_gate_dz(normal(device, n, d_ff, seed=3, dtype=BF), zg, zu)
    for dz in (dzg, dzu):
        F = gq.gq_fisher_accumulate(x, dz, groups)
        ref = O.fisher(f64(x), f64(dz), groups)
        assert np.linalg.norm(f64(F) - ref) <= 1e-2 * np.linalg.norm(ref)
