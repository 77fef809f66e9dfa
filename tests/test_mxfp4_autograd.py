"""Activations that require a gradient: mxfp4_gemm and mxfp4_gemm_dx pass it on, each by the other.

Tolerances as in the other MXFP4 tests: T float32 additions of exact products are off by at most
(T + 8) 2^-23 sum |a w|, and a bfloat16 result by half a step more.
"""
import numpy as np
import pytest
import torch

import post_weight_quantization_gq_amd as gq
from post_weight_quantization_gq_amd import binding as B

BF, F32 = torch.bfloat16, torch.float32


def test_refusals_of_activations_that_require_a_gradient():
    """A given output would cut the graph; host tensors are refused as without a gradient."""
    Q, S = torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 8, dtype=torch.uint8)
    x = torch.zeros(5, 200, requires_grad=True)
    g = torch.zeros(5, 64, requires_grad=True)

    def refused(fn, *a, **k):
        with pytest.raises(B.GQError) as e:
            fn(*a, **k)
        return e.value

    e = refused(gq.mxfp4_gemm, x, Q, S, y=torch.zeros(5, 64))
    assert e.status == B.GQ_EINVAL and "gradient" in e.message
    e = refused(gq.mxfp4_gemm_dx, g, Q, S, 200, y=torch.zeros(5, 200))
    assert e.status == B.GQ_EINVAL and "gradient" in e.message
    assert "GPU tensor" in refused(gq.mxfp4_gemm, x, Q, S).message
    assert "GPU tensor" in refused(gq.mxfp4_gemm_dx, g, Q, S, 200).message
    with torch.no_grad():
        assert "GPU tensor" in refused(gq.mxfp4_gemm, x, Q, S, y=torch.zeros(5, 64)).message


def _weight(device, d_out, d_in, experts=None, seed=0):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    shape = (d_out, d_in) if experts is None else (experts, d_out, d_in)
    return gq.mxfp4_quantize(torch.randn(shape, generator=gen, device=device))


def _rand(device, *shape, seed, dtype=F32):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device=device).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 24, 300])
@pytest.mark.parametrize("dtype,out", [(BF, None), (BF, F32), (F32, None), (F32, BF)])
@pytest.mark.parametrize("grouped", [False, True])
def test_gradient_of_a_product(device, n, dtype, out, grouped):
    """The gradient is mxfp4_gemm_dx's, in x's type, and the formula's; the product is the same
    with and without one; rows of no expert have a gradient of zero."""
    d_in, d_out, E = 520, 264, 3
    Q, S = _weight(device, d_out, d_in, E if grouped else None)
    at = [n // 6, n // 3, n // 3, n - n // 8]
    off = torch.tensor(at, device=device) if grouped else None
    x = _rand(device, n, d_in, seed=1, dtype=dtype)
    g = _rand(device, n, d_out, seed=2, dtype=out or dtype)
    plain = gq.mxfp4_gemm(x, Q, S, offsets=off, out_dtype=out)
    assert not plain.requires_grad
    leaf = x.clone().requires_grad_()
    y = gq.mxfp4_gemm(leaf, Q, S, offsets=off, out_dtype=out)
    assert y.requires_grad and y.dtype == (out or dtype) and torch.equal(y.detach(), plain)
    y.backward(g)
    assert leaf.grad.dtype == dtype
    assert torch.equal(leaf.grad, gq.mxfp4_gemm_dx(g, Q, S, d_in, offsets=off, out_dtype=dtype))
    W = gq.mxfp4_dequantize(Q, S, d_in, dtype=F32).double()
    terms = d_out * (3 if g.dtype == F32 else 1)
    parts = [(W[e], slice(at[e], at[e + 1])) for e in range(E)] if grouped else [(W, slice(0, n))]
    for w, r in parts:
        ref, size = g[r].double() @ w, g[r].double().abs() @ w.abs()
        limit = (terms + 8) * 2.0 ** -23 * size
        if dtype == BF:
            limit += 2.0 ** -8 * ref.abs() + 2.0 ** -134
        assert ((leaf.grad[r].double() - ref).abs() <= limit).all()
    if grouped:
        assert (leaf.grad[:at[0]] == 0).all() and (leaf.grad[at[-1]:] == 0).all()
    with torch.no_grad():
        assert not gq.mxfp4_gemm(leaf, Q, S, offsets=off).requires_grad


@pytest.mark.gpu
def test_gradient_against_differences(device):
    """y is linear in x: the loss's difference over a step is the gradient's product with it."""
    n, d_in, d_out = 20, 256, 96
    Q, S = _weight(device, d_out, d_in)
    x = _rand(device, n, d_in, seed=1).requires_grad_()
    g = _rand(device, n, d_out, seed=2)
    step = _rand(device, n, d_in, seed=3)
    (gq.mxfp4_gemm(x, Q, S) * g).sum().backward()
    x0, x1 = x.detach(), x.detach() + step
    taken = x1.double() - x0.double()
    left = ((gq.mxfp4_gemm(x1, Q, S).double() - gq.mxfp4_gemm(x0, Q, S).double()) * g.double()).sum()
    right = (x.grad.double() * taken).sum()
    w = gq.mxfp4_dequantize(Q, S, d_in, dtype=F32).double().abs()
    slack = (3 * d_in + 8) * 2.0 ** -23 * (((x0.double().abs() + x1.double().abs()) @ w.T) * g.double().abs()).sum()
    slack += (3 * d_out + 8) * 2.0 ** -23 * ((g.double().abs() @ w) * taken.abs()).sum()
    assert abs(float(left - right)) <= float(slack)


@pytest.mark.gpu
def test_gradient_of_the_gradient(device):
    """d (v . dx) / dg is the product of v, through mxfp4_gemm_dx and through a backward pass that
    is recorded itself."""
    n, d_in, d_out = 40, 384, 136
    Q, S = _weight(device, d_out, d_in)
    g = _rand(device, n, d_out, seed=2).requires_grad_()
    v = _rand(device, n, d_in, seed=3)
    want = gq.mxfp4_gemm(v, Q, S)
    (got,) = torch.autograd.grad(gq.mxfp4_gemm_dx(g, Q, S, d_in), g, v)
    assert torch.equal(got, want)
    x = _rand(device, n, d_in, seed=1).requires_grad_()
    (dx,) = torch.autograd.grad(gq.mxfp4_gemm(x, Q, S), x, g, create_graph=True)
    (got,) = torch.autograd.grad(dx, g, v)
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_chain_of_layers(device, dtype):
    """Two quantised layers with a bias between them: the gradient is the two products in turn,
    from gradients that arrive expanded, and as a part of a larger one off 16 bytes."""
    n, d, h = 30, 256, 384
    Q1, S1 = _weight(device, h, d, seed=1)
    Q2, S2 = _weight(device, d, h, seed=2)
    x = _rand(device, n, d, seed=3, dtype=dtype).requires_grad_()
    bias = _rand(device, h, seed=4, dtype=dtype).requires_grad_()

    def layers(x):
        return gq.mxfp4_gemm(gq.mxfp4_gemm(x, Q1, S1) + bias, Q2, S2)

    ones = torch.ones(n, d, dtype=dtype, device=device)
    du = gq.mxfp4_gemm_dx(ones, Q2, S2, h)
    want = gq.mxfp4_gemm_dx(du, Q1, S1, d)
    dx, db = torch.autograd.grad(layers(x).sum(), (x, bias))            # an expanded gradient
    assert torch.equal(dx, want)
    assert torch.equal(db, du.sum(0))
    z = torch.cat([_rand(device, 3, seed=5, dtype=dtype), layers(x).flatten()])
    (dx,) = torch.autograd.grad(z, x, torch.ones_like(z))
    assert torch.equal(dx, want)
    with pytest.raises(B.GQError):
        gq.mxfp4_gemm(x.t().contiguous().t(), Q1, S1)                   # strided, as without a gradient


@pytest.mark.gpu
def test_backward_on_another_stream_and_in_a_graph(device):
    n, d_in, d_out = 40, 1024, 512
    Q, S = _weight(device, d_out, d_in)
    xs = [_rand(device, n, d_in, seed=i) for i in range(4)]
    g = _rand(device, n, d_out, seed=9)
    dx = gq.mxfp4_gemm_dx(g, Q, S, d_in)
    want = [gq.mxfp4_gemm(x, Q, S) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, y0 in zip(xs, want):
        leaf = x.clone().requires_grad_()
        side.wait_stream(torch.cuda.current_stream())
        y = gq.mxfp4_gemm(leaf, Q, S, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        (got,) = torch.autograd.grad(y, leaf, g)
        assert torch.equal(y.detach(), y0) and torch.equal(got, dx)
    # captured: the product and its gradient, of a leaf that no eager graph holds
    static = xs[0].clone().requires_grad_()
    weight = g.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gq.mxfp4_gemm(static, Q, S)
        (got,) = torch.autograd.grad(y, static, weight)
    for i, x in enumerate(xs[:3]):
        with torch.no_grad():
            static.copy_(x)
        weight.copy_(g * (i + 1))
        eager = gq.mxfp4_gemm_dx(weight, Q, S, d_in)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.detach(), want[i]) and torch.equal(got, eager)


@pytest.mark.gpu
def test_no_rows(device):
    Q, S = _weight(device, 64, 128)
    x = torch.empty(0, 128, device=device, requires_grad=True)
    gq.mxfp4_gemm(x, Q, S).sum().backward()
    assert x.grad.shape == (0, 128)


@pytest.mark.gpu
def test_a_weight_changed_before_the_backward_pass_is_noticed(device):
    """The graph holds the weight's tensors: torch refuses a backward pass over changed ones."""
    Q, S = _weight(device, 64, 128)
    x = _rand(device, 8, 128, seed=1).requires_grad_()
    y = gq.mxfp4_gemm(x, Q, S)
    S.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
